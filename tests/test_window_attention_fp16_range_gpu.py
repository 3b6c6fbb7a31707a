"""What fp16's range does to the window attention's 16-bit operands: weights far below a row's largest, and gradients of any
size, against the fp64 definition. The oracle's bounds count a rounding of P and of dS relative to their values; how far below
fp16's smallest they may fall it takes from the operands' powers of two (oracle/attention_ops.py)."""
import numpy as np
import pytest
import torch

from linear_attention_sequence_qkv_gb300 import gdn
from oracle import attention_ops as A
from test_window_attention_gpu import check, dev, held, make, n64  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("size", [1.0, 2.0 ** -7, 2.0 ** -13, 2.0 ** -17, 2.0 ** 9])
@pytest.mark.parametrize("B,T,Hq,Hk,d,window,sinks", [(1, 700, 4, 2, 128, 300, 4), (1, 520, 3, 1, 64, 2000, 0), (2, 300, 2, 2, 96, 64, 140), (1, 900, 2, 1, 128, 1700, 0)])
def test_gradients_of_any_size(dev, B, T, Hq, Hk, d, window, sinks, size):  # noqa: F811
    """dq with keys, then dk with queries so large (their partner so small) that results of small gradients are fp16's normal values."""
    for large in ("k", "q"):
        q, k, v, dout = make(dev, B, T, T, Hq, Hk, d, "fp16", q_std=1.0)
        up = 64.0 if size <= 1.0 else 2.0 ** -7
        (k if large == "k" else q).mul_(up)
        (q if large == "k" else k).mul_(1.0 / up)
        dout.mul_(size)
        kw = dict(d=d, window=window, sinks=sinks)
        f = gdn.window_attention_forward(q, k, v, **kw)
        g = gdn.window_attention_backward(q, k, v, f.out, f.lse, dout, **kw)
        for b in range(B):
            at = lambda x: x[b].reshape(T, -1, d)  # noqa: E731
            r = A.window_attention(n64(at(q)), n64(at(k)), n64(at(v)), window, sinks, f.desc.scale, "fp16", n64(at(dout)))
            for n in ("dq", "dv") if large == "k" else ("dk", "dv"):
                held(at(getattr(g, n)), r[n], r[n + "_err"], "fp16", f"{n} of gradients of {size}")


@pytest.mark.parametrize("size", [2.0 ** -10, 2.0 ** -16])
def test_the_norm_of_the_difference(dev, size):  # noqa: F811
    """dq and dk over 1000 keys in the 2-norm. dS (relative 2^-11 at most, uniform: 2^-11 / sqrt 3 at most in the root mean square),
    q or k exact, delta from the rounded output (another such rounding, of one sum for all keys of a row), the result's rounding:
    below 3 2^-11 together, whatever the size."""
    T, d = 1000, 128
    q, k, v, dout = make(dev, 1, T, T, 4, 2, d, "fp16", q_std=1.0)
    k.mul_(512.0), q.mul_(1 / 512.0)   # dq of normal values
    dout.mul_(size)
    kw = dict(d=d, window=T, sinks=0)
    f = gdn.window_attention_forward(q, k, v, **kw)
    g = gdn.window_attention_backward(q, k, v, f.out, f.lse, dout, **kw)
    at = lambda x: n64(x[0].reshape(T, -1, d))  # noqa: E731
    r = A.window_attention(at(q), at(k), at(v), T, 0, f.desc.scale, "fp16", at(dout))
    rel = np.linalg.norm(at(g.dq) - r["dq"]) / np.linalg.norm(r["dq"])
    print(f"[window] fp16 gradients of {size}: dq off by {rel:.2e}")
    assert rel <= 3 * 2.0 ** -11


def test_gradients_whose_products_pass_fp16s_largest(dev):  # noqa: F811
    """Two far values and a large gradient: dS reaches 10^5, dq stays small because k is."""
    q, k, v, dout = make(dev, 1, 40, 40, 2, 1, 64, "fp16", q_std=1.0)
    q.mul_(2.0 ** 7), k.mul_(2.0 ** -7), v.mul_(1000.0), dout.mul_(500.0)
    kw = dict(d=64, window=40, sinks=0)
    f = gdn.window_attention_forward(q, k, v, **kw)
    g = gdn.window_attention_backward(q, k, v, f.out, f.lse, dout, **kw)
    at = lambda x: n64(x[0].reshape(40, -1, 64))  # noqa: E731
    r = A.window_attention(at(q), at(k), at(v), 40, 0, f.desc.scale, "fp16", at(dout))
    assert np.abs(r["dq"]).max() < 65504
    held(g.dq, r["dq"], r["dq_err"], "fp16", "dq of products beyond 65504")


def test_packed_sequences_of_gradients_of_different_sizes(dev):  # noqa: F811
    """Each sequence by its own sizes: what one holds changes no bit of another's gradients, and zeros stay zeros."""
    lengths = [150, 60, 200, 90]
    at = np.cumsum([0] + lengths)
    cu = torch.tensor(at, dtype=torch.int32, device=dev)
    q, k, v, dout = make(dev, 1, 500, 500, 4, 2, 128, "fp16", q_std=1.0)
    k.mul_(64.0), q.mul_(1 / 64.0)
    for n, size in enumerate((2.0 ** -14, 1.0, 2.0 ** -8, 0.0)):
        dout[0, at[n]:at[n + 1]] *= size
    kw = dict(d=128, window=70, sinks=2, cu_seqlens=cu)
    f = gdn.window_attention_forward(q, k, v, **kw)
    g = gdn.window_attention_backward(q, k, v, f.out, f.lse, dout, **kw)
    for n, m in enumerate(lengths):
        rows = lambda x: x[0, at[n]:at[n + 1]].reshape(m, -1, 128)  # noqa: E731
        r = A.window_attention(n64(rows(q)), n64(rows(k)), n64(rows(v)), 70, 2, f.desc.scale, "fp16", n64(rows(dout)))
        for x in ("dq", "dv"):
            held(rows(getattr(g, x)), r[x], r[x + "_err"], "fp16", f"{x} of sequence {n}")
    dout[0, 150:210] *= 2.0 ** 10
    v[0, 170] *= 100.0
    f = gdn.window_attention_forward(q, k, v, **kw)
    h = gdn.window_attention_backward(q, k, v, f.out, f.lse, dout, **kw)
    for x in ("dq", "dk", "dv"):
        a, b = getattr(g, x)[0], getattr(h, x)[0]
        assert torch.equal(a[:150], b[:150]) and torch.equal(a[210:], b[210:]), x
    assert not g.dq[0, 410:].any() and not g.dk[0, 410:].any() and not g.dv[0, 410:].any()


def test_a_value_that_is_not_finite_leaves_other_rows_their_precision(dev):  # noqa: F811
    """The sizes are taken over what is finite: rows that do not see the NaN keep their gradients' exactness."""
    q, k, v, dout = make(dev, 1, 300, 300, 2, 1, 64, "fp16", q_std=1.0)
    k.mul_(64.0), q.mul_(1 / 64.0), dout.mul_(2.0 ** -13)
    dout[0, 290] *= 0.25
    kw = dict(d=64, window=40, sinks=0)
    f = gdn.window_attention_forward(q, k, v, **kw)
    clean = gdn.window_attention_backward(q, k, v, f.out, f.lse, dout, **kw)
    dout[0, 290, 5] = float("inf")
    g = gdn.window_attention_backward(q, k, v, f.out, f.lse, dout, **kw)
    assert torch.equal(g.dq[0, :128], clean.dq[0, :128])   # the tiles of queries in which the row is not


@pytest.mark.parametrize("packed", [False, True])
def test_many_short_sequences_each_of_its_own_size(dev, packed):  # noqa: F811
    """More sequences and heads in a CTA's rows than it has shared words for."""
    N, T, H, d = 32768, 2, 32, 8
    g = torch.Generator(device=dev).manual_seed(3)
    randn = lambda: torch.randn((N, T, H * d), generator=g, device=dev, dtype=torch.float16)  # noqa: E731
    q, k, v, dout = randn() / 64, randn() * 64, randn(), randn()
    dout *= 2.0 ** -torch.randint(0, 15, (N, 1, 1), generator=g, device=dev).to(torch.float16)
    kw = dict(d=d, window=2, sinks=0)
    if packed:
        q, k, v, dout = (x.view(1, N * T, H * d) for x in (q, k, v, dout))
        kw["cu_seqlens"] = torch.arange(0, N * T + 1, T, dtype=torch.int32, device=dev)
    f = gdn.window_attention_forward(q, k, v, **kw)
    grads = gdn.window_attention_backward(q, k, v, f.out, f.lse, dout, **kw)
    for n in list(range(0, N, 1111)) + [N - 1]:
        at = lambda x: n64(x.view(N, T, H, d)[n])  # noqa: E731
        r = A.window_attention(at(q), at(k), at(v), 2, 0, f.desc.scale, "fp16", at(dout))
        for x in ("dq", "dv"):
            tol = A.bound(r[x], r[x + "_err"], "fp16")
            assert (np.abs(at(getattr(grads, x)) - r[x]) <= tol).all(), (x, n)


def far_weights(dev, Tk, dtype="fp16"):
    """One key of score 0 whose value is 0, all others of score -17.5 and value 1: their weights of 2.5e-8 are below half of
    fp16's smallest value, and add up to Tk 2.5e-8."""
    act = {"fp16": torch.float16, "bf16": torch.bfloat16}[dtype]
    q, k, v = (torch.zeros((1, n, 64), dtype=act, device=dev) for n in (2, Tk, Tk))
    q[..., 0] = 1.0
    k[:, 1:, 0], v[:, 1:] = -17.5, 1.0
    return q, k, v


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_many_small_weights(dev, dtype):  # noqa: F811
    Tk = 40000
    q, k, v = far_weights(dev, Tk, dtype)
    dout = torch.randn(q.shape, generator=torch.Generator().manual_seed(1)).to(q.dtype).to(dev) * 4096.0
    kw = dict(d=64, window=Tk, sinks=0, scale=1.0)
    f = gdn.window_attention_forward(q, k, v, **kw)
    g = gdn.window_attention_backward(q, k, v, f.out, f.lse, dout, **kw)
    check(q, k, v, dout, f, g, [(0, 0, 2, 0, Tk)], 64, Tk, 0, 1.0, dtype)


@pytest.mark.parametrize("group", [1, 12])
def test_many_small_weights_in_a_step(dev, group):  # noqa: F811
    """As many sequences as leave each to one CTA, and a key of score 0 for each of its warps, so that all of the others are small."""
    N, Hk, Tk, d = 38, 8, 40000, 8
    c = gdn.alloc_window_cache(N, Hk, d, window=Tk, dtype=torch.float16, device=dev)
    c.k.zero_(), c.v.fill_(1.0)
    c.k[..., 0] = -17.5
    c.k[:, :, 0:64:16], c.v[:, :, 0:64:16] = 0.0, 0.0
    c.lengths.fill_(Tk - 1)
    q = torch.zeros((N, 1, group * Hk, d), dtype=torch.float16, device=dev)
    q[..., 0] = 1.0
    k, v = c.k[:, :, -1].reshape(N, 1, Hk * d), c.v[:, :, -1].reshape(N, 1, Hk * d)
    got = gdn.window_attention_step(q.view(N, 1, -1), k, v, c, scale=1.0)
    r = A.window_attention(n64(q[0, :, :1]), n64(c.k[0, 0])[:, None], n64(c.v[0, 0])[:, None], Tk, 0, 1.0, "fp16")
    wide = lambda x: np.broadcast_to(x, (N, group * Hk, d))  # noqa: E731
    held(got, wide(r["out"]), wide(r["out_err"]), "fp16", "step over many small weights")
