"""Window attention on the GPU against the fp64 definition, forward and backward; each case held to the bound that
oracle/attention_ops.py derives."""
import numpy as np
import pytest
import torch

from linear_attention_sequence_qkv_gb300 import build, gdn
from oracle import attention_ops as A

pytestmark = pytest.mark.gpu
ACT = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    build.build()
    gdn.load()
    return torch.device("cuda:0")


def n64(t):
    return t.detach().double().cpu().numpy()


def held(got, ref, err, dtype, what):
    got = n64(got).reshape(ref.shape)
    fine = np.isfinite(ref)
    assert np.array_equal(got[~fine], ref[~fine]), what
    tol = A.bound(ref[fine], err[fine], dtype)
    use = (np.abs(got[fine] - ref[fine]) / tol).max() if tol.size else 0.0
    print(f"[window] {dtype} {what}: bound_use={use:.3f}")
    assert use <= 1.0, (what, use)


def make(dev, B, Tq, Tk, Hq, Hk, d, dtype, pad=0, seed=0, q_std=2.0):
    """q, k, v as views into one buffer where their lengths agree, rows `pad` elements longer."""
    g = torch.Generator().manual_seed(seed + 1000 * Tq + 10 * Tk + d)
    randn = lambda t, c, std=1.0: (torch.randn((B, t, c + pad), generator=g) * std).to(ACT[dtype]).to(dev)  # noqa: E731
    if Tq == Tk:
        x = randn(Tq, (Hq + 2 * Hk) * d)
        q, k, v = x[..., pad:].split([Hq * d, Hk * d, Hk * d], dim=-1)
        q.mul_(q_std)
    else:
        q, k, v = randn(Tq, Hq * d, q_std)[..., pad:], randn(Tk, Hk * d)[..., pad:], randn(Tk, Hk * d)[..., pad:]
    dout = torch.randn((B, Tq, Hq * d), generator=g).to(ACT[dtype]).to(dev)
    return q, k, v, dout


def check(q, k, v, dout, f, g, spans, d, window, sinks, scale, dtype, heads=None):
    """Against the oracle, sequence by sequence: spans of (batch row, first query, queries, first key, keys)."""
    Hq, Hk = q.shape[-1] // d, k.shape[-1] // d
    T = q.shape[1]
    names = ("out",) if g is None else ("out", "dq", "dk", "dv")
    for b, q0, nq, k0, nk in spans:
        at = lambda x, r0, n: x[b, r0:r0 + n].reshape(n, x.shape[-1] // d, d)  # noqa: E731
        r = A.window_attention(n64(at(q, q0, nq)), n64(at(k, k0, nk)), n64(at(v, k0, nk)), window, sinks, scale, dtype,
                               None if g is None else n64(at(dout, q0, nq)))
        got = {"out": at(f.out, q0, nq)}
        if g is not None:
            got.update(dq=at(g.dq, q0, nq), dk=at(g.dk, k0, nk), dv=at(g.dv, k0, nk))
        for n in names:
            held(got[n], r[n], r[n + "_err"], dtype, n)
        if f.lse is not None:
            held(f.lse[:, b * T + q0:b * T + q0 + nq], r["lse"], r["lse_err"], "fp32", "lse")


def both(dev, B, Tq, Tk, Hq, Hk, d, window, sinks, dtype, pad=0, scale=None, backward=True):
    q, k, v, dout = make(dev, B, Tq, Tk, Hq, Hk, d, dtype, pad)
    kw = dict(d=d, window=window, sinks=sinks, scale=scale)
    f = gdn.window_attention_forward(q, k, v, **kw)
    g = gdn.window_attention_backward(q, k, v, f.out, f.lse, dout, **kw) if backward else None
    assert gdn.gdn_device_status(f.workspace) == gdn.GDN_OK
    assert g is None or gdn.gdn_device_status(g.workspace) == gdn.GDN_OK
    check(q, k, v, dout, f, g, [(b, 0, Tq, 0, Tk) for b in range(B)], d, window, sinks, f.desc.scale, dtype)


CASES = [  # B, Tq, Tk, Hq, Hk, d, window, sinks
    (1, 1, 1, 1, 1, 64, 1, 0), (1, 1, 1, 2, 1, 128, 8, 4), (2, 5, 5, 3, 1, 64, 2, 1), (1, 64, 64, 2, 2, 64, 16, 0),
    (1, 127, 127, 2, 1, 128, 50, 4), (2, 128, 128, 4, 2, 128, 128, 0), (1, 129, 129, 3, 3, 64, 1, 0), (1, 129, 129, 1, 1, 128, 1000, 7),
    (1, 300, 300, 4, 1, 128, 64, 4), (1, 300, 300, 2, 1, 64, 100, 130), (2, 257, 257, 6, 2, 80, 129, 3), (1, 500, 500, 8, 1, 96, 37, 1),
    (1, 700, 700, 2, 1, 128, 128, 300), (1, 600, 600, 5, 5, 72, 255, 64), (1, 1, 400, 4, 2, 128, 100, 4), (2, 3, 260, 4, 4, 64, 1000, 0),
    (1, 130, 400, 6, 2, 128, 200, 4), (1, 200, 330, 3, 1, 64, 17, 140), (1, 200, 70, 2, 1, 128, 30, 4), (1, 40, 1, 2, 1, 64, 3, 1),
    (1, 20, 0, 2, 1, 64, 3, 1), (1, 0, 20, 2, 1, 64, 3, 1), (1, 640, 640, 16, 2, 64, 160, 4), (1, 384, 384, 1, 1, 8, 130, 2)]


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("B,Tq,Tk,Hq,Hk,d,window,sinks", CASES)
def test_cases(dev, B, Tq, Tk, Hq, Hk, d, window, sinks, dtype):
    both(dev, B, Tq, Tk, Hq, Hk, d, window, sinks, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("d", [1, 7, 33, 100, 136, 200, 256])
def test_head_widths(dev, d, dtype):
    both(dev, 1, 150, 150, 4, 2, d, 40, 3, dtype)


@pytest.mark.parametrize("dtype,pad", [("bf16", 1), ("bf16", 4), ("fp16", 3), ("bf16", 8), ("fp32", 1), ("fp32", 2)])
def test_alignments(dev, dtype, pad):
    both(dev, 2, 140, 140, 4, 2, 64, 33, 2, dtype, pad=pad)


def test_scale_of_the_caller(dev):
    both(dev, 1, 200, 200, 2, 1, 128, 60, 4, "bf16", scale=0.2)


PACKED = [([0, 1, 5, 128, 129, 0, 300], None), ([3], None), ([1, 1, 1, 1, 1, 2], None), ([200, 0, 77, 256], [260, 5, 77, 900]),
          ([10, 130, 4], [0, 100, 9]), ([0, 0, 0, 6], None), ([400, 33], [400, 1])]


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("lengths,keys", PACKED)
@pytest.mark.parametrize("Hq,Hk,d,window,sinks", [(4, 2, 64, 50, 3), (3, 1, 128, 200, 130)])
def test_packed(dev, lengths, keys, Hq, Hk, d, window, sinks, dtype):
    keys_ = keys or lengths
    cuq, cuk = ([0] + np.cumsum(x).tolist() for x in (lengths, keys_))
    q, k, v, dout = make(dev, 1, cuq[-1], cuk[-1], Hq, Hk, d, dtype)
    kw = dict(d=d, window=window, sinks=sinks, cu_seqlens=torch.tensor(cuq, dtype=torch.int32, device=dev),
              cu_seqlens_k=torch.tensor(cuk, dtype=torch.int32, device=dev) if keys else None)
    f = gdn.window_attention_forward(q, k, v, **kw)
    g = gdn.window_attention_backward(q, k, v, f.out, f.lse, dout, **kw)
    assert gdn.gdn_device_status(f.workspace) == gdn.GDN_OK and gdn.gdn_device_status(g.workspace) == gdn.GDN_OK
    check(q, k, v, dout, f, g, [(0, cuq[n], lengths[n], cuk[n], keys_[n]) for n in range(len(lengths))], d, window, sinks,
          f.desc.scale, dtype)


@pytest.mark.parametrize("bad", [[0, 7, 9], [1, 5, 10], [0, 8, 5, 10], [0, 12, 10]])
def test_malformed_offsets_write_nothing(dev, bad):
    q, k, v, dout = make(dev, 1, 10, 10, 2, 1, 64, "bf16")
    cu = torch.tensor(bad, dtype=torch.int32, device=dev)
    kw = dict(d=64, window=4, sinks=1, cu_seqlens=cu)
    f = gdn.alloc_window_attention(gdn.window_attention_desc_for(q, k, v, **kw), dev)
    f.out.fill_(7), f.lse.fill_(7)
    gdn.window_attention_forward(q, k, v, bufs=f, **kw)
    assert gdn.gdn_device_status(f.workspace) == gdn.GDN_ERR_DEVICE_SEQLENS
    assert bool((f.out == 7).all()) and bool((f.lse == 7).all())
    g = gdn.alloc_window_attention_grads(f.desc, dev)
    for t in (g.dq, g.dk, g.dv):
        t.fill_(7)
    gdn.window_attention_backward(q, k, v, f.out, f.lse, dout, grads=g, **kw)
    assert gdn.gdn_device_status(g.workspace) == gdn.GDN_ERR_DEVICE_SEQLENS
    assert all(bool((t == 7).all()) for t in (g.dq, g.dk, g.dv))


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("fp16", 64), ("fp32", 64), ("bf16", 100)])
@pytest.mark.parametrize("poison", [float("nan"), float("inf"), float("-inf")])
def test_what_is_not_seen_has_no_influence(dev, dtype, d, poison):
    """Keys and values after a query, before its window and of other sequences may be anything."""
    lengths, window, sinks = [150, 60, 200], 40, 2
    cu = torch.tensor([0] + list(np.cumsum(lengths)), dtype=torch.int32, device=dev)
    q, k, v, _ = make(dev, 1, sum(lengths), sum(lengths), 4, 2, d, dtype)
    kw = dict(d=d, window=window, sinks=sinks, cu_seqlens=cu)
    clean = gdn.window_attention_forward(q, k, v, **kw)
    bad = [149, 150 + 30, 210 + 100]   # the last of one sequence, one inside each of the others
    for t in bad:
        k[0, t], v[0, t] = poison, poison
    got = gdn.window_attention_forward(q, k, v, **kw)
    hit = torch.zeros(sum(lengths), dtype=torch.bool, device=dev)
    hit[149:150] = True
    hit[180:210] = True
    hit[310:350] = True
    same = (got.out == clean.out)[0].all(-1)
    assert bool(same[~hit].all()), (~same & ~hit).nonzero()[:10].flatten().tolist()
    assert not bool(torch.isfinite(got.out[0, 149]).any())


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("fp16", 64), ("fp32", 64)])
def test_gradients_of_other_sequences_stay_clean(dev, dtype, d):
    lengths = [150, 60, 200]
    cu = torch.tensor([0] + list(np.cumsum(lengths)), dtype=torch.int32, device=dev)
    q, k, v, dout = make(dev, 1, sum(lengths), sum(lengths), 4, 2, d, dtype)
    kw = dict(d=d, window=40, sinks=2, cu_seqlens=cu)
    f = gdn.window_attention_forward(q, k, v, **kw)
    clean = gdn.window_attention_backward(q, k, v, f.out, f.lse, dout, **kw)
    for x in (q, k, v, dout):
        x[0, 150:210] = float("nan")
    f = gdn.window_attention_forward(q, k, v, **kw)
    got = gdn.window_attention_backward(q, k, v, f.out, f.lse, dout, **kw)
    for n in ("dq", "dk", "dv"):
        a, b = getattr(got, n)[0], getattr(clean, n)[0]
        assert torch.equal(a[:150], b[:150]) and torch.equal(a[210:], b[210:]), n


def test_large_scores_and_equal_ones(dev):
    """Scores of a few hundred, all equal scores, and one key far above the others."""
    q, k, v, dout = make(dev, 1, 300, 300, 2, 1, 128, "bf16")
    kw = dict(d=128, window=90, sinks=4)
    for change in (lambda: q.mul_(20.0), lambda: k.zero_(), lambda: k[:, 7::50].fill_(6.0)):
        change()
        f = gdn.window_attention_forward(q, k, v, **kw)
        g = gdn.window_attention_backward(q, k, v, f.out, f.lse, dout, **kw)
        check(q, k, v, dout, f, g, [(0, 0, 300, 0, 300)], 128, 90, 4, f.desc.scale, "bf16")


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("fp16", 64), ("fp32", 96), ("bf16", 33)])
def test_run_to_run_identical_streams_and_graphs(dev, dtype, d):
    q, k, v, dout = make(dev, 2, 330, 330, 4, 2, d, dtype)
    kw = dict(d=d, window=100, sinks=5)
    f = gdn.window_attention_forward(q, k, v, **kw)
    g = gdn.window_attention_backward(q, k, v, f.out, f.lse, dout, **kw)
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    f2 = gdn.window_attention_forward(q, k, v, stream=other, **kw)
    g2 = gdn.window_attention_backward(q, k, v, f2.out, f2.lse, dout, stream=other, **kw)
    torch.cuda.current_stream().wait_stream(other)
    f3, g3 = gdn.alloc_window_attention(f.desc, dev), gdn.alloc_window_attention_grads(f.desc, dev)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gdn.window_attention_forward(q, k, v, bufs=f3, **kw)
        gdn.window_attention_backward(q, k, v, f3.out, f3.lse, dout, grads=g3, **kw)
    for _ in range(2):
        f3.out.zero_(), g3.dk.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in ((f, f2), (f, f3)):
            assert torch.equal(a.out, b.out) and torch.equal(a.lse, b.lse)
        for a, b in ((g, g2), (g, g3)):
            assert torch.equal(a.dq, b.dq) and torch.equal(a.dk, b.dk) and torch.equal(a.dv, b.dv)


def test_a_shared_key_row_and_no_lse(dev):
    """Batch rows that share one k and v (stride 0), and a forward without lse."""
    q, k, v, _ = make(dev, 3, 50, 50, 2, 1, 64, "bf16")
    k, v = k[:1].expand(3, -1, -1), v[:1].expand(3, -1, -1)
    f = gdn.window_attention_forward(q, k, v, d=64, window=20, want_lse=False)
    assert f.lse is None
    check(q, k, v, None, f, None, [(b, 0, 50, 0, 50) for b in range(3)], 64, 20, 0, f.desc.scale, "bf16")


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_guard_bands(dev, dtype):
    """Nothing is written around the outputs, and the inputs stay as they are."""
    q, k, v, dout = make(dev, 1, 133, 133, 3, 1, 64, dtype)
    kw = dict(d=64, window=30, sinks=2)
    big = {n: torch.full((133 + 20, c * 64), 7.0, dtype=ACT[dtype], device=dev) for n, c in (("out", 3), ("dq", 3), ("dk", 1), ("dv", 1))}
    view = {n: t[10:-10][None] for n, t in big.items()}
    r = gdn.window_attention_desc_for(q, k, v, **kw)
    f, g = gdn.alloc_window_attention(r, dev), gdn.alloc_window_attention_grads(r, dev)
    lse = torch.full((3 * 133 + 64,), 7.0, device=dev)
    f.out, f.lse = view["out"], lse[32:-32].view(3, 133)
    g.dq, g.dk, g.dv = view["dq"], view["dk"], view["dv"]
    before = [t.clone() for t in (q, k, v, dout)]
    gdn.window_attention_forward(q, k, v, bufs=f, **kw)
    gdn.window_attention_backward(q, k, v, f.out, f.lse, dout, grads=g, **kw)
    for t in big.values():
        assert bool((t[:10] == 7).all()) and bool((t[-10:] == 7).all())
    assert bool((lse[:32] == 7).all()) and bool((lse[-32:] == 7).all())
    assert all(torch.equal(a, b) for a, b in zip(before, (q, k, v, dout)))
    check(q, k, v, dout, f, g, [(0, 0, 133, 0, 133)], 64, 30, 2, r.scale, dtype)
