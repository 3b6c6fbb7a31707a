"""The operators of an attention layer as they are used together: head norms with rotary positions, window attention,
group norm over the heads' outputs; in training (packed sequences, gradients against torch's own differentiation of the
same chain in fp64), in serving (a prompt in pieces, then token by token, equals one pass), from host threads, in graphs,
with waits that run out, and over long sequences and large caches."""
import threading

import numpy as np
import pytest
import torch

from linear_attention_sequence_qkv_gb300 import build, gdn
from oracle import attention_ops as A

pytestmark = pytest.mark.gpu
ACT = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
HQ, HK, D, ROT, WINDOW, SINKS = 4, 2, 64, 32, 40, 3


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    build.build()
    gdn.load()
    return torch.device("cuda:0")


def make(dev, T, dtype, seed=0):
    g = torch.Generator().manual_seed(seed)
    randn = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    s = {"qkv": randn(1, T, (HQ + 2 * HK) * D).to(ACT[dtype]).to(dev), "dout": randn(T, 1, HQ * D).to(ACT[dtype]).to(dev)}
    s["q"], s["k"], s["v"] = s["qkv"].split([HQ * D, HK * D, HK * D], dim=-1)
    s["qw"], s["kw"] = ((1.0 + 0.1 * randn(D)).to(dev) for _ in range(2))
    s["nw"] = (1.0 + 0.1 * randn(HQ * D)).to(dev)
    s["table"] = gdn.rotary_table(ROT, device=dev)
    return s


ROTARY = dict(d=D, rot=ROT)
MASK = dict(d=D, window=WINDOW, sinks=SINKS)


def chain(s, cu=None):
    q, k = gdn.norm_rotary(s["q"], s["k"], s["qw"], s["kw"], s["table"], cu_seqlens=cu, **ROTARY)
    f = gdn.window_attention_forward(q, k, s["v"], cu_seqlens=cu, **MASK)
    o = f.out.view(-1, 1, HQ * D)
    return q, k, f, o, gdn.group_norm_forward(o, s["nw"], None, groups=HQ)


def chain_backward(s, q, k, f, o, n, cu=None):
    gn = gdn.group_norm_backward(o, s["nw"], None, n.mean, n.rstd, s["dout"], groups=HQ)
    ga = gdn.window_attention_backward(q, k, s["v"], f.out, f.lse, gn.dx.view(1, -1, HQ * D), cu_seqlens=cu, **MASK)
    return gn, ga, gdn.norm_rotary_backward(s["q"], s["k"], s["qw"], s["kw"], s["table"], ga.dq, ga.dk, cu_seqlens=cu, **ROTARY)


def reference(s, lengths):
    """(out, gradients of q, k, v and the weights) in fp64 by torch's differentiation."""
    leaf = {n: s[n].detach().cpu().double().requires_grad_(True) for n in ("q", "k", "v", "qw", "kw", "nw")}
    freq = torch.from_numpy(A.frequencies(ROT))

    def turn(x, w, pos):
        y = x.view(-1, x.shape[-1] // D, D)
        y = y / (y.pow(2).mean(-1, keepdim=True) + 1e-6).sqrt() * w
        a = pos[:, None].double() * freq
        c, si = a.cos()[:, None], a.sin()[:, None]
        y1, y2 = y[..., :ROT // 2], y[..., ROT // 2:ROT]
        return torch.cat([y1 * c - y2 * si, y2 * c + y1 * si, y[..., ROT:]], -1)

    rows, t = [], 0
    for L in lengths:
        p = torch.arange(L)
        q, k = turn(leaf["q"][0, t:t + L], leaf["qw"], p), turn(leaf["k"][0, t:t + L], leaf["kw"], p)
        v = leaf["v"][0, t:t + L].view(L, HK, D)
        see = torch.from_numpy(A.visible(L, L, WINDOW, SINKS))
        for h in range(0, HQ if L else 0):
            x = (q[:, h] @ k[:, h // (HQ // HK)].T) * D ** -0.5
            rows.append((t, h, torch.softmax(x.masked_fill(~see, -torch.inf), -1) @ v[:, h // (HQ // HK)]))
        t += L
    o = torch.zeros(t, HQ, D, dtype=torch.float64)
    for t0, h, x in rows:
        o = o.index_put((torch.arange(t0, t0 + x.shape[0]), torch.tensor(h)), x)
    var, mean = torch.var_mean(o, dim=-1, keepdim=True, correction=0)
    z = ((o - mean) / (var + 1e-5).sqrt()).reshape(t, 1, HQ * D) * leaf["nw"]
    out = torch.nn.functional.silu(z)
    return out.detach(), torch.autograd.grad(out, list(leaf.values()), s["dout"].cpu().double())


@pytest.mark.parametrize("dtype,tol", [("fp32", 1e-4), ("bf16", 5e-2), ("fp16", 7e-3)])
def test_training_step(dev, dtype, tol):
    """Tolerance relative to each result's 2-norm: per operator a rounding of its operands and of its result (2^-8, 2^-11 or
    2^-24 at most each, four operators with two of them), magnified by the group norm, whose rows of few keys' averages have
    an rstd of up to about 3, and by the gradients' second use of the rounded values: 8 x 2 x 3 of half that step on
    average, which is 1.5 2^-5 in bf16."""
    lengths = [70, 1, 0, 200, 33, 129]
    s = make(dev, sum(lengths), dtype)
    cu = torch.tensor([0] + np.cumsum(lengths).tolist(), dtype=torch.int32, device=dev)
    q, k, f, o, n = chain(s, cu)
    gn, ga, gr = chain_backward(s, q, k, f, o, n, cu)
    out, want = reference(s, lengths)
    off = lambda got, w: float((got.cpu().double().reshape(w.shape) - w).norm() / w.norm())  # noqa: E731
    got = {"out": off(n.out, out)}
    for name, g, w in zip(("q", "k", "v", "qw", "kw", "nw"), (gr.dq, gr.dk, ga.dv, gr.dq_weight, gr.dk_weight, gn.dweight), want):
        got[name] = off(g, w)
    print("[attention layer]", dtype, {k: f"{v:.2g}" for k, v in got.items()})
    assert all(v <= tol for v in got.values()), got


@pytest.mark.parametrize("dtype,tol", [("fp32", 2e-5), ("bf16", 2e-2)])
def test_prompt_in_pieces_then_tokens(dev, dtype, tol):
    """The same chain up to the attention's output: every row against the pass over the whole sequence, whose operands
    are the same bits (a norm or a rotation does not depend on what else is in its call) and whose sums are in another
    order: two results, each within an operand rounding of P (2^-8) and a rounding (2^-8) of the exact one."""
    T = 150
    s = make(dev, T, dtype, seed=4)
    whole = chain(s)[2].out
    cache = gdn.alloc_window_cache(1, HK, D, window=WINDOW, sinks=SINKS, dtype=ACT[dtype], device=dev)
    past_k, rows = [], []
    for a, b in ((0, 1), (1, 64), (64, 100)):
        off = cache.lengths.clone()
        q, k = gdn.norm_rotary(s["q"][:, a:b], s["k"][:, a:b], s["qw"], s["kw"], s["table"], offsets=off, **ROTARY)
        past_k.append(k)
        rows.append(gdn.window_attention_forward(q, torch.cat(past_k, 1), s["v"][:, :b], **MASK).out)
        gdn.window_cache_write(k, s["v"][:, a:b], cache)
        cache.lengths += b - a
    for t in range(100, T):
        q, k = gdn.norm_rotary(s["q"][:, t:t + 1], s["k"][:, t:t + 1], s["qw"], s["kw"], s["table"], offsets=cache.lengths, **ROTARY)
        rows.append(gdn.window_attention_step(q, k, s["v"][:, t:t + 1], cache))
        cache.lengths += 1
    got = torch.cat(rows, 1)
    scale = whole.float().abs().clamp(min=whole.float().abs().mean().item())
    assert float(((got - whole).float().abs() / scale).max()) <= tol * 4
    assert float((got - whole).float().norm() / whole.float().norm()) <= tol


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("fp16", 64)])
def test_waits_that_run_out_are_reported_and_leave_nothing(dev, dtype, d):
    g = torch.Generator().manual_seed(3)
    q, k, v, do = ((torch.randn((1, 600, h * d), generator=g)).to(ACT[dtype]).to(dev) for h in (4, 2, 2, 4))
    kw = dict(d=d, window=100, sinks=4)
    f = gdn.window_attention_forward(q, k, v, **kw)
    r = gdn.window_attention_backward(q, k, v, f.out, f.lse, do, **kw)
    want = [t.clone() for t in (f.out, f.lse, r.dq, r.dk, r.dv)]
    gdn.gdn_set_wait_test_mode(1)
    try:
        gdn.window_attention_forward(q, k, v, bufs=f, **kw)
        assert gdn.gdn_device_status(f.workspace) == gdn.GDN_ERR_DEVICE_TIMEOUT
        gdn.window_attention_backward(q, k, v, want[0], want[1], do, grads=r, **kw)
        assert gdn.gdn_device_status(r.workspace) == gdn.GDN_ERR_DEVICE_TIMEOUT
    finally:
        gdn.gdn_set_wait_test_mode(0)
    gdn.window_attention_forward(q, k, v, bufs=f, **kw)
    gdn.window_attention_backward(q, k, v, f.out, f.lse, do, grads=r, **kw)
    assert gdn.gdn_device_status(f.workspace) == gdn.GDN_OK and gdn.gdn_device_status(r.workspace) == gdn.GDN_OK
    assert all(torch.equal(a, b) for a, b in zip((f.out, f.lse, r.dq, r.dk, r.dv), want))


def test_two_host_threads(dev):
    """Each with a stream, its own sizes and buffers, its first CUDA calls among them: the results of calls on their own."""
    jobs = []
    for dtype, d, T, window in (("bf16", 128, 300, 64), ("fp32", 64, 200, 30)):
        g = torch.Generator().manual_seed(d)
        q, k, v, do = (torch.randn((1, T, h * d), generator=g).to(ACT[dtype]).to(dev) for h in (4, 2, 2, 4))
        jobs.append((q, k, v, do, dict(d=d, window=window, sinks=2)))

    def once(job, stream=None):
        q, k, v, do, kw = job
        f = gdn.window_attention_forward(q, k, v, stream=stream, **kw)
        r = gdn.window_attention_backward(q, k, v, f.out, f.lse, do, stream=stream, **kw)
        return f.out, r.dq, r.dk, r.dv

    want = [once(j) for j in jobs]
    torch.cuda.synchronize()
    errors = []

    def work(job, ref):
        try:
            torch.cuda.set_device(dev)
            stream = torch.cuda.Stream()
            for _ in range(30):
                got = once(job, stream)
                stream.synchronize()
                if not all(torch.equal(a, b) for a, b in zip(got, ref)):
                    errors.append("differs")
        except Exception as e:
            errors.append(repr(e))

    threads = [threading.Thread(target=work, args=a) for a in zip(jobs, want)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors


@pytest.mark.parametrize("sinks,Hq,Hk,d", [(5, 2, 1, 64), (200, 3, 1, 128), (0, 2, 2, 128)])
def test_long_sequences_agree_with_the_fp32_kernels(dev, sinks, Hq, Hk, d):
    """Many chunks of the sinks' rest, through the tensor cores and through the fp32 kernels (held to the oracle at sizes
    that it can do) on the same 16-bit values. P, dS and the results are rounded to 16 bits on one side: 3 x 2^-9 relative
    in the mean, 2e-2 allowed for the 2-norm of the difference."""
    T, window = 20000, 300
    g = torch.Generator().manual_seed(sinks)
    q, k, v, do = (torch.randn((1, T, h * d), generator=g).to(torch.bfloat16).to(dev) for h in (Hq, Hk, Hk, Hq))
    kw = dict(d=d, window=window, sinks=sinks)
    res = []
    for cast in (lambda x: x, lambda x: x.float()):
        a = [cast(x) for x in (q, k, v, do)]
        f = gdn.window_attention_forward(*a[:3], **kw)
        r = gdn.window_attention_backward(*a[:3], f.out, f.lse, a[3], **kw)
        assert gdn.gdn_device_status(r.workspace) == gdn.GDN_OK
        res.append((f.out, f.lse, r.dq, r.dk, r.dv))
    for n, a, b in zip(("out", "lse", "dq", "dk", "dv"), *res):
        off = float((a.double() - b.double()).norm() / b.double().norm())
        top = b.float()[:, :max(sinks, 1)] if n in ("dk", "dv") else None   # the sinks' own rows too
        if top is not None:
            off = max(off, float((a.double()[:, :top.shape[1]] - top.double()).norm() / top.double().norm()))
        print("[long]", n, off)
        assert off <= 2e-2, (n, off)


def test_cache_of_more_than_2_31_elements(dev):
    """Slots far behind 2^31 elements: the last sequence's rows of a cache of 2.3e9 elements."""
    N, Hk, d, window, sinks, slack = 3, 2, 128, 70, 2, 3000000
    cache = gdn.alloc_window_cache(N, Hk, d, window=window, sinks=sinks, slots=sinks + window + slack, device=dev)
    assert cache.k.numel() > 1 << 31
    g = torch.Generator().manual_seed(8)
    far = slack + 50   # near the ring's end, so that the window's slots go round it
    cache.lengths.fill_(far)
    k, v = (torch.randn((N, 100, Hk * d), generator=g).to(torch.bfloat16).to(dev) for _ in range(2))
    q, kn, vn = (torch.randn((N, 1, h * d), generator=g).to(torch.bfloat16).to(dev) for h in (4, Hk, Hk))
    first = (torch.randn((N, sinks, Hk * d), generator=g).to(torch.bfloat16).to(dev) for _ in range(2))
    start = gdn.WindowCache(cache.k, cache.v, torch.zeros_like(cache.lengths), window, sinks)
    fk, fv = first
    gdn.window_cache_write(fk, fv, start)
    gdn.window_cache_write(k, v, cache)
    cache.lengths += 100
    out = gdn.window_attention_step(q, kn, vn, cache)
    n64 = lambda x, h: x.double().cpu().numpy().reshape(N, -1, h, d)  # noqa: E731
    K = np.concatenate([n64(fk, Hk), n64(k, Hk)[:, 100 - window + 1:], n64(kn, Hk)], 1)
    V = np.concatenate([n64(fv, Hk), n64(v, Hk)[:, 100 - window + 1:], n64(vn, Hk)], 1)
    for n in range(N):
        r = A.window_attention(n64(q, 4)[n], K[n], V[n], K.shape[1], 0, d ** -0.5, "bf16")
        use = (np.abs(n64(out, 4)[n] - r["out"]) / A.bound(r["out"], r["out_err"], "bf16")).max()
        assert use <= 1.0, (n, use)
