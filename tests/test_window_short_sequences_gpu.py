"""Gradients of the window attention's short sequences: a query that sees one key has none for q and k, exactly; and where a few
keys share the weight, dP - delta cancels, so that delta is not to come from the rounded output."""
import numpy as np
import pytest
import torch

from linear_attention_sequence_qkv_gb300 import gdn
from oracle import attention_ops as A
from test_window_attention_gpu import ACT, dev, make, n64  # noqa: F401

pytestmark = pytest.mark.gpu


def both(q, k, v, dout, kw):
    f = gdn.window_attention_forward(q, k, v, **kw)
    return f, gdn.window_attention_backward(q, k, v, f.out, f.lse, dout, **kw)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("B,T,Hq,Hk,d,window", [(1, 1, 1, 1, 64, 16), (3, 1, 4, 2, 128, 1), (2, 1, 3, 1, 96, 1000), (2, 200, 4, 2, 128, 1), (1, 300, 3, 1, 64, 1),
                                                (1, 70, 2, 2, 40, 1), (2, 50, 2, 1, 33, 1)])
def test_one_key(dev, B, T, Hq, Hk, d, window, dtype):  # noqa: F811
    q, k, v, dout = make(dev, B, T, T, Hq, Hk, d, dtype)
    f, g = both(q, k, v, dout, dict(d=d, window=window, sinks=0))
    assert torch.equal(f.out.view(B, T, Hk, -1, d), v.reshape(B, T, Hk, 1, d).expand(B, T, Hk, Hq // Hk, d))
    assert not g.dq.any() and not g.dk.any()
    want = n64(dout).reshape(B, T, Hk, -1, d).sum(3).reshape(B, T, -1)   # P is 1 up to a few of fp32's roundings
    assert (np.abs(n64(g.dv) - want) <= A.bound(want, 2.0 ** -18 * np.abs(n64(dout)).reshape(B, T, Hk, -1, d).sum(3).reshape(B, T, -1), dtype)).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_first_queries_of_sequences(dev, dtype):  # noqa: F811
    """dq of a sequence's first query is 0 whatever follows, with queries that follow a past it is not the first any more."""
    lengths, keys = [1, 5, 1, 140, 1, 2], [1, 5, 4, 140, 0, 1]
    cuq, cuk = ([0] + np.cumsum(x).tolist() for x in (lengths, keys))
    q, k, v, dout = make(dev, 1, cuq[-1], cuk[-1], 4, 2, 64, dtype)
    cu = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)  # noqa: E731
    f, g = both(q, k, v, dout, dict(d=64, window=30, sinks=1, cu_seqlens=cu(cuq), cu_seqlens_k=cu(cuk)))
    zero = [cuq[0], cuq[1], cuq[3], cuq[4], cuq[5], cuq[5] + 1]   # sees one key, or none
    some = [t for t in range(cuq[-1]) if t not in zero]
    assert not g.dq[0, zero].any() and bool(g.dq[0, some].any(-1).all())
    assert not g.dk[0, cuk[0]].any() and not g.dk[0, cuk[5]].any()


def few_keys(q, k, v, dout, window, sinks, scale, dtype):
    """dq and dk with bounds that hold delta to fp32: the oracle's for fp32, and what rounding dS to the type adds, half a step of each
    value (2^-7 more for what was rounded before) and the least that fp16 keeps of it (see the oracle)."""
    r = A.window_attention(q, k, v, window, sinks, scale, "fp32", dout)
    rel, least = A.HALF_STEP[dtype]
    see, G = A.visible(q.shape[0], k.shape[0], window, sinks), q.shape[1] // k.shape[1]
    eq, ek = np.zeros(q.shape), np.zeros(k.shape)
    for h in range(q.shape[1]):
        K, V, g = k[:, h // G], v[:, h // G], dout[:, h]
        s = np.where(see, scale * (q[:, h] @ K.T), -np.inf)
        w = np.where(see.any(1)[:, None], np.exp(s - np.where(see.any(1), s.max(1), 0.0)[:, None]), 0.0)
        P = w / np.where(see.any(1), w.sum(1), 1.0)[:, None]
        dP = g @ V.T
        b = 2 * np.sqrt((dout ** 2).sum(-1).max() * (v ** 2).sum(-1).max())
        e = rel * (1 + 2.0 ** -7) * scale * P * np.abs(dP - (P * dP).sum(1)[:, None]) + (least * scale * b * 2.0 ** -13 if dtype == "fp16" else least) * see
        eq[:, h] = e @ np.abs(K)
        ek[:, h // G] += e.T @ np.abs(q[:, h])
    return {"dq": (r["dq"], r["dq_err"] + eq), "dk": (r["dk"], r["dk_err"] + ek)}


def held_to_few(q, k, v, dout, g, spans, d, window, sinks, scale, dtype):
    worst = 0.0
    for b, q0, nq, k0, nk in spans:
        at = lambda x, r0, n: n64(x[b, r0:r0 + n].reshape(n, x.shape[-1] // d, d))  # noqa: E731
        r = few_keys(at(q, q0, nq), at(k, k0, nk), at(v, k0, nk), at(dout, q0, nq), window, sinks, scale, dtype)
        for n, x in (("dq", at(g.dq, q0, nq)), ("dk", at(g.dk, k0, nk))):
            worst = max(worst, (np.abs(x - r[n][0]) / A.bound(r[n][0], r[n][1], dtype)).max(initial=0.0))
    print(f"[short] {dtype} d={d} window={window} sinks={sinks}: bound_use={worst:.3f}")
    assert worst <= 1.0


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("Hq,Hk,d,window,sinks", [(4, 2, 64, 16, 0), (3, 3, 128, 100, 2), (6, 1, 96, 3, 0), (2, 2, 64, 2, 1), (2, 1, 33, 50, 0), (4, 4, 200, 5, 0), (3, 1, 128, 4, 8)])
@pytest.mark.parametrize("B,Tq,Tk", [(9, 2, 2), (5, 8, 8), (3, 3, 6), (4, 1, 8), (2, 1, 2), (3, 5, 3), (2, 7, 7)])
def test_few_keys(dev, B, Tq, Tk, Hq, Hk, d, window, sinks, dtype):  # noqa: F811
    """Every query sees at most 8 keys, far scores (a standard deviation of 4) among them."""
    q, k, v, dout = make(dev, B, Tq, Tk, Hq, Hk, d, dtype, q_std=4.0)
    f, g = both(q, k, v, dout, dict(d=d, window=window, sinks=sinks))
    held_to_few(q, k, v, dout, g, [(b, 0, Tq, 0, Tk) for b in range(B)], d, window, sinks, f.desc.scale, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_few_keys_of_packed_sequences(dev, dtype):  # noqa: F811
    """Sequences of 0 to 8 tokens beside long ones, whose later queries come from the output as before."""
    lengths = ([0, 1, 2, 3, 4, 5, 6, 7, 8] * 40 + [300]) * 2
    cuq = [0] + np.cumsum(lengths).tolist()
    q, k, v, dout = make(dev, 1, cuq[-1], cuq[-1], 4, 2, 128, dtype, q_std=4.0)
    f, g = both(q, k, v, dout, dict(d=128, window=64, sinks=2, cu_seqlens=torch.tensor(cuq, dtype=torch.int32, device=dev)))
    held_to_few(q, k, v, dout, g, [(0, cuq[n], lengths[n], cuq[n], lengths[n]) for n in range(len(lengths)) if 0 < lengths[n] <= 8], 128, 64, 2, f.desc.scale, dtype)
    assert gdn.gdn_device_status(g.workspace) == gdn.GDN_OK


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("fp16", 64), ("bf16", 33)])
def test_first_positions_do_not_see_what_is_masked(dev, dtype, d):  # noqa: F811
    """Keys that a first position does not see, of its sequence and of the next, may be anything."""
    lengths = [6, 5, 4]
    cu = torch.tensor([0, 6, 11, 15], dtype=torch.int32, device=dev)
    q, k, v, dout = make(dev, 1, 15, 15, 2, 1, d, dtype)
    kw = dict(d=d, window=2, sinks=0, cu_seqlens=cu)
    f, clean = both(q, k, v, dout, kw)
    for x in (q, k, v, dout):
        x[0, 6:11] = float("nan")
    f, g = both(q, k, v, dout, kw)
    for n in ("dq", "dk", "dv"):
        a, b = getattr(g, n)[0], getattr(clean, n)[0]
        assert torch.equal(a[:6], b[:6]) and torch.equal(a[11:], b[11:]), n


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("fp16", 64), ("fp16", 33)])
def test_short_sequences_in_a_graph_and_on_another_stream(dev, dtype, d):  # noqa: F811
    lengths = [1, 2, 30, 0, 7, 64, 65, 3]
    cuq = [0] + np.cumsum(lengths).tolist()
    q, k, v, dout = make(dev, 1, cuq[-1], cuq[-1], 4, 2, d, dtype)
    kw = dict(d=d, window=10, sinks=1, cu_seqlens=torch.tensor(cuq, dtype=torch.int32, device=dev))
    f, g = both(q, k, v, dout, kw)
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    g2 = gdn.window_attention_backward(q, k, v, f.out, f.lse, dout, stream=other, **kw)
    torch.cuda.current_stream().wait_stream(other)
    g3 = gdn.alloc_window_attention_grads(f.desc, dev)
    graph, first = torch.cuda.CUDAGraph(), dout.clone()
    with torch.cuda.graph(graph):
        gdn.window_attention_backward(q, k, v, f.out, f.lse, dout, grads=g3, **kw)
    for size in (1.0, 2.0 ** -5, 1.0):   # what one replay found of the inputs' sizes does not stay for the next
        dout.copy_(first * size)
        graph.replay()
        torch.cuda.synchronize()
    for n in ("dq", "dk", "dv"):
        assert torch.equal(getattr(g, n), getattr(g2, n)) and torch.equal(getattr(g, n), getattr(g3, n)), n
