"""The sinks' queries beyond the window in the window attention's backward: many tiles of sinks, packed sequences of which only
some have such queries, chunks that the plan makes longer."""
import numpy as np
import pytest
import torch

from linear_attention_sequence_qkv_gb300 import gdn
from test_window_attention_gpu import ACT, check, dev, make  # noqa: F401

pytestmark = pytest.mark.gpu


def both(q, k, v, dout, kw):
    f = gdn.window_attention_forward(q, k, v, **kw)
    g = gdn.window_attention_backward(q, k, v, f.out, f.lse, dout, **kw)
    assert gdn.gdn_device_status(g.workspace) == gdn.GDN_OK
    again = gdn.window_attention_backward(q, k, v, f.out, f.lse, dout, **kw)
    assert all(torch.equal(getattr(g, n), getattr(again, n)) for n in ("dq", "dk", "dv"))
    return f, g


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("B,Tq,Tk,Hq,Hk,d,window,sinks", [(2, 1500, 1500, 4, 2, 64, 40, 700), (1, 1000, 1700, 2, 2, 128, 300, 5000),
                                                          (1, 1300, 900, 3, 1, 64, 1, 257), (3, 1281, 1281, 2, 1, 128, 640, 512)])
def test_many_tiles_of_sinks(dev, B, Tq, Tk, Hq, Hk, d, window, sinks, dtype):  # noqa: F811
    q, k, v, dout = make(dev, B, Tq, Tk, Hq, Hk, d, dtype)
    f, g = both(q, k, v, dout, dict(d=d, window=window, sinks=sinks))
    check(q, k, v, dout, f, g, [(b, 0, Tq, 0, Tk) for b in range(B)], d, window, sinks, f.desc.scale, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("lengths,keys", [([900, 0, 30, 1300, 129, 1, 500], None), ([100, 5, 700, 0, 300], [900, 700, 700, 600, 100]),
                                          ([1, 2, 3, 4, 5] * 250 + [1000] + [3] * 1200 + [700], None), ([40] * 60, None), ([800], None)])
@pytest.mark.parametrize("Hq,Hk,d,window,sinks", [(4, 2, 64, 50, 300), (3, 1, 128, 130, 4)])
def test_packed_sequences_with_and_without(dev, lengths, keys, Hq, Hk, d, window, sinks, dtype):  # noqa: F811
    keys_ = keys or lengths
    cuq, cuk = ([0] + np.cumsum(x).tolist() for x in (lengths, keys_))
    q, k, v, dout = make(dev, 1, cuq[-1], cuk[-1], Hq, Hk, d, dtype)
    kw = dict(d=d, window=window, sinks=sinks, cu_seqlens=torch.tensor(cuq, dtype=torch.int32, device=dev),
              cu_seqlens_k=torch.tensor(cuk, dtype=torch.int32, device=dev) if keys else None)
    f, g = both(q, k, v, dout, kw)
    some = sorted(range(len(lengths)), key=lambda n: -lengths[n])[:6] + list(range(0, len(lengths), 300))
    check(q, k, v, dout, f, g, [(0, cuq[n], lengths[n], cuk[n], keys_[n]) for n in sorted(set(some))], d, window, sinks, f.desc.scale, dtype)


def reference(q, k, v, dout, window, sinks, scale, rows=2048):
    """Gradients in fp64, queries by the block against the sinks and their band."""
    T = q.shape[0]
    q, k, v, dout = (x.double() for x in (q, k, v, dout))
    dq, dk, dv = (torch.zeros_like(x) for x in (q, k, v))
    for a in range(0, T, rows):
        b = min(a + rows, T)
        lo = max(0, a - window + 1)
        key = torch.cat([torch.arange(0, min(sinks, lo), device=q.device), torch.arange(lo, b, device=q.device)])
        pos = torch.arange(a, b, device=q.device)[:, None]
        seen = (key <= pos) & ((pos - key < window) | (key < sinks))
        kb, vb = k[key], v[key]
        P = torch.softmax(torch.where(seen, scale * (q[a:b] @ kb.T), -torch.inf), -1)
        g = dout[a:b]
        dP = g @ vb.T
        dS = scale * P * (dP - (P * dP).sum(-1, keepdim=True))
        dq[a:b] = dS @ kb
        dk.index_add_(0, key, dS.T @ q[a:b])
        dv.index_add_(0, key, P.T @ g)
    return dq, dk, dv


# Relative error in the 2-norm. 16 bits: half a step each for dS (or P), for delta's rounded output and for the result. fp32: a score's
# error, (2 d + 8) 2^-24 sum |q||k| scale, is 136 x 6e-8 x 4.1 x ... = 3.3e-5 x 1.3 at most, the sums' far below it.
@pytest.mark.parametrize("dtype,tol", [("bf16", 3 * 2.0 ** -8), ("fp16", 3 * 2.0 ** -11), ("fp32", 4.4e-5)])
def test_chunks_that_grow_with_the_sinks(dev, dtype, tol):  # noqa: F811
    T, H, d, window, sinks = 65536, 2, 64, 128, 4096
    q, k, v, dout = make(dev, 1, T, T, H, H, d, dtype, q_std=1.0)
    f, g = both(q, k, v, dout, dict(d=d, window=window, sinks=sinks))
    # partial sums of 64 KB (128 rows of 2 x 64 in fp32): 8 x 152 chunks, rounded up for a head, one begun and one own for each of 32 tiles
    assert g.ws_bytes <= (8 * 152 + H * (1 + 2 * 32)) * 65536 + (1 << 20)
    for h in range(H):
        at = lambda x: x[0].view(T, H, d)[:, h] if x.is_contiguous() else x[0].reshape(T, H, d)[:, h]  # noqa: E731
        ref = reference(at(q), at(k), at(v), at(dout), window, sinks, f.desc.scale)
        for n, r in zip(("dq", "dk", "dv"), ref):
            x = at(getattr(g, n)).double()
            for what, part in (("all", slice(None)), ("sinks", slice(0, sinks))):
                rel = float((x[part] - r[part]).norm() / r[part].norm())
                print(f"[rest] {dtype} head {h} {n} {what}: {rel:.2e}")
                assert rel <= tol, (n, what, rel)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("lengths,Hq,Hk,d,window,sinks", [([900, 0, 30, 1300, 129, 1, 500], 4, 2, 64, 50, 300), ([3] * 500 + [700], 3, 1, 128, 130, 4),
                                                          ([2000], 2, 2, 96, 7, 1500), ([300, 300], 6, 3, 33, 20, 140), ([60], 8, 1, 64, 9, 3)])
def test_nothing_is_written_behind_the_workspace(dev, lengths, Hq, Hk, d, window, sinks, dtype):  # noqa: F811
    at = np.cumsum([0] + lengths).tolist()
    q, k, v, dout = make(dev, 1, at[-1], at[-1], Hq, Hk, d, dtype)
    kw = dict(d=d, window=window, sinks=sinks, cu_seqlens=torch.tensor(at, dtype=torch.int32, device=dev))
    f = gdn.window_attention_forward(q, k, v, **kw)
    need = gdn.gdn_window_attention_backward_workspace_bytes(f.desc)
    big = torch.full((need + 2 * 4096,), 0xa5, dtype=torch.uint8, device=dev)
    g = gdn.alloc_window_attention_grads(f.desc, dev)
    g.workspace = big[4096:4096 + need]
    gdn.window_attention_backward(q, k, v, f.out, f.lse, dout, grads=g, **kw)
    assert gdn.gdn_device_status(g.workspace) == gdn.GDN_OK
    assert bool((big[:4096] == 0xa5).all()) and bool((big[4096 + need:] == 0xa5).all())
    check(q, k, v, dout, f, g, [(0, at[n], lengths[n], at[n], lengths[n]) for n in sorted(set(np.argsort(lengths)[-4:].tolist()))], d, window, sinks,
          f.desc.scale, dtype)
