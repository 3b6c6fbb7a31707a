"""The window attention's cache on the GPU: its filling is exact, a step is held to the oracle's bound, and both
follow the prefill."""
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


def cache_of(dev, N, Hk, d, window, sinks, slots, dtype, lengths, seed=0):
    g = torch.Generator().manual_seed(seed)
    c = gdn.alloc_window_cache(N, Hk, d, window=window, sinks=sinks, slots=slots, dtype=ACT[dtype], device=dev)
    for t in (c.k, c.v):
        t.copy_(torch.randn(t.shape, generator=g).to(ACT[dtype]))
    c.lengths.copy_(torch.tensor(lengths, dtype=torch.int32))
    return c


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("N,T,Hk,d,window,sinks,slack,lengths,pad", [
    (1, 1, 1, 64, 1, 0, 0, [0], 0), (3, 5, 2, 64, 4, 2, 0, [0, 3, 100], 0), (2, 40, 3, 128, 8, 3, 1, [2, -1], 0),
    (4, 7, 1, 7, 16, 0, 5, [0, 1, 15, 2147483000], 1), (2, 300, 2, 80, 100, 130, 0, [0, 77], 0), (2, 33, 4, 100, 32, 4, 0, [31, 5], 3),
    (2, 0, 1, 64, 3, 1, 0, [0, 4], 0)])
def test_write(dev, N, T, Hk, d, window, sinks, slack, lengths, pad, dtype):
    c = cache_of(dev, N, Hk, d, window, sinks, sinks + window + slack, dtype, lengths)
    kv = torch.randn((N, T, 2 * Hk * d + pad), generator=torch.Generator().manual_seed(9)).to(ACT[dtype]).to(dev)
    k, v = kv[..., pad:pad + Hk * d], kv[..., pad + Hk * d:]
    want = [A.cache_write(n64(t), [n64(x[n]).reshape(T, Hk, d) for n in range(N)], lengths, sinks) for t, x in ((c.k, k), (c.v, v))]
    gdn.window_cache_write(k, v, c)
    assert np.array_equal(n64(c.k), want[0]) and np.array_equal(n64(c.v), want[1])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("d", [64, 100])
def test_write_packed(dev, d, dtype):
    counts, lengths, sinks = [0, 1, 30, 200, 5, 0, 64], [0, 9, 2, 0, -3, 4, 50], 3
    cu = torch.tensor([0] + list(np.cumsum(counts)), dtype=torch.int32, device=dev)
    c = cache_of(dev, 7, 2, d, 40, sinks, 45, dtype, lengths)
    kv = torch.randn((1, sum(counts), 4 * d), generator=torch.Generator().manual_seed(9)).to(ACT[dtype]).to(dev)
    k, v = kv[..., :2 * d], kv[..., 2 * d:]
    at = np.cumsum([0] + counts)
    want = [A.cache_write(n64(t), [n64(x[0, at[n]:at[n + 1]]).reshape(-1, 2, d) for n in range(7)], lengths, sinks)
            for t, x in ((c.k, k), (c.v, v))]
    gdn.window_cache_write(k, v, c, cu_seqlens=cu)
    assert np.array_equal(n64(c.k), want[0]) and np.array_equal(n64(c.v), want[1])
    before = c.k.clone()
    ws = torch.empty(4096, dtype=torch.uint8, device=dev)
    bad = cu.clone()
    bad[-1] -= 1
    gdn.window_cache_write(k, v, c, cu_seqlens=bad, workspace=ws)
    assert gdn.gdn_device_status(ws) == gdn.GDN_ERR_DEVICE_SEQLENS and torch.equal(before, c.k)


STEPS = [  # N, Hq, Hk, d, window, sinks, slack, lengths
    (1, 1, 1, 64, 1, 0, 0, [0]), (1, 2, 1, 128, 8, 4, 0, [0]), (3, 4, 2, 64, 16, 2, 0, [0, 5, 500]), (4, 6, 2, 128, 33, 3, 1, [2, -1, 35, 36]),
    (2, 8, 1, 80, 100, 0, 7, [50, 1000]), (2, 5, 5, 96, 64, 130, 0, [100, 400]), (3, 12, 4, 128, 700, 4, 0, [699, 704, 5000]),
    (2, 3, 1, 7, 20, 1, 0, [3, 90]), (2, 4, 2, 100, 64, 4, 0, [10, 200]), (2, 16, 1, 64, 300, 4, 0, [1, 2000]), (1, 2, 2, 256, 90, 4, 3, [333]),
    (2, 40, 2, 64, 130, 4, 0, [0, 1000]), (1, 4, 1, 128, 5000, 4, 0, [6000]), (2, 2, 1, 128, 2, 0, 0, [2147483646, 0])]


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("N,Hq,Hk,d,window,sinks,slack,lengths", STEPS)
def test_step(dev, N, Hq, Hk, d, window, sinks, slack, lengths, dtype):
    c = cache_of(dev, N, Hk, d, window, sinks, sinks + window + slack, dtype, lengths)
    # slots that no position has reached yet, and those outside the window, may hold anything
    t = torch.tensor(lengths).view(-1, 1)
    i = torch.arange(c.k.shape[2]).view(1, -1)
    ring = c.k.shape[2] - sinks
    held = torch.where(i < sinks, i, t - (t - i) % ring)
    seen = (held >= torch.clamp(i, max=sinks)) & (held < t) & ((held > t - window) | (i < sinks))
    for x in (c.k, c.v):
        x[(~seen).to(dev)[:, None, :].expand(-1, Hk, -1)] = float("nan")
    g = torch.Generator().manual_seed(4)
    q = (2.0 * torch.randn((N, 1, Hq * d), generator=g)).to(ACT[dtype]).to(dev)
    kv = torch.randn((N, 1, 2 * Hk * d), generator=g).to(ACT[dtype]).to(dev)
    k, v = kv[..., :Hk * d], kv[..., Hk * d:]
    want = [A.cache_write(n64(x), [n64(y[n]).reshape(1, Hk, d) for n in range(N)], lengths, sinks) for x, y in ((c.k, k), (c.v, v))]
    out = gdn.window_attention_step(q, k, v, c)
    assert np.array_equal(n64(c.k), want[0], equal_nan=True) and np.array_equal(n64(c.v), want[1], equal_nan=True)
    ref, err = A.step(n64(q).reshape(N, Hq, d), np.nan_to_num(want[0]), np.nan_to_num(want[1]), lengths, window, sinks, d ** -0.5, dtype)
    use = (np.abs(n64(out).reshape(ref.shape) - ref) / A.bound(ref, err, dtype)).max()
    print(f"[step] {dtype}: bound_use={use:.3f}")
    assert use <= 1.0


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_steps_follow_a_prefill(dev, dtype):
    """A prompt in two pieces, then token by token, equals one pass over the whole sequence: every row is held to the
    oracle of the whole sequence, which is the definition of both."""
    Hq, Hk, d, window, sinks, T = 4, 2, 64, 50, 3, 140
    g = torch.Generator().manual_seed(1)
    q = (2.0 * torch.randn((2, T, Hq * d), generator=g)).to(ACT[dtype]).to(dev)
    k, v = (torch.randn((2, T, Hk * d), generator=g).to(ACT[dtype]).to(dev) for _ in range(2))
    c = gdn.alloc_window_cache(2, Hk, d, window=window, sinks=sinks, dtype=ACT[dtype], device=dev)
    rows = []
    for a, b in ((0, 60), (60, 100)):
        rows.append(gdn.window_attention_forward(q[:, a:b], k[:, :b], v[:, :b], d=d, window=window, sinks=sinks).out)
        gdn.window_cache_write(k[:, a:b], v[:, a:b], c)
        c.lengths += b - a
    ws, step_out = None, torch.empty((2, 1, Hq * d), dtype=ACT[dtype], device=dev)
    qt, kt, vt = q[:, :1].clone(), k[:, :1].clone(), v[:, :1].clone()
    r = gdn.window_attention_desc_for(qt, kt, vt, d=d, window=window, sinks=sinks, slots=c.k.shape[2])
    ws = torch.empty(gdn.gdn_window_attention_step_workspace_bytes(r), dtype=torch.uint8, device=dev)
    graph = None
    for t in range(100, T):   # the first step eager, the others replayed
        for x, y in ((qt, q), (kt, k), (vt, v)):
            x.copy_(y[:, t:t + 1])
        if t == 101:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                gdn.window_attention_step(qt, kt, vt, c, out=step_out, workspace=ws)
                c.lengths += 1
        if graph is not None:
            graph.replay()
        else:
            gdn.window_attention_step(qt, kt, vt, c, out=step_out, workspace=ws)
            c.lengths += 1
        rows.append(step_out.clone())
    got = torch.cat(rows, dim=1)
    for b in range(2):
        ref = A.window_attention(*(n64(x[b]).reshape(T, -1, d) for x in (q, k, v)), window, sinks, d ** -0.5, dtype)
        use = (np.abs(n64(got[b]).reshape(T, Hq, d) - ref["out"]) / A.bound(ref["out"], ref["out_err"], dtype)).max()
        assert use <= 1.0, use


def test_step_is_run_to_run_identical_and_keeps_to_its_rows(dev):
    c = cache_of(dev, 3, 2, 128, 600, 4, 604, "bf16", [50, -1, 5000])
    q, kv = (torch.randn((3, 1, n * 128), generator=torch.Generator().manual_seed(n)).to(torch.bfloat16).to(dev) for n in (8, 4))
    k, v = kv[..., :256], kv[..., 256:]
    big = torch.full((5, 1, 8 * 128), 7.0, dtype=torch.bfloat16, device=dev)
    a = gdn.window_attention_step(q, k, v, c, out=big[1:4])
    idle = c.k[1].clone()
    b = gdn.window_attention_step(q, k, v, c)
    assert torch.equal(a, b) and torch.equal(idle, c.k[1]) and not a[1].any()
    assert bool((big[0] == 7).all()) and bool((big[4] == 7).all())
