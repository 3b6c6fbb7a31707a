"""Rotary positions on the GPU against the fp64 definition."""
import numpy as np
import pytest
import torch

from linear_attention_sequence_qkv_gb300 import build, gdn
from oracle import layer_ops as O

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


def held(got, x, positions, f, d, rot, layout, dtype, inverse=False, scale=1.0):
    """Tolerance: the angle's fraction of a turn is rounded to 24 bits (2^-25 turns, 2 pi of that in the angle,
    and a few U32 in cos, sin and the two products): 8 U32 of |x1| + |x2|; then one rounding. For 16-bit types cos
    and sin are the hardware's, whose documented absolute errors on [-pi, pi] are 2^-21.19 and 2^-21.41, that is
    7 U32 more: 16 in all. Copied channels are exact."""
    B, T = x.shape[:2]
    xr = n64(x).reshape(B, T, -1, d)
    ref = O.rotary(xr, positions, f, rot, layout, inverse, scale)
    mag = np.broadcast_to(np.linalg.norm(xr[..., :rot], axis=-1, keepdims=True), ref.shape)
    i = np.arange(rot // 2)
    i1, i2 = (i, i + rot // 2) if layout == "half" else (2 * i, 2 * i + 1)
    mag = np.zeros_like(ref)
    mag[..., i1] = mag[..., i2] = (np.abs(xr[..., i1]) + np.abs(xr[..., i2])) * abs(scale)
    y = n64(got).reshape(ref.shape)
    assert np.array_equal(y[..., rot:], xr[..., rot:])
    tol = O.bound(ref, (8 if dtype == "fp32" else 16) * O.U32 * mag, dtype)
    use = (np.abs(y - ref) / tol)[..., :rot].max() if ref.size else 0.0
    print(f"[rotary] {dtype} {layout}: bound_use={use:.3f}")
    assert use <= 1.0


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("B,T,Hq,Hk,d,rot", [(1, 1, 1, 0, 2, 2), (2, 5, 3, 1, 64, 64), (3, 1, 32, 8, 128, 32), (1, 130, 2, 2, 80, 20),
                                             (2, 33, 1, 5, 256, 64), (1, 7, 4, 4, 7, 6), (1, 9, 2, 1, 100, 96), (1, 3, 6, 2, 512, 512)])
def test_rows(dev, B, T, Hq, Hk, d, rot, layout, dtype):
    g = torch.Generator().manual_seed(T * d + rot)
    qk = torch.randn((B, T, (Hq + Hk) * d), generator=g).to(ACT[dtype]).to(dev)
    q, k = qk[..., :Hq * d], qk[..., Hq * d:] if Hk else None
    off = torch.randint(0, 1 << 20, (B,), generator=g).to(torch.int32).to(dev)
    f = O.frequencies(rot)
    pos = n64(off)[:, None] + np.arange(T)
    for inverse in (False, True):
        qo, ko = gdn.rotary(q, k, gdn.rotary_table(rot, device=dev), d=d, rot=rot, layout=layout, inverse=inverse, offsets=off)
        held(qo, q, pos, f, d, rot, layout, dtype, inverse)
        if Hk:
            held(ko, k, pos, f, d, rot, layout, dtype, inverse)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_positions_and_scalings(dev, dtype):
    g = torch.Generator().manual_seed(3)
    B, T, H, d, rot = 2, 40, 3, 128, 64
    q = torch.randn((B, T, H * d), generator=g).to(ACT[dtype]).to(dev)
    pos = torch.randint(-(1 << 31), (1 << 31) - 1, (B, T), generator=g).to(torch.int32)
    pos[0, :6] = torch.tensor([0, 1, -1, (1 << 31) - 1, -(1 << 31), 1 << 24])
    for kw in ({}, dict(scaling="linear", factor=8.0), dict(scaling="by_parts", factor=32.0, low=1.0, high=32.0, original=4096)):
        f = O.frequencies(rot, 10000.0, **kw)
        table = gdn.rotary_table(rot, 10000.0, device=dev, **kw)
        scale = 0.1 * np.log(32.0) + 1.0 if kw else 1.0
        # the reference angle is the table's: turns in 2^-64, exactly times the position
        turns = np.array([v % 2 ** 64 for v in table.tolist()], dtype=object)
        exact = np.array([[[float((int(p) * t) % 2 ** 64) / 2.0 ** 64 for t in turns] for p in row] for row in pos.tolist()])
        assert np.allclose(np.cos(2 * np.pi * exact[0, 1]), np.cos(f), atol=1e-12)
        qo, _ = gdn.rotary(q, None, table, d=d, rot=rot, scale=scale, positions=pos.to(dev))
        # the oracle with one position per token and the exact angle as its frequency
        for b in range(B):
            for t in (0, 1, 2, 3, 4, 5, 17, 39):
                held(qo[b:b + 1, t:t + 1], q[b:b + 1, t:t + 1], np.ones((1, 1)), 2 * np.pi * exact[b, t], d, rot, "half", dtype,
                     scale=scale)


def test_packed_positions_restart(dev):
    lengths = [0, 5, 1, 0, 70, 3]
    cu = torch.tensor([0] + list(np.cumsum(lengths)), dtype=torch.int32, device=dev)
    T, H, d = sum(lengths), 2, 64
    q = torch.randn((1, T, H * d), generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).to(dev)
    off = torch.tensor([9, 100, 0, 5, 70000, 1], dtype=torch.int32, device=dev)
    table, f = gdn.rotary_table(d, device=dev), O.frequencies(d)
    at = np.concatenate([np.arange(n) for n in lengths])
    base = np.concatenate([np.full(n, o) for n, o in zip(lengths, off.tolist())])
    held(gdn.rotary(q, None, table, d=d, cu_seqlens=cu)[0], q, at[None], f, d, d, "half", "bf16")
    held(gdn.rotary(q, None, table, d=d, cu_seqlens=cu, offsets=off)[0], q, (at + base)[None], f, d, d, "half", "bf16")
    # positions given: cu_seqlens is still checked, and counts nothing
    pos = torch.arange(T, dtype=torch.int32, device=dev)[None].contiguous()
    held(gdn.rotary(q, None, table, d=d, cu_seqlens=cu, positions=pos)[0], q, np.arange(T)[None], f, d, d, "half", "bf16")


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("pad", [0, 8, 3])
def test_in_place_and_strided_outputs(dev, layout, pad):
    """In place in a wider buffer: the other channels keep their bits; strided outputs likewise."""
    B, T, H, d, rot = 2, 19, 3, 64, 32
    buf = torch.randn((B, T, H * d + pad), generator=torch.Generator().manual_seed(2)).to(torch.float16).to(dev)
    before = buf.clone()
    q = buf[..., pad:]
    table, f = gdn.rotary_table(rot, device=dev), O.frequencies(rot)
    gdn.rotary(q, None, table, d=d, rot=rot, layout=layout, q_out=q)
    assert torch.equal(buf[..., :pad], before[..., :pad])
    held(q, before[..., pad:], np.broadcast_to(np.arange(T), (B, T)), f, d, rot, layout, "fp16")
    wide = torch.full((B, T, H * d + 16), 5.0, dtype=torch.float16, device=dev)
    gdn.rotary(before[..., pad:], None, table, d=d, rot=rot, layout=layout, q_out=wide[..., 8:8 + H * d])
    assert torch.equal(wide[..., 8:8 + H * d], q) and (wide[..., :8] == 5).all() and (wide[..., 8 + H * d:] == 5).all()


def test_malformed_seqlens_write_nothing(dev):
    q = torch.randn((1, 20, 64), device=dev)
    table = gdn.rotary_table(64, device=dev)
    ws = torch.empty(256, dtype=torch.uint8, device=dev)
    for cu in ([0, 21, 20], [1, 5, 20], [0, 5, 19], [0, -1, 20]):
        out = torch.full_like(q, 7.0)
        gdn.rotary(q, None, table, d=64, cu_seqlens=torch.tensor(cu, dtype=torch.int32, device=dev), q_out=out, workspace=ws)
        assert gdn.gdn_device_status(ws) == gdn.GDN_ERR_DEVICE_SEQLENS and (out == 7.0).all()
    gdn.rotary(q, None, table, d=64, q_out=out, workspace=ws)
    assert gdn.gdn_device_status(ws) == gdn.GDN_OK


def test_non_finite_values_stay_in_their_pair(dev):
    q = torch.randn((1, 4, 128), device=dev).to(torch.bfloat16)
    table = gdn.rotary_table(64, device=dev)
    clean = gdn.rotary(q, None, table, d=64)[0]
    q[0, 2, 70] = float("inf")        # head 1, channel 6: pair (6, 38)
    got = gdn.rotary(q, None, table, d=64)[0]
    same = torch.ones_like(got, dtype=torch.bool)
    same[0, 2, [70, 102]] = False
    assert torch.equal(got[same], clean[same]) and not torch.isfinite(got[~same]).any()


def test_no_tokens_and_many_tokens(dev):
    table = gdn.rotary_table(64, device=dev)
    q = torch.empty((2, 0, 64), device=dev)
    assert gdn.rotary(q, None, table, d=64)[0].shape == (2, 0, 64)
    # more tokens than one wave of any launch, and more than 2^31 elements
    T, H = 300000, 128
    q = torch.randn((1, T, H * 64), dtype=torch.bfloat16, device=dev)
    assert q.numel() > 2 ** 31
    out = gdn.rotary(q, None, table, d=64)[0]
    f = O.frequencies(64)
    for t0 in (0, 65530, T - 10):
        held(out[:, t0:t0 + 10], q[:, t0:t0 + 10], np.arange(t0, t0 + 10)[None], f, 64, 64, "half", "bf16")


def test_captured_and_replayed(dev):
    q = torch.randn((4, 1, 8 * 64), device=dev).to(torch.bfloat16)
    off = torch.zeros(4, dtype=torch.int32, device=dev)
    table, out = gdn.rotary_table(64, device=dev), torch.empty_like(q)
    ws = torch.empty(256, dtype=torch.uint8, device=dev)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gdn.rotary(q, None, table, d=64, offsets=off, q_out=out, workspace=ws)
    for step in (3, 100):
        off.fill_(step)                # the offsets are read when the graph runs
        graph.replay()
        torch.cuda.synchronize()
        held(out, q, np.full((4, 1), step), O.frequencies(64), 64, 64, "half", "bf16")


@pytest.mark.parametrize("d,rot", [(192, 48), (80, 20), (66, 66), (64, 2)])
def test_one_of_the_tensors_in_place(dev, d, rot):
    B, T, H = 2, 37, 3
    g = torch.Generator().manual_seed(d)
    q, k = (torch.randn((B, T, h * d), generator=g).to(torch.bfloat16).to(dev) for h in (H, 1))
    table = gdn.rotary_table(rot, device=dev)
    want_q, want_k = gdn.rotary(q, k, table, d=d, rot=rot)
    held(want_q, q, np.broadcast_to(np.arange(T), (B, T)), O.frequencies(rot), d, rot, "half", "bf16")
    in_place, kept = q.clone(), k.clone()
    _, ko = gdn.rotary(in_place, kept, table, d=d, rot=rot, q_out=in_place)
    assert torch.equal(in_place, want_q) and torch.equal(ko, want_k) and torch.equal(kept, k)
    in_place, kept = k.clone(), q.clone()
    qo, _ = gdn.rotary(kept, in_place, table, d=d, rot=rot, k_out=in_place)
    assert torch.equal(in_place, want_k) and torch.equal(qo, want_q) and torch.equal(kept, q)
