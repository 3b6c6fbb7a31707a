"""Group norm with an activation on the GPU against the fp64 definition."""
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
    return None if t is None else t.detach().double().cpu().numpy()


def make(dev, N, L, C, dtype, seed=0, pad=0, w32=False):
    g = torch.Generator().manual_seed(seed)
    randn = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    x = (randn(N, L, C + pad) * (1.0 + 0.3 * randn(C + pad)) + 0.5 * randn(C + pad)).to(ACT[dtype]).to(dev)[..., pad:]
    wt = torch.float32 if w32 else ACT[dtype]
    return x, (1.0 + 0.1 * randn(C)).to(wt).to(dev), (0.1 * randn(C)).to(wt).to(dev), randn(N, L, C).to(ACT[dtype]).to(dev)


def held(got, r, name, dtype):
    ref, tol = r[name], O.bound(r[name], r[name + "_err"], dtype)
    got = n64(got).reshape(ref.shape)
    assert np.isfinite(got).all(), f"{name}: not finite"
    use = (np.abs(got - ref) / tol).max() if ref.size else 0.0
    print(f"[group norm] {name} {dtype}: bound_use={use:.3f}")
    assert use <= 1.0, f"{name}: {use:.3f} of the bound"


def check_all(x, w, b, dy, G, act, dtype, eps=1e-5):
    r = O.group_norm(n64(x), n64(w), n64(b), G, act, eps, n64(dy))
    f = gdn.group_norm_forward(x, w, b, groups=G, act=act, eps=eps)
    held(f.out, r, "out", dtype)
    held(f.mean, r, "mean", "fp32")
    held(f.rstd, r, "rstd", "fp32")
    g = gdn.group_norm_backward(x, w, b, f.mean, f.rstd, dy, groups=G, act=act, eps=eps)
    held(g.dx, r, "dx", dtype)
    held(g.dweight, r, "dweight", "fp32")
    held(g.dbias, r, "dbias", "fp32")
    return f, g


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("N,L,C,G", [(1, 1, 2, 1), (3, 1, 64, 8), (5, 1, 24, 3), (7, 1, 195, 3), (2, 1, 2048, 2), (9, 1, 512, 4),
                                     (4, 1, 65, 1), (33, 1, 96, 2), (1, 1, 8200, 1), (300, 1, 256, 16)])
def test_per_token(dev, N, L, C, G, dtype):
    check_all(*make(dev, N, L, C, dtype, seed=N + C), G, "silu", dtype)


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("N,L,C,G", [(1, 2, 8, 2), (2, 5, 24, 3), (1, 100, 65, 5), (3, 64, 128, 1), (2, 700, 96, 4), (1, 3000, 40, 5),
                                     (2, 1025, 256, 2), (1, 77, 2048, 8), (2, 6, 33, 33)])
def test_over_positions(dev, N, L, C, G, dtype):
    check_all(*make(dev, N, L, C, dtype, seed=L + C), G, "silu", dtype)


@pytest.mark.parametrize("N,L,C,G", [(6, 1, 128, 4), (2, 50, 96, 3), (5, 1, 195, 13)])
@pytest.mark.parametrize("act", ["silu", "none"])
@pytest.mark.parametrize("pad", [0, 8, 1])
def test_views_activations_and_fp32_weights(dev, N, L, C, G, act, pad):
    x, w, b, dy = make(dev, N, L, C, "bf16", pad=pad, w32=True)
    f, _ = check_all(x, w, b, dy, G, act, "bf16")
    # the instance and position strides alone change nothing
    dense = gdn.group_norm_forward(x.contiguous(), w, b, groups=G, act=act)
    assert np.allclose(n64(dense.out), n64(f.out), rtol=2.0 ** -7, atol=1e-6)


@pytest.mark.parametrize("N,L,C,G", [(6, 1, 128, 4), (2, 50, 96, 3)])
def test_without_weight_or_bias(dev, N, L, C, G):
    x, w, b, dy = make(dev, N, L, C, "fp32")
    for ww, bb in ((None, None), (w, None), (None, b)):
        check_all(x, ww, bb, dy, G, "silu", "fp32")


@pytest.mark.parametrize("L,C,G", [(1, 256, 2), (40, 64, 4)])
def test_large_offset_and_constant_groups(dev, L, C, G):
    """A mean far from zero against the deviation costs no digits of the centred values (they are centred before they
    are squared); a group of equal values gives its bias."""
    x, w, b, dy = make(dev, 3, L, C, "fp32")
    check_all(x + 1000.0, w, b, dy, G, "none", "fp32")
    x[1, :, :C // G] = 2.5
    f, g = check_all(x, w, b, dy, G, "none", "fp32")
    assert torch.equal(f.out[1, :, :C // G], b[:C // G].expand(L, -1))


def test_infinities_stay_in_their_group(dev):
    x, w, b, _ = make(dev, 4, 1, 128, "bf16")
    clean = gdn.group_norm_forward(x, w, b, groups=4).out
    x[2, 0, 40] = float("inf")
    got = gdn.group_norm_forward(x, w, b, groups=4).out
    same = torch.ones_like(got, dtype=torch.bool)
    same[2, 0, 32:64] = False
    assert torch.equal(got[same], clean[same]) and torch.isnan(got[2, 0, 40])


def test_saturated_activation(dev):
    """z of several hundred on both sides: SiLU is z or -0, its gradient 1 or 0, nothing overflows."""
    x, w, b, dy = make(dev, 4, 1, 64, "fp32")
    check_all(x, w * 300.0, b, dy, 2, "silu", "fp32")


def test_nothing_to_do(dev):
    for N, L in ((0, 5), (3, 0)):
        x = torch.empty((N, L, 32), device=dev)
        w = torch.ones(32, device=dev)
        f = gdn.group_norm_forward(x, w, w, groups=4)
        g = gdn.group_norm_backward(x, w, w, f.mean, f.rstd, x, groups=4)
        assert (g.dweight == 0).all() and (g.dbias == 0).all()


@pytest.mark.parametrize("N,L,C,G", [(257, 1, 512, 8), (2, 900, 192, 3)])
def test_repeatable_guarded_captured(dev, N, L, C, G):
    x, w, b, dy = make(dev, N, L, C, "bf16")
    f, g = check_all(x, w, b, dy, G, "silu", "bf16")
    n = x.numel()
    wide = torch.full((n + 512,), 3.0, dtype=x.dtype, device=dev)
    bufs = gdn.alloc_group_norm(f.desc, dev)
    bufs.out = wide[256:256 + n].view(x.shape)
    grads = gdn.alloc_group_norm_grads(f.desc, dev)
    wide2 = torch.full((n + 512,), 3.0, dtype=x.dtype, device=dev)
    grads.dx = wide2[256:256 + n].view(x.shape)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gdn.group_norm_forward(x, w, b, groups=G, bufs=bufs)
        gdn.group_norm_backward(x, w, b, bufs.mean, bufs.rstd, dy, groups=G, grads=grads)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        graph.replay()
        graph.replay()
    side.synchronize()
    assert torch.equal(bufs.out, f.out) and torch.equal(grads.dx, g.dx)
    assert torch.equal(grads.dweight, g.dweight) and torch.equal(grads.dbias, g.dbias)
    for t in (wide, wide2):
        assert (t[:256] == 3).all() and (t[256 + n:] == 3).all()


def test_offsets_past_32_bits(dev):
    N, C, G = 1100000, 4096, 32
    x = torch.randn((N, 1, C), dtype=torch.bfloat16, device=dev)
    assert x.numel() > 2 ** 32
    w, b = torch.ones(C, device=dev), torch.zeros(C, device=dev)
    f = gdn.group_norm_forward(x, w, b, groups=G)
    g = gdn.group_norm_backward(x, w, b, f.mean, f.rstd, x, groups=G)
    tail = x[-3:].contiguous()
    r = O.group_norm(n64(tail), None, None, G, "silu", 1e-5, n64(tail))
    held(f.out[-3:], r, "out", "bf16")
    held(g.dx[-3:], r, "dx", "bf16")


def test_gradient_against_differences(dev):
    """As for the recurrence: central differences of step 2^-6 along a random direction."""
    x, w, b, dy = make(dev, 3, 20, 48, "fp32")
    f = gdn.group_norm_forward(x, w, b, groups=3)
    g = gdn.group_norm_backward(x, w, b, f.mean, f.rstd, dy, groups=3)
    gen, step = torch.Generator().manual_seed(4), 2.0 ** -6
    args = [x, w, b]
    for i, grad in enumerate((g.dx, g.dweight, g.dbias)):
        v = torch.randn(args[i].shape, generator=gen).to(dev)
        ends = []
        for sign in (1.0, -1.0):
            moved = list(args)
            moved[i] = args[i] + sign * step * v
            ends.append((n64(gdn.group_norm_forward(*moved, groups=3).out) * n64(dy)).sum())
        diff, want = (ends[0] - ends[1]) / (2 * step), (n64(grad) * n64(v)).sum()
        assert abs(diff - want) <= 2e-2 * np.linalg.norm(n64(grad)), i


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("N,L,C,G", [(3, 1, 1032, 1), (2, 1, 4112, 2), (2, 1, 1003, 1), (3, 1, 2050, 2), (2, 1, 8208, 1), (1, 1, 70, 1),
                                     (5, 1, 388, 4), (2500, 1, 64, 1), (1300, 1, 33, 1), (2, 1, 16400, 1), (3, 1, 40001, 1)])
def test_wide_odd_and_many_rows(dev, N, L, C, G, dtype):
    check_all(*make(dev, N, L, C, dtype, seed=N + C), G, "silu", dtype)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("N,L,C,G", [(3, 1000, 8, 1), (70, 41, 512, 64), (2, 2047, 48, 6), (700, 3, 16, 2), (1, 9, 16400, 1), (5, 333, 130, 2)])
def test_chunks_of_positions(dev, N, L, C, G, dtype):
    check_all(*make(dev, N, L, C, dtype, seed=N + L), G, "silu", dtype)
