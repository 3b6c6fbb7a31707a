"""Head norms with rotary positions on the GPU against the fp64 definition; each case held to the bound that
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
    tol = A.bound(ref, err, dtype)
    use = (np.abs(n64(got).reshape(ref.shape) - ref) / tol).max() if ref.size else 0.0
    print(f"[norm_rotary] {dtype} {what}: bound_use={use:.3f}")
    assert use <= 1.0, (what, use)


def make(dev, B, T, Hq, Hk, d, dtype, wdtype=None, pad=0, seed=0):
    g = torch.Generator().manual_seed(seed + 1000 * T + d)
    randn = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    qk = (randn(B, T, (Hq + Hk) * d + pad) * 1.7).to(ACT[dtype]).to(dev)
    wt = ACT[wdtype or dtype]
    s = {"q": qk[..., pad:pad + Hq * d], "k": qk[..., pad + Hq * d:] if Hk else None}
    s["qw"], s["kw"] = (1 + 0.1 * randn(d)).to(wt).to(dev), (1 + 0.1 * randn(d)).to(wt).to(dev) if Hk else None
    s["gq"], s["gk"] = randn(B, T, Hq * d).to(ACT[dtype]).to(dev), randn(B, T, Hk * d).to(ACT[dtype]).to(dev) if Hk else None
    return s


def check(s, got, grads, pos, f, d, rot, layout, dtype, eps=1e-6, scale=1.0):
    for n in ("q", "k"):
        if s[n] is None:
            continue
        x = n64(s[n]).reshape(*s[n].shape[:2], -1, d)
        w = None if s[n + "w"] is None else n64(s[n + "w"])
        r = A.norm_rotary(x, w, pos, f, rot, layout, eps, scale, n64(s["g" + n]).reshape(x.shape) if grads else None, dtype != "fp32")
        held(got[0 if n == "q" else 1], r["y"], r["y_err"], dtype, n)
        if grads:
            held(getattr(grads, "d" + n), r["dx"], r["dx_err"], dtype, "d" + n)
            held(getattr(grads, f"d{n}_weight"), r["dw"], r["dw_err"], "fp32", f"d{n}_weight")


CASES = [(1, 1, 1, 0, 2, 2), (2, 5, 3, 1, 64, 64), (3, 1, 32, 8, 128, 32), (1, 130, 2, 2, 80, 20), (2, 33, 1, 5, 256, 64), (1, 7, 4, 4, 7, 6),
         (1, 9, 2, 1, 100, 96), (1, 3, 6, 2, 512, 512), (2, 40, 5, 3, 96, 48), (1, 65, 3, 2, 192, 192), (1, 2, 1, 1, 1024, 256), (4, 300, 8, 2, 128, 128)]


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("B,T,Hq,Hk,d,rot", CASES)
def test_rows(dev, B, T, Hq, Hk, d, rot, layout, dtype):
    s = make(dev, B, T, Hq, Hk, d, dtype)
    off = torch.randint(0, 1 << 20, (B,), generator=torch.Generator().manual_seed(T)).to(torch.int32).to(dev)
    table, kw = gdn.rotary_table(rot, device=dev), dict(d=d, rot=rot, layout=layout, offsets=off)
    got = gdn.norm_rotary(s["q"], s["k"], s["qw"], s["kw"], table, **kw)
    grads = gdn.norm_rotary_backward(s["q"], s["k"], s["qw"], s["kw"], table, s["gq"], s["gk"], **kw)
    check(s, got, grads, n64(off)[:, None] + np.arange(T), A.frequencies(rot), d, rot, layout, dtype)


@pytest.mark.parametrize("dtype,pad", [("bf16", 1), ("fp16", 4), ("fp32", 2), ("bf16", 8)])
def test_alignments_and_weight_types(dev, dtype, pad):
    """Rows off 16 bytes take other loads; fp32 weights, no weights, an attention factor, positions of any sign."""
    s = make(dev, 2, 21, 3, 2, 64, dtype, wdtype="fp32", pad=pad)
    s["kw"] = None
    pos = torch.randint(-(1 << 31), (1 << 31) - 1, (2, 21), generator=torch.Generator().manual_seed(pad)).to(torch.int32)
    table = gdn.rotary_table(32, device=dev)
    kw = dict(d=64, rot=32, positions=pos.to(dev), scale=1.25, eps=1e-3)
    got = gdn.norm_rotary(s["q"], s["k"], s["qw"], None, table, **kw)
    grads = gdn.norm_rotary_backward(s["q"], s["k"], s["qw"], None, table, s["gq"], s["gk"], **kw)
    turns = np.array([v % 2 ** 64 for v in table.tolist()], dtype=object)
    exact = np.array([[[float((int(p) * t) % 2 ** 64) / 2.0 ** 64 for t in turns] for p in row] for row in pos.tolist()])
    for b in range(2):
        for t in (0, 1, 20):   # a token at a time: its exact angles as the frequencies of position 1
            one = {k: v if v is None or v.dim() == 1 else v[b:b + 1, t:t + 1] for k, v in s.items()}
            check(one, [x[b:b + 1, t:t + 1] for x in got], None, np.ones((1, 1)), 2 * np.pi * exact[b, t], 64, 32, "half", dtype, 1e-3, 1.25)
    # gradients with the rounded fp64 angles: positions beyond 2^31 / 2^53 of a turn are exact in `exact` alone
    near = torch.arange(42, dtype=torch.int32).view(2, 21).to(dev)
    kw["positions"] = near
    got = gdn.norm_rotary(s["q"], s["k"], s["qw"], None, table, **kw)
    grads = gdn.norm_rotary_backward(s["q"], s["k"], s["qw"], None, table, s["gq"], s["gk"], **kw)
    check(s, got, grads, n64(near), A.frequencies(32), 64, 32, "half", dtype, 1e-3, 1.25)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_packed_positions_restart(dev, dtype):
    lengths, offs = [0, 5, 1, 0, 70, 3], [9, 0, 4, 2, 100, 7]
    cu = torch.tensor([0] + list(np.cumsum(lengths)), dtype=torch.int32, device=dev)
    off = torch.tensor(offs, dtype=torch.int32, device=dev)
    s = make(dev, 1, sum(lengths), 4, 2, 128, dtype)
    table, kw = gdn.rotary_table(128, device=dev), dict(d=128, cu_seqlens=cu, offsets=off)
    got = gdn.norm_rotary(s["q"], s["k"], s["qw"], s["kw"], table, **kw)
    grads = gdn.norm_rotary_backward(s["q"], s["k"], s["qw"], s["kw"], table, s["gq"], s["gk"], **kw)
    pos = np.concatenate([o + np.arange(n) for n, o in zip(lengths, offs)])[None]
    check(s, got, grads, pos, A.frequencies(128), 128, 128, "half", dtype)


@pytest.mark.parametrize("d,dtype", [(128, "bf16"), (100, "fp16"), (192, "fp32")])
def test_in_place_and_run_to_run(dev, d, dtype):
    s = make(dev, 2, 50, 4, 1, d, dtype)
    table = gdn.rotary_table(d // 2 // 2 * 2, device=dev)
    kw = dict(d=d, rot=d // 2 // 2 * 2)
    q, k = gdn.norm_rotary(s["q"], s["k"], s["qw"], s["kw"], table, **kw)
    a = gdn.norm_rotary_backward(s["q"], s["k"], s["qw"], s["kw"], table, s["gq"], s["gk"], **kw)
    b = gdn.norm_rotary_backward(s["q"], s["k"], s["qw"], s["kw"], table, s["gq"], s["gk"], **kw)
    for n in ("dq", "dk", "dq_weight", "dk_weight"):
        assert torch.equal(getattr(a, n), getattr(b, n)), n
    gdn.norm_rotary(s["q"], s["k"], s["qw"], s["kw"], table, q_out=s["q"], k_out=s["k"], **kw)
    assert torch.equal(q, s["q"]) and torch.equal(k, s["k"])


def test_nothing_to_do_and_bad_offsets(dev):
    s = make(dev, 2, 0, 2, 1, 64, "bf16")
    table = gdn.rotary_table(64, device=dev)
    gdn.norm_rotary(s["q"], s["k"], s["qw"], s["kw"], table, d=64)
    g = gdn.norm_rotary_backward(s["q"], s["k"], s["qw"], s["kw"], table, s["gq"], s["gk"], d=64)
    assert not g.dq_weight.any() and not g.dk_weight.any()
    s = make(dev, 1, 10, 2, 1, 64, "bf16")
    cu = torch.tensor([0, 7, 9], dtype=torch.int32, device=dev)   # does not end at 10
    out = torch.full_like(s["q"], 7.0), torch.full_like(s["k"], 7.0)
    ws = torch.empty(256, dtype=torch.uint8, device=dev)
    gdn.norm_rotary(s["q"], s["k"], s["qw"], s["kw"], table, d=64, cu_seqlens=cu, q_out=out[0], k_out=out[1], workspace=ws)
    assert gdn.gdn_device_status(ws) == gdn.GDN_ERR_DEVICE_SEQLENS
    assert bool((out[0] == 7).all()) and bool((out[1] == 7).all())
    grads = gdn.alloc_norm_rotary_grads(gdn.norm_rotary_desc_for(s["q"], s["k"], s["gq"], s["gk"], s["qw"], d=64, cu_seqlens=cu), dev)
    for n in ("dq", "dk", "dq_weight", "dk_weight"):
        getattr(grads, n).fill_(7.0)
    gdn.norm_rotary_backward(s["q"], s["k"], s["qw"], s["kw"], table, s["gq"], s["gk"], d=64, cu_seqlens=cu, grads=grads)
    assert gdn.gdn_device_status(grads.workspace) == gdn.GDN_ERR_DEVICE_SEQLENS
    for n in ("dq", "dk", "dq_weight", "dk_weight"):
        assert bool((getattr(grads, n) == 7).all()), n


def test_zero_rows_and_non_finite_heads_stay_apart(dev):
    """A head of zeros has rstd = eps^-1/2; a NaN in one head stays in that head."""
    s = make(dev, 1, 6, 4, 2, 128, "bf16")
    s["q"][0, 2, 128:256] = 0.0
    table = gdn.rotary_table(128, device=dev)
    clean = gdn.norm_rotary(s["q"], s["k"], s["qw"], s["kw"], table, d=128)
    check(s, clean, None, np.arange(6)[None], A.frequencies(128), 128, 128, "half", "bf16")
    s["q"][0, 3, 128] = float("nan")
    got = gdn.norm_rotary(s["q"], s["k"], s["qw"], s["kw"], table, d=128)[0]
    same = (got == clean[0]).view(6, 4, 128)
    assert got.view(6, 4, 128)[3, 1].isnan().all()
    same[3, 1] = True
    assert bool(same.all())


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("B,T,Hq,Hk,d,rot", [(2, 37, 6, 2, 96, 24), (1, 50, 3, 1, 80, 40), (1, 9, 2, 2, 64, 8), (2, 21, 5, 0, 256, 24),
                                             (1, 18, 2, 1, 512, 72), (1, 13, 3, 2, 16, 8), (1, 11, 1, 1, 128, 120), (1, 12, 2, 1, 8, 8)])
def test_halves_that_are_an_odd_number_of_segments(dev, B, T, Hq, Hk, d, rot, layout, dtype):
    """Half of the turned channels is a multiple of four but not of eight: partners lie across vectors of eight channels."""
    test_rows(dev, B, T, Hq, Hk, d, rot, layout, dtype)


@pytest.mark.parametrize("poison", [float("nan"), float("inf")])
def test_a_channel_that_does_not_turn_keeps_to_its_head(dev, poison):
    """A value that is not finite reaches its own head alone (the norm takes it everywhere there), across segments too."""
    s = make(dev, 1, 8, 4, 2, 96, "bf16")
    table = gdn.rotary_table(24, device=dev)
    clean = gdn.norm_rotary(s["q"], s["k"], s["qw"], s["kw"], table, d=96, rot=24)
    s["q"][0, 3, 96 + 13] = poison
    got = gdn.norm_rotary(s["q"], s["k"], s["qw"], s["kw"], table, d=96, rot=24)
    keep = torch.ones_like(clean[0], dtype=torch.bool)
    keep[0, 3, 96:192] = False
    assert torch.equal(got[0][keep], clean[0][keep]) and torch.equal(got[1], clean[1])
