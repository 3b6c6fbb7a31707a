"""The operators beside the gated delta rule over many tokens, where a CTA or a warp goes on for long: several tokens of
rotary per CTA, and parameter gradients summed over many rows, positions and tiles."""
import numpy as np
import pytest
import torch

from linear_attention_sequence_qkv_gb300 import build, gdn
from oracle import layer_ops as O
from tests.test_recurrence_gpu import backward, forward
from tests.test_rotary_gpu import held as rotary_held

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


# -------------------------------------------------------------------- rotary
def rotary_input(dev, B, T, width, dtype, pad=0, seed=0):
    g = torch.Generator(device=dev).manual_seed(seed)
    return torch.randn((B, T, width + pad), generator=g, device=dev).to(ACT[dtype])[..., pad:]


# A CTA takes as many tokens as leave 608 of them (fewer with many heads or a wide table): 54003 tokens are 88 a CTA, the
# last CTA's fewer, and a row's end falls inside one. 24 pairs and more by 88 tokens take the loop for long tables (over
# 2048 entries), whose 256 threads 24 and 40 pairs do not divide.
@pytest.mark.parametrize("B,T,Hq,Hk,d,rot,layout,dtype,pad", [
    (3, 18001, 1, 0, 64, 64, "half", "bf16", 0),
    (3, 18001, 1, 0, 64, 48, "half", "bf16", 0),
    (3, 18001, 1, 0, 80, 80, "half", "fp16", 0),
    (3, 18001, 1, 0, 80, 80, "interleaved", "fp16", 0),
    (3, 18001, 1, 0, 64, 64, "half", "fp32", 0),
    (2, 40003, 1, 0, 64, 32, "interleaved", "fp32", 0),
    (2, 20001, 1, 0, 64, 64, "interleaved", "fp32", 1),
    (3, 18001, 1, 0, 64, 48, "half", "bf16", 3),
    (3, 18001, 1, 0, 48, 48, "interleaved", "bf16", 1),
    (2, 15013, 2, 1, 96, 32, "half", "bf16", 0),
    (2, 15013, 1, 1, 40, 20, "half", "fp16", 2),
    (2, 15013, 2, 1, 7, 6, "interleaved", "fp32", 0),
    (60000, 1, 1, 0, 64, 64, "half", "bf16", 0),
])
def test_several_tokens_per_block(dev, B, T, Hq, Hk, d, rot, layout, dtype, pad):
    x = rotary_input(dev, B, T, (Hq + Hk) * d, dtype, pad, seed=T + rot)
    q, k = x[..., :Hq * d], x[..., Hq * d:] if Hk else None
    off = torch.randint(0, 1 << 20, (B,), device=dev, generator=torch.Generator(device=dev).manual_seed(1)).to(torch.int32)
    pos = n64(off)[:, None] + np.arange(T)
    f = O.frequencies(rot)
    kw = dict(d=d, rot=rot, layout=layout, inverse=True, scale=0.75, offsets=off)
    qo, ko = gdn.rotary(q, k, gdn.rotary_table(rot, device=dev), **kw)
    rotary_held(qo, q, pos, f, d, rot, layout, dtype, True, 0.75)
    if Hk:
        rotary_held(ko, k, pos, f, d, rot, layout, dtype, True, 0.75)
    # in place: the same bits
    kept = x.clone()
    q2, k2 = kept[..., :Hq * d], kept[..., Hq * d:] if Hk else None
    gdn.rotary(q2, k2, gdn.rotary_table(rot, device=dev), q_out=q2, k_out=k2, **kw)
    assert torch.equal(q2, qo) or pad or Hk     # another alignment may take other vectors
    rotary_held(q2, q, pos, f, d, rot, layout, dtype, True, 0.75)


@pytest.mark.parametrize("rot,dtype,pad", [(64, "bf16", 0), (48, "fp16", 0), (40, "fp32", 0), (64, "bf16", 1)])
@pytest.mark.parametrize("given", ["offsets", "positions", "neither"])
def test_packed_tokens_across_blocks(dev, rot, dtype, pad, given):
    """54003 packed tokens: sequences that end inside a CTA's tokens and at its border (88), of one token and of none."""
    rng = np.random.default_rng(rot)
    lengths = [88, 176, 0, 1, 87, 1, 0, 5000] + list(rng.integers(0, 90, 500)) + [0, 1]
    lengths += [54003 - sum(lengths), 0]
    assert min(lengths) >= 0
    cu = torch.tensor([0] + list(np.cumsum(lengths)), dtype=torch.int32, device=dev)
    T, d = 54003, 64
    q = rotary_input(dev, 1, T, d, dtype, pad, seed=rot)
    kw, at = {}, np.concatenate([np.arange(n) for n in lengths])
    if given == "offsets":
        off = rng.integers(0, 1 << 20, len(lengths))
        kw["offsets"] = torch.tensor(off, dtype=torch.int32, device=dev)
        at = at + np.repeat(off, lengths)
    if given == "positions":
        at = rng.integers(-(1 << 20), 1 << 20, T)
        kw["positions"] = torch.tensor(at[None], dtype=torch.int32, device=dev)
    qo, _ = gdn.rotary(q, None, gdn.rotary_table(rot, device=dev), d=d, rot=rot, cu_seqlens=cu, **kw)
    rotary_held(qo, q, at[None], O.frequencies(rot), d, rot, "half", dtype)


# ---------------------------------------------------------------- group norm
def norm_reference(x, w, b, mean, rstd, dy, G, act):
    """The backward in fp64 from the forward's own mean and rstd, and bounds on what fp32 adds to each value.

    U is half a step of fp32. xh = (x - mean) rstd: two roundings. z: those, and one of the fma. The derivative of SiLU: its
    own argument's error by at most 0.5, an exponent's argument off by |z| U and a few U for the exponential, the sum and
    the reciprocal: (|z| + 8) 4 U. The means over a group: a chain of at most 16 a lane and vector and log2 of 256 lanes, then
    the product with 1 / count: 32 U of the mean absolute term; over positions, the chain goes over a chunk's (at most
    L, and 100 where L is thousands here) and the partials that a lane reads (at most 450). dx: eight roundings more. A
    parameter's sum: 16 rows, then the warp's sums of 16 rows (at most 64 here), then the block's eight, then partial rows by 32
    chains (at most 114 each, of 3648 rows) and a tree: 16 + 64 + 8 + 114 + 5 roundings of the sum of absolute values, 207."""
    U = O.U32
    chain = 32 + (0 if x.shape[1] == 1 else min(x.shape[1], 550))
    N, L, C = x.shape
    cg = C // G
    g4 = lambda t: t.double().view(N, L, G, cg)  # noqa: E731
    par = lambda t: t.double().view(1, 1, G, cg)  # noqa: E731
    st = lambda t: t.double().view(N, 1, G, 1)  # noqa: E731
    xh = (g4(x) - st(mean)) * st(rstd)
    w4, b4, dy4 = par(w), par(b), g4(dy)
    z = xh * w4 + b4
    ez = 2 * U * (xh * w4).abs() + U * z.abs()
    if act == "silu":
        sg = torch.sigmoid(z)
        da = sg * (1 + z * (1 - sg))
        eda = 0.5 * ez + (z.abs() + 8) * 4 * U
    else:
        da, eda = torch.ones_like(z), torch.zeros_like(z)
    del z, ez
    dz = dy4 * da
    edz = dy4.abs() * eda + U * dz.abs()
    del da, eda
    t, et = dz * w4, edz * w4.abs() + U * (dz * w4).abs()
    mean_of = lambda v: v.mean((1, 3), keepdim=True)  # noqa: E731
    m1, m2 = mean_of(t), mean_of(t * xh)
    em1 = mean_of(et) + chain * U * mean_of(t.abs())
    em2 = mean_of(et * xh.abs()) + (chain + 2) * U * mean_of((t * xh).abs())
    dx = st(rstd) * (t - m1 - xh * m2)
    ex = st(rstd).abs() * (et + em1 + xh.abs() * em2 + 2 * U * (xh * m2).abs() + 8 * U * (t.abs() + m1.abs() + (xh * m2).abs()))
    r = {"dx": dx.view(N, L, C), "dx_err": ex.view(N, L, C)}
    for name, v, ev in (("dweight", dz * xh, edz * xh.abs() + 2 * U * (dz * xh).abs()), ("dbias", dz, edz)):
        r[name] = v.sum((0, 1)).view(C)
        r[name + "_err"] = (ev.sum((0, 1)) + 207 * U * v.abs().sum((0, 1))).view(C)
    return r


def norm_held(got, r, name, dtype):
    rel, least = O.HALF_STEP[dtype]
    tol = r[name].abs() * rel + r[name + "_err"] * (1 + rel) + least
    use = ((got.double() - r[name]).abs() / tol).max().item()
    print(f"[group norm, long] {name} {dtype}: bound_use={use:.3f}")
    assert use <= 1.0, f"{name}: {use:.3f} of the bound"


# Rows a warp (or a block) takes: some forty to three hundred, no multiple of 16 nor of the six that are on their way.
@pytest.mark.parametrize("N,L,C,G,dtype,act", [
    (97301, 1, 64, 1, "bf16", "silu"),      # 8 lanes a group
    (97301, 1, 128, 1, "fp16", "silu"),     # 16
    (65541, 1, 512, 4, "fp16", "silu"),     # 16, four groups
    (97301, 1, 256, 1, "bf16", "silu"),     # 32
    (97301, 1, 256, 1, "bf16", "none"),     # three blocks per SM
    (97301, 1, 128, 1, "fp32", "silu"),
    (97301, 1, 24, 1, "bf16", "silu"),      # 4 lanes, one of them without channels
    (65541, 1, 512, 1, "bf16", "silu"),     # two vectors a lane
    (97301, 1, 33, 1, "bf16", "silu"),      # element by element, two a lane
    (97301, 1, 65, 5, "fp32", "silu"),      # element by element, five groups
    (14003, 1, 1032, 1, "bf16", "silu"),    # a block per group
    (14003, 1, 2072, 1, "fp32", "silu"),    # the same, two vectors a thread
    (14003, 1, 515, 1, "fp16", "silu"),     # the same, element by element
    (64, 2001, 64, 4, "bf16", "silu"),      # over positions
    (3, 40001, 40, 5, "fp32", "silu"),
    (64, 2001, 33, 1, "fp16", "silu"),
    (2, 700, 13200, 400, "fp32", "silu"),   # many sets of channels: a partial row per warp
    (5, 1200, 8200, 1, "bf16", "silu"),     # slabs of one group
])
def test_parameter_gradients_over_many_rows(dev, N, L, C, G, dtype, act):
    """dout and the activation's derivative have a sign: a block of 16 rows left out of one warp's sum would be off by some
    16, where the bound is of the order of 0.1 to 2."""
    g = torch.Generator(device=dev).manual_seed(N + C)
    x = torch.randn((N, L, C), generator=g, device=dev).to(ACT[dtype])
    w = (1.0 + 0.1 * torch.randn(C, generator=g, device=dev)).to(ACT[dtype])
    b = (1.0 + 0.1 * torch.randn(C, generator=g, device=dev)).to(ACT[dtype])
    dy = (x.float() + 1.0).to(ACT[dtype])
    f = gdn.group_norm_forward(x, w, b, groups=G, act=act)
    got = gdn.group_norm_backward(x, w, b, f.mean, f.rstd, dy, groups=G, act=act)
    r = norm_reference(x, w, b, f.mean, f.rstd, dy, G, act)
    norm_held(got.dx, r, "dx", dtype)
    norm_held(got.dweight, r, "dweight", "fp32")
    norm_held(got.dbias, r, "dbias", "fp32")


# ----------------------------------------------------------------- recurrence
@pytest.mark.parametrize("dtype,B,T,D", [("bf16", 240, 1115, 64), ("fp32", 160, 2231, 32), ("bf16", 160, 1115, 63),
                                         ("fp16", 1, 1115, 15360), ("fp32", 1, 2231, 5120)])
def test_parameter_gradients_over_many_tiles(dev, dtype, B, T, D):
    """So many chains that one CTA walks each of them: 35 tiles, two times the 16 that a thread sums at first and three more.
    x, dout and (with short memory) the gates' gradients are mostly of one sign: the 64 tokens of 16 tiles left out of one
    thread's row would move dA_log and ddt_bias by 2e-4 of their sums, the bound is a fifth of that. With one row, it is
    five packed sequences. The sums' roundings: four tokens, 16 tiles, three of those and one, 16 groups of tokens; then
    the rows' by eight chains and those eight."""
    g = torch.Generator().manual_seed(T + D)
    randn = lambda *v: torch.randn(*v, generator=g)  # noqa: E731
    act = ACT[dtype]
    cu = torch.tensor([0, 300, 300, 301, 801, T], dtype=torch.int32) if B == 1 else None
    N = B if cu is None else 5
    s = {"x": randn(B, T, D).abs(), "a": 0.3 * randn(B, T, D), "b": randn(B, T, D), "dout": randn(B, T, D).abs()}
    s = {k: v.to(act).to(dev) for k, v in s.items()}
    s.update(A_log=(0.1 * randn(D) - 0.5).to(dev), dt_bias=(0.1 * randn(D) - 0.5).to(dev), h0=randn(N, D).abs().to(dev),
             dfinal=randn(N, D).abs().to(dev), cu=None if cu is None else cu.to(dev))
    f = forward(s, want_chunk_states=True)
    got = backward(s, f.chunk_states)
    assert gdn.gdn_device_status(got.workspace) == gdn.GDN_OK
    # rows side by side as channels of one sequence
    flat = lambda t: n64(t).transpose(1, 0, 2).reshape(T, B * D)  # noqa: E731
    wide = lambda t: np.tile(n64(t), B)  # noqa: E731
    state = lambda t: n64(t).reshape(N // B, B * D)  # noqa: E731
    r = O.recurrence(flat(s["x"]), flat(s["a"]), flat(s["b"]), wide(s["A_log"]), wide(s["dt_bias"]),
                     [0, T] if cu is None else cu.tolist(), state(s["h0"]), flat(s["dout"]), state(s["dfinal"]))
    for name, t in (("out", f.out), ("dx", got.dx), ("da", got.da), ("db", got.db)):
        ref, tol = r[name], O.bound(r[name], r[name + "_err"], dtype)
        use = (np.abs(flat(t) - ref) / tol).max()
        print(f"[recurrence, long] {name} {dtype}: bound_use={use:.3f}")
        assert use <= 1.0, name
    z = flat(s["a"]) + wide(s["dt_bias"])
    # dA_log sums dg g = da softplus(z) / sigmoid(z)
    for name, t, ratio in (("dA_log", got.dA_log, np.logaddexp(0, z) * (1 + np.exp(-z))), ("ddt_bias", got.ddt_bias, np.ones_like(z))):
        total = lambda v: v.sum(0).reshape(B, D).sum(0)  # noqa: E731
        assert np.allclose(total(r["da"] * ratio), r[name].reshape(B, D).sum(0), rtol=1e-9)
        err = total(r["da_err"] * ratio) + (4 + 16 + 4 + 16 + B / 8 + 8) * O.U32 * total(np.abs(r["da"]) * ratio)
        ref = r[name].reshape(B, D).sum(0)
        use = (np.abs(n64(t) - ref) / O.bound(ref, err, "fp32")).max()
        print(f"[recurrence, long] {name} {dtype}: bound_use={use:.3f} bound={(err / np.abs(ref)).max():.2e}")
        assert use <= 1.0, name


@pytest.mark.parametrize("dtype,D", [("bf16", 72), ("fp32", 9)])
def test_thousands_of_short_sequences(dev, dtype, D):
    """Five thousand sequences of none to five tokens, with runs of empty ones at both ends."""
    rng = np.random.default_rng(D)
    lengths = [0] * 300 + list(rng.integers(0, 6, 4000)) + [0] * 500 + [1] * 40 + [0] * 200
    T, N = int(sum(lengths)), len(lengths)
    cu = np.concatenate([[0], np.cumsum(lengths)])
    g = torch.Generator().manual_seed(D)
    randn = lambda *v: torch.randn(*v, generator=g)  # noqa: E731
    s = {k: randn(1, T, D).to(ACT[dtype]).to(dev) for k in ("x", "a", "b", "dout")}
    s.update(A_log=(0.5 * randn(D) - 1.0).to(dev), dt_bias=(randn(D) - 2.0).to(dev), h0=randn(N, D).to(dev),
             dfinal=randn(N, D).to(dev), cu=torch.tensor(cu, dtype=torch.int32, device=dev))
    f = forward(s, want_chunk_states=True)
    got = backward(s, f.chunk_states)
    assert gdn.gdn_device_status(got.workspace) == gdn.GDN_OK
    flat = lambda t: n64(t).reshape(-1, D)  # noqa: E731
    r = O.recurrence(flat(s["x"]), flat(s["a"]), flat(s["b"]), n64(s["A_log"]), n64(s["dt_bias"]), cu.tolist(), n64(s["h0"]),
                     flat(s["dout"]), n64(s["dfinal"]))
    for name, t in (("out", f.out), ("final", f.final_state), ("dx", got.dx), ("da", got.da), ("db", got.db),
                    ("dA_log", got.dA_log), ("ddt_bias", got.ddt_bias), ("dstate", got.dinitial_state)):
        tol = O.bound(r[name], r[name + "_err"], dtype if name in ("out", "dx", "da", "db") else "fp32")
        use = (np.abs(n64(t).reshape(r[name].shape) - r[name]) / tol).max()
        print(f"[recurrence, many] {name} {dtype}: bound_use={use:.3f}")
        assert use <= 1.0, name
