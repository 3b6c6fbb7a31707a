"""Gated linear recurrence on the GPU against the fp64 definition (oracle/layer_ops.py), within the
error bounds computed there plus one rounding to the activation type."""
import numpy as np
import pytest
import torch

from linear_attention_sequence_qkv_gb300 import build, gdn
from oracle import layer_ops as O

pytestmark = pytest.mark.gpu
ACT = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
GRADS = ("dx", "da", "db", "dA_log", "ddt_bias", "dstate")


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    build.build()
    gdn.load()
    return torch.device("cuda:0")


def n64(t):
    return t.detach().double().cpu().numpy()


def make(dev, B, T, D, dtype, lengths=None, seed=0, layout="dense", long_memory=True, init=True):
    """Inputs on the GPU; layout "wide": x, a, b are views into one [B, T, 3D + 1] buffer."""
    g = torch.Generator().manual_seed(seed)
    randn = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    cu = None
    if lengths is not None:
        cu = torch.tensor([0] + list(np.cumsum(lengths)), dtype=torch.int32)
        B, T = 1, int(cu[-1])
    buf = randn(B, T, 3 * D + (1 if layout == "wide" else 0)).to(ACT[dtype]).to(dev)
    x, a, b = (buf[..., i * D:(i + 1) * D] for i in range(3))
    if layout == "dense":
        x, a, b = (t.contiguous() for t in (x, a, b))
    N = B if cu is None else len(lengths)
    A_log = randn(D) * 0.5 + (-1.0 if long_memory else 1.0)
    bias = randn(D) - (4.0 if long_memory else 0.0)
    s = dict(x=x, a=a, b=b, A_log=A_log.to(dev), dt_bias=bias.to(dev), cu=None if cu is None else cu.to(dev),
             h0=randn(N, D).to(dev) if init else None, dout=randn(B, T, D).to(ACT[dtype]).to(dev),
             dfinal=randn(N, D).to(dev), starts=[i * T for i in range(B + 1)] if cu is None else cu.tolist(), dtype=dtype)
    return s


def oracle(s, grads=True):
    D = s["x"].shape[-1]
    flat = lambda t: n64(t).reshape(-1, D)  # noqa: E731
    return O.recurrence(flat(s["x"]), flat(s["a"]), flat(s["b"]), n64(s["A_log"]), n64(s["dt_bias"]), s["starts"],
                        None if s["h0"] is None else n64(s["h0"]), flat(s["dout"]) if grads else None, n64(s["dfinal"]))


def forward(s, **kw):
    return gdn.recurrence_forward(s["x"], s["a"], s["b"], s["A_log"], s["dt_bias"], s["cu"], s["h0"], **kw)


def backward(s, chunk_states, **kw):
    return gdn.recurrence_backward(s["x"], s["a"], s["b"], s["A_log"], s["dt_bias"], s["dout"], s["dfinal"], chunk_states,
                                   s["cu"], s["h0"], **kw)


def held(got, r, name, dtype):
    ref, tol = r[name], O.bound(r[name], r[name + "_err"], dtype)
    got = n64(got).reshape(ref.shape)
    assert np.isfinite(got).all(), f"{name}: not finite"
    use = (np.abs(got - ref) / tol).max() if ref.size else 0.0
    print(f"[recurrence] {name} {dtype}: bound_use={use:.3f}")
    assert use <= 1.0, f"{name}: {use:.3f} of the bound"


def check_all(s):
    r = oracle(s)
    f = forward(s, want_chunk_states=True)
    assert gdn.gdn_device_status(f.workspace) == gdn.GDN_OK
    held(f.out, r, "out", s["dtype"])
    held(f.final_state, r, "final", "fp32")
    g = backward(s, f.chunk_states)
    assert gdn.gdn_device_status(g.workspace) == gdn.GDN_OK
    for name, t in zip(GRADS, (g.dx, g.da, g.db, g.dA_log, g.ddt_bias, g.dinitial_state)):
        held(t, r, name, s["dtype"] if name in ("dx", "da", "db") else "fp32")
    # without the forward's chunk states: the same values, bit for bit
    g2 = backward(s, None)
    for name in ("dx", "da", "db", "dA_log", "ddt_bias", "dinitial_state"):
        assert torch.equal(getattr(g, name), getattr(g2, name)), name
    return f, g


SHAPES = [(1, 1, 1), (3, 1, 8), (2, 2, 3), (1, 63, 40), (2, 64, 64), (1, 65, 100), (2, 129, 257), (1, 300, 72), (5, 17, 130)]


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("B,T,D", SHAPES)
def test_rows(dev, B, T, D, dtype):
    check_all(make(dev, B, T, D, dtype, seed=B * T + D))


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("B,T,D,long_memory", [(1, 2000, 64, True), (2, 1111, 24, True), (1, 1500, 9, False)])
def test_long_rows(dev, B, T, D, long_memory, dtype):
    check_all(make(dev, B, T, D, dtype, long_memory=long_memory, seed=T))


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("lengths", [[1], [0], [0, 0, 5, 0], [64, 64], [63, 1, 1, 64, 0, 200, 3], [1] * 70, [500, 2, 700]])
def test_packed(dev, lengths, dtype):
    check_all(make(dev, 1, 0, 72, dtype, lengths=lengths, seed=sum(lengths)))


@pytest.mark.parametrize("D", [64, 96, 33])
def test_views_and_no_state(dev, D):
    s = make(dev, 2, 150, D, "bf16", layout="wide", init=False)
    s["dfinal"] = torch.zeros_like(s["dfinal"])
    check_all(s)
    # batch rows that are one broadcast row: each row's own gradients
    s = make(dev, 1, 70, D, "bf16")
    for k in ("x", "a", "b"):
        s[k] = s[k].expand(3, -1, -1)
    s["h0"], s["dfinal"] = s["h0"].expand(3, -1).contiguous(), s["dfinal"].expand(3, -1).contiguous()
    s["dout"], s["starts"] = s["dout"].expand(3, -1, -1).contiguous(), [0, 70, 140, 210]
    check_all(s)


def test_packed_equals_separate_calls(dev):
    lengths = [130, 1, 0, 77, 256]
    s = make(dev, 1, 0, 64, "fp32", lengths=lengths)
    r = oracle(s, grads=False)
    out = forward(s).out
    for n, (t0, t1) in enumerate(zip(s["starts"][:-1], s["starts"][1:])):
        if t1 > t0:
            one = gdn.recurrence_forward(s["x"][:, t0:t1], s["a"][:, t0:t1], s["b"][:, t0:t1], s["A_log"], s["dt_bias"], None,
                                         s["h0"][n:n + 1])
            tol = O.bound(r["out"][t0:t1], r["out_err"][t0:t1], "fp32")
            assert (np.abs(n64(one.out[0]) - n64(out[0, t0:t1])) <= 2 * tol).all()


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_extreme_gates(dev, dtype):
    """Gates at both ends: no decay at all, none left, writes shut and open."""
    vals = torch.tensor([-100.0, -30.0, -17.0, -10.0, -1.0, 0.0, 1.0, 10.0, 30.0, 100.0])
    s = make(dev, 1, 100, 64, dtype, long_memory=False)
    s["a"] = vals[torch.randint(0, 10, (1, 100, 64), generator=torch.Generator().manual_seed(1))].to(ACT[dtype]).to(dev)
    s["b"] = vals[torch.randint(0, 10, (1, 100, 64), generator=torch.Generator().manual_seed(2))].to(ACT[dtype]).to(dev)
    s["dt_bias"].zero_()
    s["A_log"] = torch.linspace(-12.0, 3.0, 64, device=dev)
    check_all(s)


def test_gates_at_infinity(dev):
    """a = -inf: the state is kept and nothing written; a = inf: it is replaced; b = -inf: nothing is written.
    Their gradients are finite (zero where the gates are saturated)."""
    s = make(dev, 1, 4, 8, "fp32")
    s["a"][0, 1], s["a"][0, 2], s["b"][0, 3] = -float("inf"), float("inf"), -float("inf")
    f = forward(s, want_chunk_states=True)
    out = f.out[0]
    assert torch.equal(out[1], out[0])
    assert torch.allclose(out[2], torch.sigmoid(s["b"][0, 2]) * s["x"][0, 2], rtol=1e-6)
    alpha = torch.exp(-torch.exp(s["A_log"]) * torch.nn.functional.softplus(s["a"][0, 3] + s["dt_bias"]))
    assert torch.allclose(out[3], alpha * out[2], rtol=1e-5)
    g = backward(s, f.chunk_states)
    assert torch.isfinite(g.dx).all() and torch.isfinite(g.db).all() and torch.isfinite(g.da[0, [0, 1, 3]]).all()
    assert (g.da[0, 1] == 0).all() and (g.dx[0, 1] == 0).all() and (g.db[0, 3] == 0).all()


def test_nan_stays_in_its_channel_and_sequence(dev):
    s = make(dev, 1, 0, 64, "bf16", lengths=[100, 100, 100])
    f = forward(s, want_chunk_states=True)
    clean, g = f.out.clone(), backward(s, f.chunk_states)
    s["dout"][0, 160, 9] = float("nan")      # reaches back to its sequence's first token
    g2 = backward(s, f.chunk_states)
    bad = torch.isnan(g2.dx)
    assert bad[0, 100:161, 9].all() and bad.sum() == 61 and torch.equal(g2.dx[~bad], g.dx[~bad])
    assert torch.isnan(g2.dinitial_state).nonzero().tolist() == [[1, 9]]
    s["x"][0, 130, 7] = float("nan")
    got = forward(s).out
    bad = torch.isnan(got)
    assert bad[0, 130:200, 7].all() and bad.sum() == 70
    assert torch.equal(got[~bad], clean[~bad])


def test_malformed_seqlens_write_nothing(dev):
    s = make(dev, 1, 0, 64, "bf16", lengths=[60, 70])
    for cu in ([0, 131, 130], [1, 60, 130], [0, 60, 129], [0, -5, 130], [0, 60, 131]):
        s["cu"] = torch.tensor(cu, dtype=torch.int32, device=dev)
        d = gdn.recurrence_desc_for(s["x"], s["a"], s["b"], s["cu"])
        f, g = gdn.alloc_recurrence(d, dev, want_chunk_states=True), gdn.alloc_recurrence_grads(d, dev)
        for t in (f.out, f.final_state, f.chunk_states, g.dx, g.da, g.db, g.dA_log, g.ddt_bias, g.dinitial_state):
            t.fill_(7.0)
        forward(s, bufs=f)
        assert gdn.gdn_device_status(f.workspace) == gdn.GDN_ERR_DEVICE_SEQLENS
        for cs in (f.chunk_states, None):
            backward(s, cs, grads=g)
            assert gdn.gdn_device_status(g.workspace) == gdn.GDN_ERR_DEVICE_SEQLENS
        for t in (f.out, f.final_state, f.chunk_states, g.dx, g.da, g.db, g.dA_log, g.ddt_bias, g.dinitial_state):
            assert (t == 7.0).all()
    # the next well-formed call on the same workspaces
    s["cu"] = torch.tensor([0, 60, 130], dtype=torch.int32, device=dev)
    forward(s, bufs=f)
    assert gdn.gdn_device_status(f.workspace) == gdn.GDN_OK
    held(f.out, oracle(s), "out", "bf16")


def test_no_tokens(dev):
    s = make(dev, 3, 0, 40, "bf16")
    f = forward(s, want_chunk_states=True)
    assert torch.equal(f.final_state, s["h0"])
    g = backward(s, f.chunk_states)
    assert torch.equal(g.dinitial_state, s["dfinal"])
    assert (g.dA_log == 0).all() and (g.ddt_bias == 0).all()


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("B,D", [(1, 1), (3, 40), (7, 257), (64, 512)])
def test_steps_follow_the_forward(dev, B, D, dtype):
    s = make(dev, B, 5, D, dtype, layout="wide")
    r = oracle(s, grads=False)
    state = s["h0"].clone()
    outs = [gdn.recurrence_step(s["x"][:, t:t + 1], s["a"][:, t:t + 1], s["b"][:, t:t + 1], s["A_log"], s["dt_bias"], state)
            for t in range(5)]
    held(torch.cat(outs, 1), r, "out", dtype)
    held(state, r, "final", "fp32")


def test_split_call_continues_from_the_final_state(dev):
    s = make(dev, 2, 200, 64, "fp32")
    r = oracle(s, grads=False)
    half = lambda t, lo, hi: t[:, lo:hi]  # noqa: E731
    first = gdn.recurrence_forward(*(half(s[k], 0, 77) for k in "xab"), s["A_log"], s["dt_bias"], None, s["h0"])
    # initial and final state may be one tensor
    bufs = gdn.alloc_recurrence(gdn.recurrence_desc_for(*(half(s[k], 77, 200) for k in "xab")), dev)
    bufs.final_state = first.final_state
    rest = gdn.recurrence_forward(*(half(s[k], 77, 200) for k in "xab"), s["A_log"], s["dt_bias"], None, first.final_state,
                                  bufs=bufs)
    held(torch.cat([first.out, rest.out], 1), r, "out", "fp32")
    held(rest.final_state, r, "final", "fp32")


def test_repeatable_and_guarded(dev):
    """Two runs give the same bits; nothing is written around the outputs."""
    s = make(dev, 2, 333, 200, "bf16")
    f, g = check_all(s)
    f2 = forward(s, want_chunk_states=True)
    assert torch.equal(f.out, f2.out) and torch.equal(f.chunk_states, f2.chunk_states)
    g2 = backward(s, f2.chunk_states)
    for name in ("dx", "da", "db", "dA_log", "ddt_bias", "dinitial_state"):
        assert torch.equal(getattr(g, name), getattr(g2, name)), name
    n = f.out.numel()
    wide = torch.full((n + 512,), 3.0, dtype=torch.bfloat16, device=dev)
    b = gdn.alloc_recurrence(f.desc, dev)
    b.out = wide[256:256 + n].view(f.out.shape)
    forward(s, bufs=b)
    assert torch.equal(b.out, f.out) and (wide[:256] == 3).all() and (wide[256 + n:] == 3).all()


def test_captured_and_replayed_on_another_stream(dev):
    s = make(dev, 1, 0, 128, "bf16", lengths=[300, 41])
    d = gdn.recurrence_desc_for(s["x"], s["a"], s["b"], s["cu"])
    f, g = gdn.alloc_recurrence(d, dev, want_chunk_states=True), gdn.alloc_recurrence_grads(d, dev)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        forward(s, bufs=f)
        backward(s, f.chunk_states, grads=g)
    side = torch.cuda.Stream()
    for seed in (5, 6):
        new = make(dev, 1, 0, 128, "bf16", lengths=[300, 41], seed=seed)
        for k in ("x", "a", "b", "dout"):
            s[k].copy_(new[k])
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            graph.replay()
        side.synchronize()
        r = oracle(s)
        held(f.out, r, "out", "bf16")
        held(g.da, r, "da", "bf16")
        held(g.dA_log, r, "dA_log", "fp32")


def test_two_calls_at_once(dev):
    """Calls on two streams with their own buffers."""
    ss = [make(dev, 1, 700, 256, "bf16", seed=i) for i in (1, 2)]
    want = [forward(s).out.clone() for s in ss]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = []
    for _ in range(5):
        got = []
        for s, st in zip(ss, streams):
            with torch.cuda.stream(st):
                got.append(forward(s).out)
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        assert torch.equal(w, g)


def test_offsets_past_32_bits(dev):
    """More than 2^32 elements a tensor: the tail of the row, checked from the state carried into it, and its gradients from a call over the tail alone."""
    T, D = 262144 + 70, 16384
    g = torch.Generator(device=dev).manual_seed(0)
    x = torch.randn((1, T, D), generator=g, dtype=torch.bfloat16, device=dev)
    a = torch.randn((1, T, D), generator=g, dtype=torch.bfloat16, device=dev)
    A_log, bias = torch.full((D,), -1.0, device=dev), torch.full((D,), -4.0, device=dev)
    f = gdn.recurrence_forward(x, a, x, A_log, bias, want_chunk_states=True)
    t0 = 262144
    assert t0 * D >= 2 ** 32
    tail = [t[:, t0:].contiguous() for t in (x, a, x)]
    state = f.chunk_states[:, t0 // gdn.GDN_RECURRENCE_CHUNK].contiguous()
    one = gdn.recurrence_forward(*tail, A_log, bias, None, state, want_chunk_states=True)
    r = O.recurrence(*(n64(t).reshape(-1, D)[:, :512] for t in tail), n64(A_log)[:512], n64(bias)[:512], [0, T - t0],
                     n64(state)[:, :512])
    tol = O.bound(r["out"], r["out_err"], "bf16")
    assert (np.abs(n64(f.out[0, t0:, :512]) - r["out"]) <= tol).all()
    assert (f.out[0, t0:].float() - one.out[0].float()).abs().max() <= 2.0 ** -6 * one.out.float().abs().max()
    del one
    grads = gdn.recurrence_backward(x, a, x, A_log, bias, x, None, f.chunk_states)
    short = gdn.recurrence_backward(*tail, A_log, bias, tail[0], None, None, None, state)
    # the tail's gradients depend on nothing before it but the carried state
    for name in ("dx", "da", "db"):
        u, v = getattr(grads, name)[0, t0:].float(), getattr(short, name)[0].float()
        assert ((u - v).abs() <= 2.0 ** -7 * v.abs() + 1e-5).all(), name


def test_gradient_against_differences(dev):
    """The forward's own directional difference: central, step 2^-6, so off by its third derivative (of order 1
    here, times 2^-12 / 6) and by the outputs' fp32 errors over the step."""
    s = make(dev, 2, 90, 64, "fp32", long_memory=False)
    f = forward(s, want_chunk_states=True)
    g = backward(s, f.chunk_states)
    gen = torch.Generator().manual_seed(9)
    step = 2.0 ** -6
    loss = lambda r: (n64(r.out) * n64(s["dout"])).sum() + (n64(r.final_state) * n64(s["dfinal"])).sum()  # noqa: E731
    for key, grad in (("x", g.dx), ("a", g.da), ("b", g.db), ("A_log", g.dA_log), ("dt_bias", g.ddt_bias),
                      ("h0", g.dinitial_state)):
        v = torch.randn(s[key].shape, generator=gen).to(dev)
        ends = []
        for sign in (1.0, -1.0):
            moved = dict(s)
            moved[key] = s[key] + sign * step * v
            ends.append(loss(forward(moved)))
        diff, want = (ends[0] - ends[1]) / (2 * step), (n64(grad) * n64(v)).sum()
        scale = np.linalg.norm(n64(grad)) * np.sqrt(1.0)   # the derivative along v is of this size
        assert abs(diff - want) <= 2e-2 * scale, (key, diff, want, scale)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_wait_timeout_reported_then_next_call_correct(dev, dtype):
    """The bounded waits for tiles (gdn_set_wait_test_mode): reported, and the next call is right."""
    s = make(dev, 1, 1000, 256, dtype)
    f = forward(s, want_chunk_states=True)
    g = backward(s, f.chunk_states)
    assert gdn.gdn_device_status(g.workspace) == gdn.GDN_OK
    torch.cuda.synchronize()
    gdn.gdn_set_wait_test_mode(1)
    try:
        bad = forward(s)
        status = gdn.gdn_device_status(bad.workspace), gdn.gdn_device_status(backward(s, f.chunk_states).workspace)
    finally:
        gdn.gdn_set_wait_test_mode(0)
    assert status == (gdn.GDN_ERR_DEVICE_TIMEOUT,) * 2
    again = forward(s, bufs=bad)
    assert gdn.gdn_device_status(again.workspace) == gdn.GDN_OK and torch.equal(again.out, f.out)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("B,T,D", [(1, 1000, 64), (12, 530, 32), (13, 530, 30), (20, 420, 32), (21, 420, 31), (28, 400, 32),
                                   (29, 400, 32), (1, 513, 832), (1, 513, 835)])
def test_every_number_of_ctas_per_row(dev, B, T, D, dtype):
    """Rows by channel slabs around the counts where the number of CTAs per row changes, rows long enough to use them."""
    check_all(make(dev, B, T, D, dtype, seed=B + T + D))


@pytest.mark.parametrize("D", [64, 63])
def test_long_packed_row_of_few_channels(dev, D):
    lengths = [700, 0, 1, 31, 32, 33, 1, 900, 511, 0]
    check_all(make(dev, 1, sum(lengths), D, "bf16", seed=D, lengths=lengths))


def test_elements_next_to_unmapped_rows_are_not_needed(dev):
    """Odd rows at the very start and end of their own buffers, guarded by NaN: nothing outside the rows counts."""
    B, T, D = 2, 75, 37
    s = make(dev, B, T, D, "fp16", seed=5)
    whole = forward(s, want_chunk_states=True)
    grads = backward(s, whole.chunk_states)
    for name in ("x", "a", "b"):
        buf = torch.full((B * T * D + 2 * D,), float("nan"), dtype=s[name].dtype, device=dev)
        view = buf[D:D + B * T * D].view(B, T, D)
        view.copy_(s[name])
        s[name] = view
    again = forward(s, want_chunk_states=True)
    assert torch.equal(again.out, whole.out) and torch.equal(again.final_state, whole.final_state)
    after = backward(s, again.chunk_states)
    for name in ("dx", "da", "db", "dA_log", "ddt_bias", "dinitial_state"):
        assert torch.equal(getattr(after, name), getattr(grads, name)), name


@pytest.mark.parametrize("which", ["chunk_states", "dout", "x", "A_log", "dt_bias", "h0", "dfinal"])
def test_tensors_aligned_to_their_elements_only(dev, which):
    """Each tensor in turn starts one element behind a 16-byte boundary: the same values, or to rounding."""
    s = make(dev, 2, 70, 64, "bf16", seed=3)
    r = oracle(s)
    chunk = forward(s, want_chunk_states=True).chunk_states

    def shifted(t):
        buf = torch.zeros(t.numel() + 8, dtype=t.dtype, device=dev)
        view = buf[1:1 + t.numel()].view(t.shape)
        view.copy_(t)
        assert view.data_ptr() % 16 == t.element_size() and view.is_contiguous()
        return view

    if which == "chunk_states":
        chunk = shifted(chunk)
    else:
        s[which] = shifted(s[which])
    f = forward(s)
    held(f.out, r, "out", "bf16")
    g = backward(s, chunk)
    assert gdn.gdn_device_status(g.workspace) == gdn.GDN_OK
    for name, t in zip(GRADS, (g.dx, g.da, g.db, g.dA_log, g.ddt_bias, g.dinitial_state)):
        held(t, r, name, "bf16" if name in ("dx", "da", "db") else "fp32")


def test_timeout_of_the_recomputed_states_is_reported(dev):
    """A backward that recomputes the states and itself waits for no copy still reports the forward's timeout."""
    s = make(dev, 1, 1000, 256, "bf16")
    want = backward(s, None)
    buf = torch.zeros(s["dout"].numel() + 8, dtype=torch.bfloat16, device=dev)
    view = buf[1:1 + s["dout"].numel()].view(s["dout"].shape)   # no copies into shared memory from here
    view.copy_(s["dout"])
    s["dout"] = view
    torch.cuda.synchronize()
    gdn.gdn_set_wait_test_mode(1)
    try:
        status = gdn.gdn_device_status(backward(s, None).workspace)
    finally:
        gdn.gdn_set_wait_test_mode(0)
    assert status == gdn.GDN_ERR_DEVICE_TIMEOUT
    g = backward(s, None)
    assert gdn.gdn_device_status(g.workspace) == gdn.GDN_OK
    assert torch.allclose(g.dx.float(), want.dx.float(), rtol=1e-2, atol=1e-2)
