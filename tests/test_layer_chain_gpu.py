"""The operators beside the gated delta rule as they are used together: a rotating recurrent layer core,
x -> rotary(+) -> gated linear recurrence -> rotary(-) -> group norm with SiLU, over packed sequences.

Rotating by +p theta before the recurrence and by -p theta after it makes the state of each channel pair, whose
two channels share their gates, a complex number with the eigenvalue alpha e^(-i theta): the chain is checked
against that complex recurrence in fp64, forward and backward, and token by token."""
import numpy as np
import pytest
import torch

from linear_attention_sequence_qkv_gb300 import build, gdn
from oracle import layer_ops as O

pytestmark = pytest.mark.gpu
H, DH, ROT = 4, 32, 32
D = H * DH


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    build.build()
    gdn.load()
    return torch.device("cuda:0")


def pair_shared(t):
    """Both channels of each interleaved pair get the first one's value."""
    return t[..., 0::2].repeat_interleave(2, dim=-1).contiguous()


def make(dev, lengths, dtype, seed=0):
    g = torch.Generator().manual_seed(seed)
    randn = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    T = sum(lengths)
    s = {"x": randn(1, T, D), "a": pair_shared(randn(1, T, D)), "b": pair_shared(randn(1, T, D)), "dout": randn(T, 1, D)}
    s = {k: v.to(dtype).to(dev) for k, v in s.items()}
    s.update(A_log=pair_shared(0.5 * randn(D) - 1.0).to(dev), dt_bias=pair_shared(randn(D) - 3.0).to(dev),
             w=(1.0 + 0.1 * randn(D)).to(dev), bias=(0.1 * randn(D)).to(dev),
             cu=torch.tensor([0] + list(np.cumsum(lengths)), dtype=torch.int32, device=dev), lengths=lengths,
             table=gdn.rotary_table(ROT, device=dev))
    return s


def chain(s):
    kw = dict(d=DH, rot=ROT, layout="interleaved", cu_seqlens=s["cu"])
    v, _ = gdn.rotary(s["x"], None, s["table"], **kw)
    f = gdn.recurrence_forward(v, s["a"], s["b"], s["A_log"], s["dt_bias"], s["cu"], want_chunk_states=True)
    y, _ = gdn.rotary(f.out, None, s["table"], inverse=True, **kw)
    y = y.view(-1, 1, D)
    n = gdn.group_norm_forward(y, s["w"], s["bias"], groups=H)
    return v, f, y, n


def chain_backward(s, v, f, y, n):
    kw = dict(d=DH, rot=ROT, layout="interleaved", cu_seqlens=s["cu"])
    gn = gdn.group_norm_backward(y, s["w"], s["bias"], n.mean, n.rstd, s["dout"], groups=H)
    dh, _ = gdn.rotary(gn.dx.view(1, -1, D), None, s["table"], **kw)
    gr = gdn.recurrence_backward(v, s["a"], s["b"], s["A_log"], s["dt_bias"], dh, None, f.chunk_states, s["cu"])
    dx, _ = gdn.rotary(gr.dx, None, s["table"], inverse=True, **kw)
    return dx, gr, gn


def reference(s, x):
    """The complex recurrence in fp64 torch, differentiable."""
    a, b = s["a"].cpu().double()[0, :, 0::2], s["b"].cpu().double()[0, :, 0::2]
    g = -s["A_log"].cpu().double()[0::2].exp() * torch.nn.functional.softplus(a + s["dt_bias"].cpu().double()[0::2])
    u = torch.sqrt(-torch.expm1(2 * g)) * torch.sigmoid(b) * torch.complex(x[0, :, 0::2], x[0, :, 1::2])
    theta = torch.from_numpy(np.tile(O.frequencies(ROT), H))
    eig = torch.exp(torch.complex(g, -theta.expand_as(g)))
    rows, t = [], 0
    for L in s["lengths"]:
        h = torch.zeros(D // 2, dtype=torch.complex128)
        for _ in range(L):
            h = eig[t] * h + u[t]
            rows.append(h)
            t += 1
    y = torch.view_as_real(torch.stack(rows)).reshape(-1, 1, D)
    yg = y.view(-1, 1, H, DH)
    var, mean = torch.var_mean(yg, dim=-1, keepdim=True, correction=0)
    z = ((yg - mean) / torch.sqrt(var + 1e-5)).reshape(y.shape) * s["w"].cpu().double() + s["bias"].cpu().double()
    return torch.nn.functional.silu(z)


@pytest.mark.parametrize("dtype,tol", [(torch.float32, 1e-4), (torch.bfloat16, 4e-2), (torch.float16, 5e-3)])
def test_rotating_layer_forward_and_backward(dev, dtype, tol):
    """Tolerance relative to each result's 2-norm: three roundings to the activation type on the way (2^-8, 2^-11 or
    2^-24 each), magnified by the norm's rstd (below 3 here) and the gradients' second use of them."""
    s = make(dev, [70, 1, 200, 33], dtype)
    v, f, y, n = chain(s)
    dx, gr, gn = chain_backward(s, v, f, y, n)
    x = s["x"].cpu().double().requires_grad_(True)
    ref = reference(s, x)
    (want,) = torch.autograd.grad(ref, x, s["dout"].cpu().double())
    off = lambda got, w: float((got.cpu().double() - w).norm() / w.norm())  # noqa: E731
    print("[chain]", dtype, off(n.out, ref.detach()), off(dx, want))
    assert off(n.out, ref.detach()) <= tol and off(dx, want) <= tol


def test_tokens_one_by_one_equal_the_packed_pass(dev):
    s = make(dev, [40], torch.float32)
    n = chain(s)[3]
    state = torch.zeros((1, D), device=dev)
    off = torch.zeros(1, dtype=torch.int32, device=dev)
    rows = []
    for t in range(40):
        v, _ = gdn.rotary(s["x"][:, t:t + 1], None, s["table"], d=DH, rot=ROT, layout="interleaved", offsets=off)
        h = gdn.recurrence_step(v, s["a"][:, t:t + 1], s["b"][:, t:t + 1], s["A_log"], s["dt_bias"], state)
        y, _ = gdn.rotary(h, None, s["table"], d=DH, rot=ROT, layout="interleaved", offsets=off, inverse=True)
        rows.append(gdn.group_norm_forward(y, s["w"], s["bias"], groups=H).out)
        off += 1
    got = torch.cat(rows, 0)
    assert float((got - n.out).norm() / n.out.norm()) <= 1e-5


def test_norm_of_the_delta_rule_output(dev):
    """The group norm over the heads of gdn_forward's output, the layer it stands beside."""
    from linear_attention_sequence_qkv_gb300.workloads import WORKLOADS, make_inputs, replace, to_device
    w = replace(WORKLOADS["ragged_fp16"], T=70)
    out = gdn.forward(to_device(make_inputs(w), dev)).out            # [B, T, Hv, dv]
    x = out.view(-1, 1, w.Hv * w.dv)
    f = gdn.group_norm_forward(x, groups=w.Hv, act="none")
    r = O.group_norm(x.double().cpu().numpy(), None, None, w.Hv, "none", 1e-5)
    got = f.out.double().cpu().numpy()
    assert (np.abs(got - r["out"]) <= O.bound(r["out"], r["out_err"], "fp16")).all()


def test_memory_of_a_call_on_another_stream_is_that_streams_own(dev):
    """A function given a stream allocates on it: memory that the current stream may still be using is not written."""
    B, T, D = 2, 256, 512
    g = torch.Generator().manual_seed(4)
    x, a, b, dy = (torch.randn((B, T, D), generator=g).to(torch.bfloat16).to(dev) for _ in range(4))
    A_log, bias, state = torch.zeros(D, device=dev), torch.full((D,), -2.0, device=dev), torch.zeros((B, D), device=dev)
    table = gdn.rotary_table(64, device=dev)
    mean, rstd = (lambda f: (f.mean, f.rstd))(gdn.group_norm_forward(x, groups=8))
    one = [t[:, :1] for t in (x, a, b)]
    calls = {
        "forward": lambda s: gdn.recurrence_forward(x, a, b, A_log, bias, stream=s).out,
        "backward": lambda s: gdn.recurrence_backward(x, a, b, A_log, bias, dy, stream=s).dx,
        "step": lambda s: gdn.recurrence_step(*one, A_log, bias, state.clone() if s is None else steps, stream=s),
        "rotary": lambda s: gdn.rotary(x, None, table, d=64, stream=s)[0],
        "norm": lambda s: gdn.group_norm_forward(x, groups=8, stream=s).out,
        "norm backward": lambda s: gdn.group_norm_backward(x, None, None, mean, rstd, dy, groups=8, stream=s).dx,
    }
    side = torch.cuda.Stream()
    for as_handle in (False, True):
        for name, call in calls.items():
            steps = state.clone()
            want = call(None).clone()
            torch.cuda.synchronize()
            used = torch.empty_like(want)
            at = used.data_ptr()
            del used   # the current stream's next tensor of this size would be here
            got = call(side.cuda_stream if as_handle else side)
            assert got.data_ptr() != at, name
            torch.cuda.synchronize()
            assert torch.equal(got, want), name


def test_workspaces_of_the_wrong_kind_are_refused(dev):
    x = torch.zeros((1, 4, 64), device=dev)
    table = gdn.rotary_table(64, device=dev)
    for ws in (torch.zeros(256, dtype=torch.uint8), torch.zeros(256, device=dev),
               torch.zeros((16, 16), dtype=torch.uint8, device=dev)):
        with pytest.raises(ValueError):
            gdn.rotary(x, None, table, d=64, workspace=ws)
    f = gdn.group_norm_forward(x, groups=2)
    f.workspace = torch.zeros(4096, dtype=torch.uint8)
    with pytest.raises(ValueError):
        gdn.group_norm_forward(x, groups=2, bufs=f)


def test_captured_chain_with_a_live_eager_result(dev):
    """The layer forward and backward captured into one graph while eager results of the same inputs live; replays
    on new inputs equal eager calls on them, and leave the earlier results alone."""
    B, T, D, d = 2, 96, 256, 64
    g = torch.Generator().manual_seed(9)
    x, a, b, dy = (torch.randn((B, T, D), generator=g).to(torch.bfloat16).to(dev) for _ in range(4))
    A_log, bias, table = torch.zeros(D, device=dev), torch.full((D,), -2.0, device=dev), gdn.rotary_table(d, device=dev)

    def layer():
        q, _ = gdn.rotary(x, None, table, d=d)
        f = gdn.recurrence_forward(q, a, b, A_log, bias, want_chunk_states=True)
        n = gdn.group_norm_forward(f.out, groups=4)
        gn = gdn.group_norm_backward(f.out, None, None, n.mean, n.rstd, dy, groups=4)
        gr = gdn.recurrence_backward(q, a, b, A_log, bias, gn.dx, None, f.chunk_states)
        dx, _ = gdn.rotary(gr.dx, None, table, d=d, inverse=True)
        return n.out, dx, gr.da, gr.dA_log

    eager = layer()
    kept = [t.clone() for t in eager]
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer()
    torch.cuda.current_stream().wait_stream(side)
    with torch.cuda.graph(graph):
        out = layer()
    for seed in (1, 2):
        x.copy_(torch.randn((B, T, D), generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16))
        graph.replay()
        for got, want in zip(out, layer()):
            assert torch.equal(got, want)
    for t, k in zip(eager, kept):
        assert torch.equal(t, k)
