"""Calls from two host threads at once, on streams and buffers of their own, whose kernels are the same and whose shared
memory differs: each call's limit of it holds for the whole process."""
import threading

import pytest
import torch

from linear_attention_sequence_qkv_gb300 import build, gdn
from linear_attention_sequence_qkv_gb300.workloads import WORKLOADS, make_cotangents, make_inputs, replace, to_device

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    build.build()
    gdn.load()
    return torch.device("cuda:0")


def both(calls, reps):
    """Every call of two functions of a stream, `reps` times each in a thread of its own: the errors they raised."""
    torch.cuda.synchronize()
    errors, start = [], threading.Barrier(2)

    def work(call, stream):
        stream.synchronize()
        start.wait()
        for i in range(reps):
            try:
                call(stream)
            except Exception as e:
                errors.append(str(e))
            if i % 64 == 63:
                stream.synchronize()

    threads = [threading.Thread(target=work, args=(c, torch.cuda.Stream())) for c in calls]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    return errors


CASES = [("fp32", (64, 64), (256, 64)), ("fp32", (512, 32), (32, 32)), ("bf16", (64, 128), (64, 512)),
         ("bf16", (256, 128), (64, 64)), ("fp16", (128, 64), (64, 64)), ("bf16", (32, 64), (512, 512))]


@pytest.mark.parametrize("dtype,first,second", CASES)
@pytest.mark.parametrize("backward", [False, True])
def test_two_head_shapes(dev, dtype, first, second, backward):
    calls, checks = [], []
    for dk, dv in (first, second):
        w = replace(WORKLOADS["tiny_fp32"], dtype=dtype, T=70, Hk=1, Hv=1, dk=dk, dv=dv)
        inp = make_inputs(w)
        dout = make_cotangents(inp, final=False)[0].to(dev)
        inp = to_device(inp, dev)
        bufs, grads = gdn.forward(inp), gdn.backward(inp, dout)
        torch.cuda.synchronize()
        checks.append((bufs.out, bufs.out.clone(), grads.dk_raw, grads.dk_raw.clone()))
        if backward:
            calls.append(lambda s, inp=inp, dout=dout, grads=grads: gdn.backward(inp, dout, grads=grads, stream=s))
        else:
            calls.append(lambda s, inp=inp, bufs=bufs: gdn.forward(inp, bufs, stream=s))
    assert both(calls, 1000) == []
    for out, want, dk_raw, want_dk in checks:
        assert torch.equal(out, want) and torch.equal(dk_raw, want_dk)


def test_two_widths_of_states_across_spans(dev):
    calls, checks = [], []
    for dk in (512, 256):
        A, B = torch.randn(3, 1, dk, dk, device=dev) * dk ** -0.5, torch.randn(3, 1, dk, 32, device=dev)
        H = torch.empty_like(B)
        call = lambda s, A=A, B=B, H=H, dk=dk: gdn.gdn_span_scan(3, 1, dk, 32, A, B, None, H, stream=s)  # noqa: E731
        call(None)
        torch.cuda.synchronize()
        checks.append((H, H.clone()))
        calls.append(call)
    assert both(calls, 3000) == []
    for H, want in checks:
        assert torch.equal(H, want)


@pytest.mark.parametrize("dtype,dk,dv", [("bf16", 64, 64), ("bf16", 128, 128), ("fp32", 64, 64)])
def test_stages_as_a_threads_first_calls(dev, dtype, dk, dv):
    """The chunk stage encodes its tensor maps before it launches anything: the thread has no context yet."""
    w = replace(WORKLOADS["tiny_fp32"], dtype=dtype, T=130, Hk=1, Hv=2, dk=dk, dv=dv)
    inp = to_device(make_inputs(w), dev)
    want = gdn.forward(inp)
    d, bufs, stream, got = want.desc, gdn.alloc(want.desc, dev), torch.cuda.Stream().cuda_stream, []
    gdn.gdn_prologue(d, inp.q_raw, inp.k_raw, inp.v_raw, inp.a, inp.b, inp.conv_w, inp.A_log, inp.dt_bias, None,
                     bufs.workspace, bufs.ws_bytes)
    torch.cuda.synchronize()

    def rest():
        got.append(gdn.gdn_chunk_rule(d, None, inp.initial_state, bufs.final_state, bufs.workspace, bufs.ws_bytes, stream,
                                      check=False))
        got.append(gdn.gdn_epilogue(d, inp.gate, inp.norm_w, bufs.out, bufs.workspace, bufs.ws_bytes, stream, check=False))

    t = threading.Thread(target=rest)
    t.start()
    t.join()
    torch.cuda.synchronize()
    assert got == [gdn.GDN_OK] * 2
    assert torch.equal(bufs.out, want.out) and torch.equal(bufs.final_state, want.final_state)
