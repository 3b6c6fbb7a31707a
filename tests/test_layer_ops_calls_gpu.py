"""Calls of the operators beside the gated delta rule that are not one after the other from one host thread: several threads
at once, a thread's first call, and calls whose waits run out."""
import threading
import time

import pytest
import torch

from linear_attention_sequence_qkv_gb300 import build, gdn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    build.build()
    gdn.load()
    return torch.device("cuda:0")


def at_once(calls, reps):
    """Each of `calls` (a function that launches on the stream it is given and returns a status) in a host thread
    and on a stream of its own, `reps` times; the statuses that were not GDN_OK."""
    torch.cuda.synchronize()
    bad, start = [], threading.Barrier(len(calls))

    def work(call, stream):
        stream.synchronize()
        start.wait()
        for i in range(reps):
            rc = call(stream)
            if rc != gdn.GDN_OK:
                bad.append(rc)
            if i % 64 == 63:
                stream.synchronize()

    threads = [threading.Thread(target=work, args=(c, torch.cuda.Stream())) for c in calls]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    return bad


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_recurrences_of_different_clusters_from_two_threads(dev, dtype):
    """One chain of a row of many tiles (the largest cluster, and the most shared memory) beside rows of one tile (clusters of
    one CTA): neither call changes what the other may launch with."""
    calls, checks = [], []
    for B, T in ((1, 600), (40, 1)):
        D = 128 // dtype.itemsize
        x, a, b, dout = (torch.randn(B, T, D, device=dev).to(dtype) for _ in range(4))
        A_log, bias = torch.zeros(D, device=dev), torch.zeros(D, device=dev)
        d = gdn.recurrence_desc_for(x, a, b)
        f, g = gdn.alloc_recurrence(d, dev, want_chunk_states=True), gdn.alloc_recurrence_grads(d, dev)

        def call(stream, d=d, x=x, a=a, b=b, A_log=A_log, bias=bias, f=f, g=g, dout=dout):
            rc = gdn.gdn_recurrence_forward(d, x, a, b, A_log, bias, None, None, f.out, f.final_state, f.chunk_states,
                                            f.workspace, f.ws_bytes, stream, check=False)
            return rc or gdn.gdn_recurrence_backward(d, x, a, b, A_log, bias, None, None, f.chunk_states, dout, None, g.dx,
                                                     g.da, g.db, g.dA_log, g.ddt_bias, g.dinitial_state, g.workspace,
                                                     g.ws_bytes, stream, check=False)

        assert call(torch.cuda.current_stream()) == gdn.GDN_OK
        torch.cuda.synchronize()
        checks.append((f, g, f.out.clone(), g.da.clone(), g.dA_log.clone()))
        calls.append(call)
    assert at_once(calls, 4000) == []
    for f, g, out, da, dA_log in checks:
        assert gdn.gdn_device_status(f.workspace) == gdn.GDN_OK and gdn.gdn_device_status(g.workspace) == gdn.GDN_OK
        assert torch.equal(f.out, out) and torch.equal(g.da, da) and torch.equal(g.dA_log, dA_log)


def test_rotations_of_different_widths_from_two_threads(dev):
    """Heads wide enough that their tables need more shared memory than every kernel may have, of two widths."""
    calls, checks = [], []
    for d in (32768, 16384):
        q = torch.randn(1, 2, d, device=dev).to(torch.bfloat16)
        table, out = gdn.rotary_table(d, device=dev), torch.empty_like(q)
        r = gdn.rotary_desc_for(q, None, out, None, d=d)
        ws = torch.empty(gdn.gdn_rotary_workspace_bytes(r), dtype=torch.uint8, device=dev)

        def call(stream, r=r, q=q, table=table, out=out, ws=ws):
            return gdn.gdn_rotary(r, q, None, table, None, None, None, out, None, ws, ws.numel(), stream, check=False)

        assert call(torch.cuda.current_stream()) == gdn.GDN_OK
        torch.cuda.synchronize()
        checks.append((out, out.clone()))
        calls.append(call)
    assert at_once(calls, 8000) == []
    for out, want in checks:
        assert torch.equal(out, want)


@pytest.mark.parametrize("backward", [False, True])
def test_first_call_of_a_host_thread(dev, backward):
    """A thread whose first use of CUDA is the call itself: no context is bound to it yet."""
    x, a, b, dout = (torch.randn(2, 50, 64, device=dev).to(torch.bfloat16) for _ in range(4))
    A_log, bias = torch.zeros(64, device=dev), torch.zeros(64, device=dev)
    d = gdn.recurrence_desc_for(x, a, b)
    f, g = gdn.alloc_recurrence(d, dev, want_chunk_states=True), gdn.alloc_recurrence_grads(d, dev)

    def call(stream):
        if backward:
            return gdn.gdn_recurrence_backward(d, x, a, b, A_log, bias, None, None, f.chunk_states, dout, None, g.dx, g.da,
                                               g.db, g.dA_log, g.ddt_bias, g.dinitial_state, g.workspace, g.ws_bytes, stream,
                                               check=False)
        return gdn.gdn_recurrence_forward(d, x, a, b, A_log, bias, None, None, f.out, f.final_state, f.chunk_states,
                                          f.workspace, f.ws_bytes, stream, check=False)

    want = gdn.recurrence_forward(x, a, b, A_log, bias, want_chunk_states=True)
    want_g = gdn.recurrence_backward(x, a, b, A_log, bias, dout, None, want.chunk_states)
    f.out.zero_(), g.dx.zero_(), f.chunk_states.copy_(want.chunk_states)
    stream, got = torch.cuda.Stream().cuda_stream, []
    torch.cuda.synchronize()
    t = threading.Thread(target=lambda: got.append(call(stream)))
    t.start()
    t.join()
    torch.cuda.synchronize()
    assert got == [gdn.GDN_OK]
    assert torch.equal(g.dx, want_g.dx) if backward else torch.equal(f.out, want.out)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("B,T,D,waits", [(1, 1000, 63, True), (1, 1000, 64, True), (3, 530, 99, True), (1, 130, 24, True),
                                         (2, 31, 5, False)])
def test_maps_that_do_not_arrive_are_reported(dev, B, T, D, waits, packed, dtype):
    """gdn_set_wait_test_mode where CTAs of a cluster wait for one another, also without copies into shared memory to wait
    for (D odd): the CTAs give up, report it, and wait for what is on its way to them but not for what nobody
    issued (a second each), and the next calls are right. One CTA per row without copies (31 tokens of 5 channels) waits
    for nothing."""
    B = 1 if packed else B
    x, a, b, dout = (torch.randn(B, T, D, device=dev).to(dtype) for _ in range(4))
    A_log, bias = torch.zeros(D, device=dev), torch.full((D,), -2.0, device=dev)
    cu = torch.tensor([0, T // 3, T // 3, T // 2 + 1, T], dtype=torch.int32, device=dev) if packed else None
    fwd = lambda: gdn.recurrence_forward(x, a, b, A_log, bias, cu, want_chunk_states=True)  # noqa: E731
    bwd = lambda cs: gdn.recurrence_backward(x, a, b, A_log, bias, dout, None, cs, cu)  # noqa: E731
    want = fwd()
    want_g = bwd(want.chunk_states)
    assert gdn.gdn_device_status(want_g.workspace) == gdn.GDN_OK
    torch.cuda.synchronize()
    gdn.gdn_set_wait_test_mode(1)
    try:
        start = time.perf_counter()
        for _ in range(10):
            got = [gdn.gdn_device_status(f.workspace) for f in (fwd(), bwd(want.chunk_states), bwd(None))]
            assert got == [gdn.GDN_ERR_DEVICE_TIMEOUT if waits else gdn.GDN_OK] * 3
        took = time.perf_counter() - start
    finally:
        gdn.gdn_set_wait_test_mode(0)
    assert took < 0.5
    for _ in range(2):
        again = fwd()
        again_g = bwd(again.chunk_states)
        assert gdn.gdn_device_status(again.workspace) == gdn.GDN_OK and gdn.gdn_device_status(again_g.workspace) == gdn.GDN_OK
        assert torch.equal(again.out, want.out) and torch.equal(again.final_state, want.final_state)
        for name in ("dx", "da", "db", "dA_log", "ddt_bias", "dinitial_state"):
            assert torch.equal(getattr(again_g, name), getattr(want_g, name)), name
