"""Host-side checks of the operators of attention layers (no GPU): descriptors, refusals before any launch, and the
Python functions' own checks."""
import ctypes
import math

import pytest
import torch

from linear_attention_sequence_qkv_gb300 import build, gdn
from test_layer_ops_host import FAKE, INVALID, UNSUPPORTED, WORKSPACE, each_refused


@pytest.fixture(scope="module")
def lib():
    build.build()
    return gdn.load()


def test_struct_sizes(lib):
    assert ctypes.sizeof(gdn.gdn_norm_rotary_desc) == 12 * 4 + 8 * 8 + 2 * 4
    assert ctypes.sizeof(gdn.gdn_window_attention_desc) == 12 * 4 + 6 * 8


def test_norm_rotary_refusals(lib):
    def desc(rot=None, **kw):
        d = gdn.gdn_norm_rotary_desc_init(2, 10, 0, 4, 2, 64, gdn.GDN_F16)
        for k, v in kw.items():
            setattr(d, k, v)
        for k, v in (rot or {}).items():
            setattr(d.rotary, k, v)
        return d

    need = gdn.gdn_norm_rotary_backward_workspace_bytes(desc())
    # q k q_weight k_weight turns positions cu offsets q_out k_out
    args = [FAKE, FAKE, FAKE, FAKE, FAKE, None, None, None, 2 * FAKE, 2 * FAKE]

    def fwd(a, d=None, ws=FAKE, n=256):
        return lib.gdn_norm_rotary_forward(ctypes.byref(d or desc()), *a, ws, n, None)

    each_refused(fwd, args, {2, 3, 5, 6, 7})
    # ... grad_q grad_k dq dk dq_weight dk_weight
    bargs = args + [3 * FAKE] * 4

    def bwd(a, d=None, ws=FAKE, n=need):
        return lib.gdn_norm_rotary_backward(ctypes.byref(d or desc()), *a, ws, n, None)

    each_refused(bwd, bargs, {2, 3, 5, 6, 7, 12, 13})
    for call, a, full in ((fwd, args, 256), (bwd, bargs, need)):
        b = list(a)
        b[5] = b[7] = FAKE                 # positions and offsets
        assert call(b) == INVALID
        for bad in (dict(rot=0), dict(rot=7), dict(rot=66), dict(layout=2), dict(inverse=1), dict(q_stride_t=255), dict(k_out_stride_t=127),
                    dict(k_stride_b=-1), dict(Hk=-1), dict(d=1), dict(scale=math.nan)):
            assert call(a, desc(bad)) == INVALID, bad
        for bad, status in ((dict(eps=-1.0), INVALID), (dict(eps=math.nan), INVALID), (dict(weight_dtype=gdn.GDN_BF16), UNSUPPORTED)):
            assert call(a, desc(**bad)) == status, bad
        assert call(a, desc(dict(dtype=5), weight_dtype=5)) == UNSUPPORTED
        assert call(a, desc(dict(d=1026, q_stride_t=9000, k_stride_t=9000, q_out_stride_t=9000, k_out_stride_t=9000,
                                 q_out_stride_b=90000, k_out_stride_b=90000))) == UNSUPPORTED
        assert call(a, ws=None) == WORKSPACE and call(a, n=full - 1) == WORKSPACE and call(a, ws=FAKE + 64) == WORKSPACE
    a = list(args)
    a[8] = FAKE                            # in place, with other strides
    assert fwd(a, desc(dict(q_out_stride_t=512, q_out_stride_b=5120))) == INVALID


@pytest.mark.parametrize("args,status", [((0, 4, 4, 0, 2, 1, 64, 4, 0, 0), INVALID), ((2, -1, 4, 0, 2, 1, 64, 4, 0, 0), INVALID),
                                         ((2, 4, 4, 3, 2, 1, 64, 4, 0, 0), INVALID), ((2, 4, 4, 0, 2, 1, 64, 0, 0, 0), INVALID),
                                         ((2, 4, 4, 0, 2, 1, 64, 4, -1, 0), INVALID), ((2, 4, 4, 0, 2, 1, 0, 4, 0, 0), INVALID),
                                         ((2, 4, 4, 0, 3, 2, 64, 4, 0, 0), UNSUPPORTED), ((2, 4, 4, 0, 2, 1, 257, 4, 0, 0), UNSUPPORTED),
                                         ((2, 4, 4, 0, 2, 1, 64, 4, 0, 3), UNSUPPORTED), ((2, 2147483647, 4, 0, 2, 1, 64, 4, 0, 0), UNSUPPORTED),
                                         ((65536, 65536, 4, 0, 2, 1, 64, 4, 0, 0), UNSUPPORTED), ((2, 4, 4, 0, 2, 1, 64, 2147483647, 5, 0), 0)])
def test_window_attention_desc(lib, args, status):
    d = gdn.gdn_window_attention_desc()
    assert lib.gdn_window_attention_desc_init(ctypes.byref(d), *args) == status
    assert lib.gdn_window_attention_desc_init(None, 1, 1, 1, 0, 1, 1, 64, 1, 0, 0) == INVALID


def test_window_attention_refusals(lib):
    def desc(packed=0, tk=20, **kw):
        d = gdn.gdn_window_attention_desc_init(1 if packed else 2, 20, tk, packed, 4, 2, 64, 5, 2, gdn.GDN_BF16)
        for k, v in kw.items():
            setattr(d, k, v)
        return d

    need, bneed = gdn.gdn_window_attention_workspace_bytes(desc()), gdn.gdn_window_attention_backward_workspace_bytes(desc())

    def fwd(a, d=None, ws=FAKE, n=need):   # q k v cu cu_k out lse
        return lib.gdn_window_attention_forward(ctypes.byref(d or desc()), *a, ws, n, None)

    def bwd(a, d=None, ws=FAKE, n=bneed):   # q k v out lse grad_out cu cu_k dq dk dv
        return lib.gdn_window_attention_backward(ctypes.byref(d or desc()), *a, ws, n, None)

    fargs, bargs = [FAKE] * 3 + [None, None] + [FAKE] * 2, [FAKE] * 6 + [None, None] + [FAKE] * 3
    each_refused(fwd, fargs, {3, 4, 6})
    each_refused(bwd, bargs, {6, 7})
    for call, a, at, full in ((fwd, fargs, 3, need), (bwd, bargs, 6, bneed)):
        for cu, cuk, d in ((FAKE, None, desc()), (None, FAKE, desc()), (FAKE, None, desc(packed=3, tk=30))):
            b = list(a)
            b[at], b[at + 1] = cu, cuk
            assert call(b, d, n=1 << 30) == INVALID
        for bad, status in ((dict(window=0), INVALID), (dict(sinks=-1), INVALID), (dict(scale=0.0), INVALID), (dict(scale=math.inf), INVALID),
                            (dict(scale=-1.0), INVALID), (dict(q_stride_t=255), INVALID), (dict(v_stride_t=127), INVALID),
                            (dict(k_stride_b=-1), INVALID), (dict(Hk=3), UNSUPPORTED), (dict(dtype=7), UNSUPPORTED)):
            assert call(a, desc(**bad)) == status, bad
        assert call(a, ws=None) == WORKSPACE and call(a, n=full - 1) == WORKSPACE and call(a, ws=FAKE + 1) == WORKSPACE


def test_cache_refusals(lib):
    def desc(T=1, **kw):
        d = gdn.gdn_window_attention_desc_init(2, T, T, 0, 4, 2, 64, 5, 2, gdn.GDN_BF16)
        for k, v in kw.items():
            setattr(d, k, v)
        return d

    def step(a, d=None, ws=FAKE, n=1 << 30):   # q k v lengths k_cache v_cache out
        return lib.gdn_window_attention_step(ctypes.byref(d or desc()), *a, ws, n, None)

    def write(a, d=None, ws=FAKE, n=1 << 30):   # k v cu lengths k_cache v_cache
        return lib.gdn_window_cache_write(ctypes.byref(d or desc(3)), *a, ws, n, None)

    sargs, wargs = [FAKE] * 7, [FAKE, FAKE, None, FAKE, FAKE, FAKE]
    each_refused(step, sargs, set())
    each_refused(write, wargs, {2})
    for call, a, T in ((step, sargs, 1), (write, wargs, 3)):
        for bad, status in ((dict(slots=6), INVALID), (dict(window=0), INVALID), (dict(Hk=3), UNSUPPORTED), (dict(dtype=7), UNSUPPORTED)):
            assert call(a, desc(T, **bad)) == status, bad
        assert call(a, ws=None) == WORKSPACE and call(a, n=255) == WORKSPACE and call(a, ws=FAKE + 1) == WORKSPACE
    assert step(sargs, desc(2)) == INVALID                   # T != 1
    n = ctypes.c_size_t(0)
    for name in ("gdn_window_attention_step_workspace_bytes", "gdn_window_cache_write_workspace_bytes"):
        assert getattr(lib, name)(ctypes.byref(desc(slots=6)), ctypes.byref(n)) == INVALID
        assert getattr(lib, name)(ctypes.byref(desc()), None) == INVALID


def test_python_functions_refuse_what_the_kernels_would_trust(lib):
    q, k = torch.zeros(2, 4, 32), torch.zeros(2, 4, 16)
    kw = dict(d=8, window=3)
    for bad in (lambda: gdn.window_attention_desc_for(q, k, k[:, :3], **kw), lambda: gdn.window_attention_desc_for(q, k, k.bfloat16(), **kw),
                lambda: gdn.window_attention_desc_for(q[:1], k, k, **kw), lambda: gdn.window_attention_desc_for(q, k, k, d=5, window=3),
                lambda: gdn.window_attention_desc_for(q, k.transpose(1, 2), k.transpose(1, 2), **kw),
                lambda: gdn.window_attention_desc_for(q, k, k, d=0, window=3),
                lambda: gdn.norm_rotary_desc_for(q, k, q, None, d=8), lambda: gdn.norm_rotary_desc_for(q, k, q, k, d=3)):
        with pytest.raises(ValueError):
            bad()
    table, w = torch.zeros(4, dtype=torch.int64), torch.ones(8)
    cache = gdn.WindowCache(torch.zeros(2, 2, 4, 8), torch.zeros(2, 2, 4, 8), torch.zeros(2, dtype=torch.int32), 3, 1)
    for call in (lambda: gdn.norm_rotary(q, k, w, w, table, d=8), lambda: gdn.norm_rotary_backward(q, k, w, w, table, q, k, d=8),
                 lambda: gdn.window_attention_forward(q, k, k, **kw), lambda: gdn.window_attention_backward(q, k, k, q, torch.zeros(4, 8), q, **kw),
                 lambda: gdn.window_cache_write(k, k, cache), lambda: gdn.window_attention_step(q[:, :1], k[:, :1], k[:, :1], cache)):
        with pytest.raises((ValueError, RuntimeError, AssertionError)):   # CPU tensors: no fallback
            call()


def test_caches_whose_keys_32_bits_do_not_count(lib):
    """Groups of 16 keys are counted from the keys in 32 bits, which must have room for the last group's rounding up."""
    d = gdn.gdn_window_attention_desc_init(1, 1, 1, 0, 1, 1, 8, 5, 2, gdn.GDN_BF16)
    for slots, want in ((2 ** 31 - 2 ** 16, WORKSPACE), (2 ** 31 - 2 ** 16 + 1, UNSUPPORTED), (2 ** 31 - 1, UNSUPPORTED)):
        d.slots = slots
        assert lib.gdn_window_attention_step(ctypes.byref(d), *[FAKE] * 7, None, 0, None) == want
        assert lib.gdn_window_cache_write(ctypes.byref(d), FAKE, FAKE, None, FAKE, FAKE, FAKE, None, 0, None) == want
