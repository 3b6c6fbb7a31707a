"""Host-side checks of the operators beside the gated delta rule (no GPU): descriptors, refusals
before any launch, the rotary table, and the Python functions' own checks."""
import ctypes
import math
from fractions import Fraction

import pytest
import torch

from linear_attention_sequence_qkv_gb300 import build, gdn
from oracle import layer_ops as O

FAKE = 1 << 20   # never dereferenced: every call below fails its checks first
INVALID, UNSUPPORTED, WORKSPACE = gdn.GDN_ERR_INVALID_ARG, gdn.GDN_ERR_UNSUPPORTED, gdn.GDN_ERR_WORKSPACE


@pytest.fixture(scope="module")
def lib():
    build.build()
    return gdn.load()


def test_struct_sizes(lib):
    assert ctypes.sizeof(gdn.gdn_recurrence_desc) == 6 * 4 + 6 * 8
    assert ctypes.sizeof(gdn.gdn_rotary_desc) == 12 * 4 + 8 * 8
    assert ctypes.sizeof(gdn.gdn_group_norm_desc) == 8 * 4 + 2 * 8


def each_refused(call, args, optional, status=INVALID):
    for i in range(len(args)):
        if i not in optional:
            a = list(args)
            a[i] = None
            assert call(a) == status, f"argument {i} null"
    for i in range(len(args)):
        a = list(args)
        a[i] = FAKE + 1
        assert call(a) == status, f"argument {i} misaligned"


@pytest.mark.parametrize("args,status", [((0, 4, 0, 8, 0), INVALID), ((2, -1, 0, 8, 0), INVALID), ((2, 4, 0, 0, 0), INVALID),
                                         ((2, 4, 3, 8, 0), INVALID), ((2, 4, 0, 8, 3), UNSUPPORTED),
                                         ((2147483647, 2147483647, 0, 8, 0), UNSUPPORTED)])
def test_recurrence_desc(lib, args, status):
    d = gdn.gdn_recurrence_desc()
    assert lib.gdn_recurrence_desc_init(ctypes.byref(d), *args) == status
    assert lib.gdn_recurrence_desc_init(None, 1, 1, 0, 1, 0) == INVALID


def test_recurrence_refusals(lib):
    d = gdn.gdn_recurrence_desc_init(2, 100, 0, 48, gdn.GDN_BF16)
    need, bneed = gdn.gdn_recurrence_workspace_bytes(d), gdn.gdn_recurrence_backward_workspace_bytes(d)
    assert bneed >= need + 2 * 2 * 48 * 4

    def fwd(a, ws=FAKE, n=need):
        return lib.gdn_recurrence_forward(ctypes.byref(d), *a, ws, n, None)

    # x a b A_log dt_bias cu initial out final chunk_states
    args = [FAKE] * 10
    args[5] = None
    each_refused(fwd, args, {5, 6, 8, 9})
    a = list(args)
    a[5] = FAKE                        # cu_seqlens with B = 2
    assert fwd(a) == INVALID
    assert fwd(args, None) == WORKSPACE and fwd(args, FAKE + 128) == WORKSPACE and fwd(args, FAKE, need - 1) == WORKSPACE

    def bwd(a, ws=FAKE, n=bneed):
        return lib.gdn_recurrence_backward(ctypes.byref(d), *a, ws, n, None)

    # x a b A_log dt_bias cu initial chunk_states grad_out grad_final dx da db dA ddt dinitial
    args = [FAKE] * 16
    args[5] = None
    each_refused(bwd, args, {5, 6, 7, 9, 15})
    assert bwd(args, None) == WORKSPACE and bwd(args, FAKE, bneed - 1) == WORKSPACE

    s = gdn.gdn_recurrence_desc_init(2, 1, 0, 48, gdn.GDN_BF16)
    each_refused(lambda a: lib.gdn_recurrence_step(ctypes.byref(s), *a, None), [FAKE] * 7, set())
    assert lib.gdn_recurrence_step(ctypes.byref(d), *[FAKE] * 7, None) == INVALID     # T != 1
    for field, v in (("x_stride_t", 47), ("a_stride_t", 0), ("b_stride_b", -1)):
        bad = gdn.gdn_recurrence_desc_init(2, 100, 0, 48, gdn.GDN_BF16)
        setattr(bad, field, v)
        args = [FAKE] * 10
        args[5] = None
        assert lib.gdn_recurrence_forward(ctypes.byref(bad), *args, FAKE, need, None) == INVALID, field
        n = ctypes.c_size_t(0)
        assert lib.gdn_recurrence_workspace_bytes(ctypes.byref(bad), ctypes.byref(n)) == INVALID


def test_rotary_refusals(lib):
    def desc(**kw):
        d = gdn.gdn_rotary_desc_init(2, 10, 0, 4, 2, 64, gdn.GDN_F16)
        for k, v in kw.items():
            setattr(d, k, v)
        return d

    # q k turns positions cu offsets q_out k_out; fresh outputs, not in place
    args = [FAKE, FAKE, FAKE, None, None, None, 2 * FAKE, 2 * FAKE]

    def call(a, d=None, ws=FAKE, n=256):
        return lib.gdn_rotary(ctypes.byref(d or desc()), *a, ws, n, None)

    each_refused(call, args, {3, 4, 5})
    a = list(args)
    a[3] = a[5] = FAKE                 # positions and offsets
    assert call(a) == INVALID
    a = list(args)
    a[6] = FAKE                        # in place, with other strides
    assert call(a, desc(q_out_stride_t=512, q_out_stride_b=5120)) == INVALID
    for bad in (dict(rot=0), dict(rot=7), dict(rot=66), dict(layout=2), dict(inverse=2), dict(q_stride_t=255),
                dict(k_out_stride_t=127), dict(q_out_stride_b=0), dict(k_stride_b=-1), dict(Hk=-1), dict(d=1)):
        assert call(args, desc(**bad)) == INVALID, bad
    assert call(args, desc(dtype=5)) == UNSUPPORTED
    assert call(args, ws=None) == WORKSPACE and call(args, n=255) == WORKSPACE and call(args, ws=FAKE + 64) == WORKSPACE


def test_group_norm_refusals(lib):
    def desc(**kw):
        d = gdn.gdn_group_norm_desc_init(3, 5, 24, 4, gdn.GDN_BF16)
        for k, v in kw.items():
            setattr(d, k, v)
        return d

    need = gdn.gdn_group_norm_workspace_bytes(desc())
    bneed = gdn.gdn_group_norm_backward_workspace_bytes(desc())

    def fwd(a, d=None, ws=FAKE, n=need):   # x weight bias out mean rstd
        return lib.gdn_group_norm_forward(ctypes.byref(d or desc()), *a, ws, n, None)

    def bwd(a, d=None, ws=FAKE, n=bneed):   # x weight bias mean rstd grad_out dx dweight dbias
        return lib.gdn_group_norm_backward(ctypes.byref(d or desc()), *a, ws, n, None)

    each_refused(fwd, [FAKE] * 6, {1, 2, 4, 5})
    each_refused(bwd, [FAKE] * 9, {1, 2, 7, 8})
    for bad, status in ((dict(C=25), INVALID), (dict(G=0), INVALID), (dict(N=-1), INVALID), (dict(L=-1), INVALID),
                        (dict(eps=-1.0), INVALID), (dict(eps=math.nan), INVALID), (dict(x_stride_l=23), INVALID),
                        (dict(x_stride_n=-1), INVALID), (dict(act=2), UNSUPPORTED), (dict(dtype=9), UNSUPPORTED),
                        (dict(weight_dtype=gdn.GDN_F16), UNSUPPORTED)):
        assert fwd([FAKE] * 6, desc(**bad)) == status, bad
        assert bwd([FAKE] * 9, desc(**bad)) == status, bad
    assert fwd([FAKE] * 6, ws=None) == WORKSPACE and fwd([FAKE] * 6, n=need - 1) == WORKSPACE
    assert bwd([FAKE] * 9, ws=FAKE + 1) == WORKSPACE and bwd([FAKE] * 9, n=bneed - 1) == WORKSPACE
    # no positions: nothing to launch
    assert fwd([None] * 6, desc(N=0)) == gdn.GDN_OK and fwd([None] * 6, desc(L=0)) == gdn.GDN_OK


@pytest.mark.parametrize("rot,theta,kw", [(128, 10000.0, {}), (64, 500000.0, dict(scaling="linear", factor=4.0)),
                                          (20, 10000.0, dict(scaling="by_parts", factor=16.0, low=1.0, high=4.0,
                                                             original=8192)), (2, 0.5, {})])
def test_rotary_table(lib, rot, theta, kw):
    """Entries are f / (2 pi) turns in units of 2^-64, whole turns dropped. Allowed: a few fp64 roundings
    (the power's, up to 4 of its own units, and four products) of the value before whole turns drop out."""
    t = gdn.rotary_table(rot, theta, device="cpu", **kw)
    f = O.frequencies(rot, theta, **kw)
    assert t.shape == (rot // 2,)
    two_pi = Fraction(2) * Fraction("3.14159265358979323846264338327950288")
    for got, want in zip(t.tolist(), f.tolist()):
        turns = Fraction(want) / two_pi
        frac = turns - math.floor(turns)
        off = abs(Fraction(got % 2 ** 64, 2 ** 64) - frac)
        assert min(off, 1 - off) <= 16 * Fraction(1, 2 ** 53) * (turns + Fraction(1, 2 ** 10))


def test_rotary_table_refusals(lib):
    out = torch.zeros(64, dtype=torch.int64)
    call = lambda *a: lib.gdn_rotary_table(*a, out.data_ptr())  # noqa: E731
    ok = (128, 10000.0, 2, 16.0, 1.0, 4.0, 8192.0)
    assert call(*ok) == gdn.GDN_OK
    for i, v in ((0, 127), (0, 0), (0, -2), (1, 0.0), (1, -1.0), (1, math.nan), (1, math.inf), (2, 3), (2, -1), (3, 0.0),
                 (3, math.nan), (5, 1.0), (5, math.nan), (6, 0.0), (6, math.inf)):
        a = list(ok)
        a[i] = v
        assert call(*a) == INVALID, (i, v)
    assert lib.gdn_rotary_table(*ok, None) == INVALID
    with pytest.raises(ValueError):
        gdn.rotary_table(128, scaling="other", device="cpu")


def test_python_functions_refuse_what_the_kernels_would_trust(lib):
    x = torch.zeros(2, 4, 8)
    v = torch.zeros(8)
    with pytest.raises(ValueError):
        gdn.recurrence_desc_for(x, x[..., :7], x)
    with pytest.raises(ValueError):
        gdn.recurrence_desc_for(x, x.to(torch.bfloat16), x)
    with pytest.raises(ValueError):
        gdn.recurrence_desc_for(x.transpose(1, 2), x.transpose(1, 2), x.transpose(1, 2))
    for call in (lambda: gdn.recurrence_forward(x, x, x, v, v), lambda: gdn.recurrence_backward(x, x, x, v, v, x),
                 lambda: gdn.recurrence_step(x[:, :1], x[:, :1], x[:, :1], v, v, x[:, 0].contiguous()),
                 lambda: gdn.rotary(x, None, torch.zeros(4, dtype=torch.int64), d=8),
                 lambda: gdn.group_norm_forward(x, v, v, groups=2)):
        with pytest.raises((ValueError, RuntimeError, AssertionError)):   # CPU tensors: no fallback
            call()
    with pytest.raises(ValueError):
        gdn.rotary_desc_for(x, None, x, None, d=3)
    with pytest.raises(ValueError):
        gdn.rotary_desc_for(x, None, x, None, d=8, layout="other")
    with pytest.raises(ValueError):
        gdn.group_norm_desc_for(x, groups=2, act="other")
    with pytest.raises(gdn.GdnError):
        gdn.group_norm_desc_for(x, groups=3)


def test_strides_of_single_elements(lib):
    # torch reports any stride for a dimension of one element; the descriptor takes its own
    x = torch.zeros(4, 1, 8).transpose(0, 1).contiguous().transpose(0, 1)
    d = gdn.recurrence_desc_for(x, x, x)
    assert d.x_stride_t == 8 and d.x_stride_b == 8
    wide = torch.zeros(1, 5, 20)[:, :, 4:12]
    d = gdn.recurrence_desc_for(wide, wide, wide)
    assert d.x_stride_t == 20


@pytest.mark.parametrize("args", [(1, 2 ** 31 - 1, 0, 8, 1), (1, 2 ** 31 - 2 ** 16 + 1, 0, 8, 1), (1, 1, 0, 2 ** 30 + 1, 1),
                                  (1, 1, 0, 2 ** 31 - 1, 1)])
def test_sizes_whose_indices_would_wrap_are_refused(lib, args):
    assert lib.gdn_recurrence_desc_init(ctypes.byref(gdn.gdn_recurrence_desc()), *args) == UNSUPPORTED
    edge = (1, min(args[1], 2 ** 31 - 2 ** 16), 0, min(args[3], 2 ** 30), 1)
    assert lib.gdn_recurrence_desc_init(ctypes.byref(gdn.gdn_recurrence_desc()), *edge) == gdn.GDN_OK


@pytest.mark.parametrize("N,L,C,G", [(1, 2 ** 31 - 1, 8, 1), (1, 1, 2 ** 24 + 1, 1)])
def test_group_norm_sizes_whose_indices_would_wrap_are_refused(lib, N, L, C, G):
    assert lib.gdn_group_norm_desc_init(ctypes.byref(gdn.gdn_group_norm_desc()), N, L, C, G, gdn.GDN_F32) == UNSUPPORTED
    edge = (N, min(L, 2 ** 31 - 2 ** 16), min(C, 2 ** 24), G)
    d = gdn.gdn_group_norm_desc_init(*edge, gdn.GDN_F32)
    assert gdn.gdn_group_norm_workspace_bytes(d) >= 256 and gdn.gdn_group_norm_backward_workspace_bytes(d) >= 256


@pytest.mark.parametrize("args", [(128, 5e-324, 0, 1.0, 1.0, 2.0, 1.0), (128, 10000.0, 1, 5e-324, 1.0, 2.0, 1.0),
                                  (64, 1e-300, 2, 1e-20, 1e305, 1e306, 1.0)])
def test_rotary_table_of_infinite_frequencies_is_refused(lib, args):
    out = torch.zeros(64, dtype=torch.int64)
    assert lib.gdn_rotary_table(*args, out.data_ptr()) == INVALID


@pytest.mark.parametrize("dtype", [gdn.GDN_F32, gdn.GDN_BF16])
def test_backward_workspace_of_many_rows_is_small(lib, dtype):
    """Partial sums of one CTA per row and channel slab where rows fill the chip, beside the states of every 4th token."""
    B, T, D = 20000, 8, 512
    need = gdn.gdn_recurrence_backward_workspace_bytes(gdn.gdn_recurrence_desc_init(B, T, 0, D, dtype))
    assert need <= 1024 + B * 2 * D * 4 + B * (T // 4) * D * 4
