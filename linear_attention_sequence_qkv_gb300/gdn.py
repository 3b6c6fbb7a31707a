"""Python binding of the C ABI in ``include/gdn.h`` (ctypes; marshalling only).

Every step of the core forward runs in ``libgdn.so``'s CUDA kernels: this
module turns torch tensors into device pointers, strides into a ``gdn_desc``,
and a torch stream into a ``cudaStream_t``. PyTorch allocates the device
memory (outputs and workspace). There is no other implementation: if the
library is missing or fails to load, every call raises.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
from dataclasses import dataclass
from typing import Optional

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libgdn.so")

GDN_OK = 0
GDN_ERR_INVALID_ARG = -1
GDN_ERR_UNSUPPORTED = -2
GDN_ERR_WORKSPACE = -3
GDN_ERR_CUDA = -4
GDN_ERR_DEVICE_SEQLENS = -5
GDN_ERR_DEVICE_RANGE = -6
GDN_ERR_DEVICE_TIMEOUT = -7

GDN_F32, GDN_BF16, GDN_F16 = 0, 1, 2
DTYPE_CODES = {torch.float32: GDN_F32, torch.bfloat16: GDN_BF16, torch.float16: GDN_F16}
ACT_TORCH = {GDN_F32: torch.float32, GDN_BF16: torch.bfloat16, GDN_F16: torch.float16}

# every entry point declared in include/gdn.h
EXPORTS = ("gdn_desc_init", "gdn_workspace_bytes", "gdn_workspace_offsets", "gdn_forward",
           "gdn_prologue", "gdn_chunk_rule", "gdn_epilogue", "gdn_device_status",
           "gdn_status_string", "gdn_chunk_kernel_kind", "gdn_forward_static_ws",
           "gdn_static_ws_device_status", "gdn_set_wait_test_mode",
           "gdn_decode_workspace_bytes", "gdn_decode_step", "gdn_backward_workspace_bytes",
           "gdn_backward", "gdn_forward_with_prefix", "gdn_span_scan",
           "gdn_recurrence_desc_init", "gdn_recurrence_workspace_bytes",
           "gdn_recurrence_backward_workspace_bytes", "gdn_recurrence_forward",
           "gdn_recurrence_backward", "gdn_recurrence_step", "gdn_rotary_desc_init",
           "gdn_rotary_table", "gdn_rotary_workspace_bytes", "gdn_rotary",
           "gdn_group_norm_desc_init", "gdn_group_norm_workspace_bytes",
           "gdn_group_norm_backward_workspace_bytes", "gdn_group_norm_forward",
           "gdn_group_norm_backward")

GDN_RECURRENCE_CHUNK = 4
ROTARY_LAYOUTS = {"half": 0, "interleaved": 1}
ROTARY_SCALINGS = {"plain": 0, "linear": 1, "by_parts": 2}
ACTIVATIONS = {"none": 0, "silu": 1}

# bytes of the library's fixed device scratch used by gdn_forward_static_ws
GDN_STATIC_WORKSPACE_BYTES = 16 * 1024 * 1024


class GdnError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status} ({status_string(status)})")


class gdn_desc(ctypes.Structure):
    _fields_ = [
        ("B", ctypes.c_int32), ("T", ctypes.c_int32), ("N", ctypes.c_int32),
        ("Hk", ctypes.c_int32), ("Hv", ctypes.c_int32), ("dk", ctypes.c_int32),
        ("dv", ctypes.c_int32), ("conv_width", ctypes.c_int32), ("dtype", ctypes.c_int32),
        ("gate_dtype", ctypes.c_int32), ("norm_w_dtype", ctypes.c_int32),
        ("reserved0", ctypes.c_int32),
        ("q_stride_b", ctypes.c_int64), ("q_stride_t", ctypes.c_int64),
        ("k_stride_b", ctypes.c_int64), ("k_stride_t", ctypes.c_int64),
        ("v_stride_b", ctypes.c_int64), ("v_stride_t", ctypes.c_int64),
        ("a_stride_b", ctypes.c_int64), ("a_stride_t", ctypes.c_int64),
        ("b_stride_b", ctypes.c_int64), ("b_stride_t", ctypes.c_int64),
        ("gate_stride_b", ctypes.c_int64), ("gate_stride_t", ctypes.c_int64),
        ("l2_eps", ctypes.c_float), ("norm_eps", ctypes.c_float), ("scale", ctypes.c_float),
        ("reserved1", ctypes.c_int32),
    ]


class gdn_workspace_layout(ctypes.Structure):
    _fields_ = [(n, ctypes.c_size_t) for n in
                ("status", "chunk_off", "q", "k", "v", "beta", "gamma", "o", "tpt", "total")]


class gdn_recurrence_desc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("B", "T", "N", "D", "dtype", "reserved0")] + [
        (n, ctypes.c_int64) for n in ("x_stride_b", "x_stride_t", "a_stride_b", "a_stride_t", "b_stride_b",
                                      "b_stride_t")]


class gdn_rotary_desc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("B", "T", "N", "Hq", "Hk", "d", "rot", "layout", "inverse", "dtype")] + [
        ("scale", ctypes.c_float), ("reserved0", ctypes.c_int32)] + [
        (n, ctypes.c_int64) for n in ("q_stride_b", "q_stride_t", "k_stride_b", "k_stride_t", "q_out_stride_b",
                                      "q_out_stride_t", "k_out_stride_b", "k_out_stride_t")]


class gdn_group_norm_desc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("N", "L", "C", "G", "dtype", "weight_dtype", "act")] + [
        ("eps", ctypes.c_float), ("x_stride_n", ctypes.c_int64), ("x_stride_l", ctypes.c_int64)]


_lib = None


def load(path: str = LIB_PATH):
    """Load ``libgdn.so`` (built in-tree by ``build.py``) and declare its ABI."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise ImportError(f"libgdn.so not built ({path}); run linear_attention_sequence_qkv_gb300/build.py")
    L = ctypes.CDLL(path)
    vp, sz, i32 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int
    dp = ctypes.POINTER(gdn_desc)
    L.gdn_desc_init.argtypes = [dp, i32, i32, i32, i32, i32, i32, i32, i32]
    L.gdn_workspace_bytes.argtypes = [dp, ctypes.POINTER(sz)]
    L.gdn_workspace_offsets.argtypes = [dp, ctypes.POINTER(gdn_workspace_layout)]
    L.gdn_forward.argtypes = [dp] + [vp] * 14 + [vp, sz, vp]
    L.gdn_prologue.argtypes = [dp] + [vp] * 9 + [vp, sz, vp]
    L.gdn_chunk_rule.argtypes = [dp, vp, vp, vp, vp, sz, vp]
    L.gdn_epilogue.argtypes = [dp, vp, vp, vp, vp, sz, vp]
    L.gdn_device_status.argtypes = [vp, ctypes.POINTER(i32), vp]
    L.gdn_status_string.argtypes = [i32]
    L.gdn_status_string.restype = ctypes.c_char_p
    L.gdn_chunk_kernel_kind.argtypes = [dp]
    L.gdn_forward_static_ws.argtypes = [dp] + [vp] * 14 + [vp]
    L.gdn_static_ws_device_status.argtypes = [ctypes.POINTER(i32), vp]
    L.gdn_set_wait_test_mode.argtypes = [i32]
    L.gdn_decode_workspace_bytes.argtypes = [dp, ctypes.POINTER(sz)]
    L.gdn_decode_step.argtypes = [dp] + [vp] * 13 + [vp, sz, vp]
    L.gdn_forward_with_prefix.argtypes = [dp] + [vp] * 15 + [vp, sz, vp]
    L.gdn_span_scan.argtypes = [i32, i32, i32, i32, vp, vp, vp, vp, vp]
    L.gdn_backward_workspace_bytes.argtypes = [dp, ctypes.POINTER(sz)]
    L.gdn_backward.argtypes = [dp] + [vp] * 25 + [vp, sz, vp]
    rp, tp, np_ = (ctypes.POINTER(c) for c in (gdn_recurrence_desc, gdn_rotary_desc, gdn_group_norm_desc))
    f64, szp = ctypes.c_double, ctypes.POINTER(sz)
    L.gdn_recurrence_desc_init.argtypes = [rp] + [i32] * 5
    L.gdn_recurrence_workspace_bytes.argtypes = [rp, szp]
    L.gdn_recurrence_backward_workspace_bytes.argtypes = [rp, szp]
    L.gdn_recurrence_forward.argtypes = [rp] + [vp] * 10 + [vp, sz, vp]
    L.gdn_recurrence_backward.argtypes = [rp] + [vp] * 16 + [vp, sz, vp]
    L.gdn_recurrence_step.argtypes = [rp] + [vp] * 7 + [vp]
    L.gdn_rotary_desc_init.argtypes = [tp] + [i32] * 7
    L.gdn_rotary_table.argtypes = [i32, f64, i32, f64, f64, f64, f64, vp]
    L.gdn_rotary_workspace_bytes.argtypes = [tp, szp]
    L.gdn_rotary.argtypes = [tp] + [vp] * 8 + [vp, sz, vp]
    L.gdn_group_norm_desc_init.argtypes = [np_] + [i32] * 5
    L.gdn_group_norm_workspace_bytes.argtypes = [np_, szp]
    L.gdn_group_norm_backward_workspace_bytes.argtypes = [np_, szp]
    L.gdn_group_norm_forward.argtypes = [np_] + [vp] * 6 + [vp, sz, vp]
    L.gdn_group_norm_backward.argtypes = [np_] + [vp] * 9 + [vp, sz, vp]
    for name in EXPORTS:
        if name != "gdn_status_string":
            getattr(L, name).restype = i32
    _lib = L
    return L


def status_string(status: int) -> str:
    return load().gdn_status_string(int(status)).decode()


def _ptr(x) -> Optional[int]:
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return x.data_ptr()


# torch.cuda.current_stream() builds a stream object, 3 us of a 4 us call; what torch's own generated code
# uses reads the handle alone
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_raw_device = getattr(torch._C, "_cuda_getDevice", None)


def _stream(s) -> Optional[int]:
    if s is None:
        if _raw_stream is None or _raw_device is None or not torch.cuda.is_initialized():
            return torch.cuda.current_stream().cuda_stream
        return _raw_stream(_raw_device())
    if isinstance(s, int):
        return s
    return s.cuda_stream


def _check(rc: int, where: str):
    if rc != GDN_OK:
        raise GdnError(rc, where)


# ------------------------------------------------------------ raw ABI calls
def gdn_desc_init(B, T, packed, Hk, Hv, dk, dv, dtype) -> gdn_desc:
    d = gdn_desc()
    _check(load().gdn_desc_init(ctypes.byref(d), B, T, packed, Hk, Hv, dk, dv, dtype),
           "gdn_desc_init")
    return d


def gdn_workspace_bytes(d: gdn_desc) -> int:
    n = ctypes.c_size_t(0)
    _check(load().gdn_workspace_bytes(ctypes.byref(d), ctypes.byref(n)), "gdn_workspace_bytes")
    return n.value


def gdn_workspace_offsets(d: gdn_desc) -> gdn_workspace_layout:
    lay = gdn_workspace_layout()
    _check(load().gdn_workspace_offsets(ctypes.byref(d), ctypes.byref(lay)), "gdn_workspace_offsets")
    return lay


def gdn_forward(d, q_raw, k_raw, v_raw, a, b, gate, conv_w, A_log, dt_bias, norm_w,
                cu_seqlens, initial_state, out, final_state, workspace, workspace_bytes,
                stream=None, check=True) -> int:
    rc = load().gdn_forward(ctypes.byref(d), _ptr(q_raw), _ptr(k_raw), _ptr(v_raw), _ptr(a),
                            _ptr(b), _ptr(gate), _ptr(conv_w), _ptr(A_log), _ptr(dt_bias),
                            _ptr(norm_w), _ptr(cu_seqlens), _ptr(initial_state), _ptr(out),
                            _ptr(final_state), _ptr(workspace), int(workspace_bytes),
                            _stream(stream))
    if check:
        _check(rc, "gdn_forward")
    return rc


def gdn_forward_static_ws(d, q_raw, k_raw, v_raw, a, b, gate, conv_w, A_log, dt_bias, norm_w,
                          cu_seqlens, initial_state, out, final_state, stream=None,
                          check=True) -> int:
    """gdn_forward on the library's fixed device scratch (no workspace argument):
    for callers that cannot allocate device memory."""
    rc = load().gdn_forward_static_ws(ctypes.byref(d), _ptr(q_raw), _ptr(k_raw), _ptr(v_raw),
                                      _ptr(a), _ptr(b), _ptr(gate), _ptr(conv_w), _ptr(A_log),
                                      _ptr(dt_bias), _ptr(norm_w), _ptr(cu_seqlens),
                                      _ptr(initial_state), _ptr(out), _ptr(final_state),
                                      _stream(stream))
    if check:
        _check(rc, "gdn_forward_static_ws")
    return rc


def gdn_static_ws_device_status(stream=None) -> int:
    """Device status word of the last gdn_forward_static_ws call on the current device."""
    st = ctypes.c_int(0)
    _check(load().gdn_static_ws_device_status(ctypes.byref(st), _stream(stream)), "gdn_static_ws_device_status")
    return st.value


def gdn_set_wait_test_mode(immediate: int) -> None:
    """Test hook: 1 makes the tensor-core kernels' main-loop waits give up at once
    unless already complete (drives the GDN_ERR_DEVICE_TIMEOUT path); 0 restores them."""
    _check(load().gdn_set_wait_test_mode(int(immediate)), "gdn_set_wait_test_mode")


def gdn_prologue(d, q_raw, k_raw, v_raw, a, b, conv_w, A_log, dt_bias, cu_seqlens,
                 workspace, workspace_bytes, stream=None, check=True) -> int:
    rc = load().gdn_prologue(ctypes.byref(d), _ptr(q_raw), _ptr(k_raw), _ptr(v_raw), _ptr(a),
                             _ptr(b), _ptr(conv_w), _ptr(A_log), _ptr(dt_bias),
                             _ptr(cu_seqlens), _ptr(workspace), int(workspace_bytes),
                             _stream(stream))
    if check:
        _check(rc, "gdn_prologue")
    return rc


def gdn_chunk_rule(d, cu_seqlens, initial_state, final_state, workspace, workspace_bytes,
                   stream=None, check=True) -> int:
    rc = load().gdn_chunk_rule(ctypes.byref(d), _ptr(cu_seqlens), _ptr(initial_state),
                               _ptr(final_state), _ptr(workspace), int(workspace_bytes),
                               _stream(stream))
    if check:
        _check(rc, "gdn_chunk_rule")
    return rc


def gdn_epilogue(d, gate, norm_w, out, workspace, workspace_bytes, stream=None, check=True) -> int:
    rc = load().gdn_epilogue(ctypes.byref(d), _ptr(gate), _ptr(norm_w), _ptr(out),
                             _ptr(workspace), int(workspace_bytes), _stream(stream))
    if check:
        _check(rc, "gdn_epilogue")
    return rc


def gdn_device_status(workspace, stream=None) -> int:
    st = ctypes.c_int(0)
    _check(load().gdn_device_status(_ptr(workspace), ctypes.byref(st), _stream(stream)),
           "gdn_device_status")
    return st.value


def gdn_chunk_kernel_kind(d: gdn_desc) -> int:
    return load().gdn_chunk_kernel_kind(ctypes.byref(d))


def gdn_decode_workspace_bytes(d: gdn_desc) -> int:
    n = ctypes.c_size_t(0)
    _check(load().gdn_decode_workspace_bytes(ctypes.byref(d), ctypes.byref(n)),
           "gdn_decode_workspace_bytes")
    return n.value


def gdn_decode_step(d, q_raw, k_raw, v_raw, a, b, gate, conv_w, A_log, dt_bias, norm_w,
                    conv_state, state, out, workspace, workspace_bytes, stream=None,
                    check=True) -> int:
    rc = load().gdn_decode_step(ctypes.byref(d), _ptr(q_raw), _ptr(k_raw), _ptr(v_raw), _ptr(a),
                                _ptr(b), _ptr(gate), _ptr(conv_w), _ptr(A_log), _ptr(dt_bias),
                                _ptr(norm_w), _ptr(conv_state), _ptr(state), _ptr(out),
                                _ptr(workspace), int(workspace_bytes), _stream(stream))
    if check:
        _check(rc, "gdn_decode_step")
    return rc


def gdn_forward_with_prefix(d, q_raw, k_raw, v_raw, a, b, gate, conv_w, A_log, dt_bias, norm_w,
                            cu_seqlens, conv_prefix, initial_state, out, final_state, workspace,
                            workspace_bytes, stream=None, check=True) -> int:
    rc = load().gdn_forward_with_prefix(ctypes.byref(d), _ptr(q_raw), _ptr(k_raw), _ptr(v_raw), _ptr(a),
                                        _ptr(b), _ptr(gate), _ptr(conv_w), _ptr(A_log), _ptr(dt_bias),
                                        _ptr(norm_w), _ptr(cu_seqlens), _ptr(conv_prefix),
                                        _ptr(initial_state), _ptr(out), _ptr(final_state), _ptr(workspace),
                                        int(workspace_bytes), _stream(stream))
    if check:
        _check(rc, "gdn_forward_with_prefix")
    return rc


def gdn_span_scan(spans, Hv, dk, dv, A, B, h0, H_in, stream=None, check=True) -> int:
    rc = load().gdn_span_scan(int(spans), int(Hv), int(dk), int(dv), _ptr(A), _ptr(B), _ptr(h0), _ptr(H_in),
                              _stream(stream))
    if check:
        _check(rc, "gdn_span_scan")
    return rc


def gdn_backward_workspace_bytes(d: gdn_desc) -> int:
    n = ctypes.c_size_t(0)
    _check(load().gdn_backward_workspace_bytes(ctypes.byref(d), ctypes.byref(n)),
           "gdn_backward_workspace_bytes")
    return n.value


def gdn_backward(d, q_raw, k_raw, v_raw, a, b, gate, conv_w, A_log, dt_bias, norm_w, cu_seqlens,
                 initial_state, grad_out, grad_final, dq_raw, dk_raw, dv_raw, da, db, dgate, dconv_w,
                 dA_log, ddt_bias, dnorm_w, dinitial_state, workspace, workspace_bytes, stream=None,
                 check=True) -> int:
    rc = load().gdn_backward(ctypes.byref(d), _ptr(q_raw), _ptr(k_raw), _ptr(v_raw), _ptr(a), _ptr(b),
                             _ptr(gate), _ptr(conv_w), _ptr(A_log), _ptr(dt_bias), _ptr(norm_w),
                             _ptr(cu_seqlens), _ptr(initial_state), _ptr(grad_out), _ptr(grad_final),
                             _ptr(dq_raw), _ptr(dk_raw), _ptr(dv_raw), _ptr(da), _ptr(db), _ptr(dgate),
                             _ptr(dconv_w), _ptr(dA_log), _ptr(ddt_bias), _ptr(dnorm_w),
                             _ptr(dinitial_state), _ptr(workspace), int(workspace_bytes), _stream(stream))
    if check:
        _check(rc, "gdn_backward")
    return rc


def _query(name, d) -> int:
    n = ctypes.c_size_t(0)
    _check(getattr(load(), name)(ctypes.byref(d), ctypes.byref(n)), name)
    return n.value


def gdn_recurrence_desc_init(B, T, packed, D, dtype) -> gdn_recurrence_desc:
    d = gdn_recurrence_desc()
    _check(load().gdn_recurrence_desc_init(ctypes.byref(d), B, T, packed, D, dtype), "gdn_recurrence_desc_init")
    return d


def gdn_recurrence_workspace_bytes(d) -> int:
    return _query("gdn_recurrence_workspace_bytes", d)


def gdn_recurrence_backward_workspace_bytes(d) -> int:
    return _query("gdn_recurrence_backward_workspace_bytes", d)


def gdn_recurrence_forward(d, x, a, b, A_log, dt_bias, cu_seqlens, initial_state, out, final_state, chunk_states,
                           workspace, workspace_bytes, stream=None, check=True) -> int:
    rc = load().gdn_recurrence_forward(ctypes.byref(d), _ptr(x), _ptr(a), _ptr(b), _ptr(A_log), _ptr(dt_bias),
                                       _ptr(cu_seqlens), _ptr(initial_state), _ptr(out), _ptr(final_state),
                                       _ptr(chunk_states), _ptr(workspace), int(workspace_bytes), _stream(stream))
    if check:
        _check(rc, "gdn_recurrence_forward")
    return rc


def gdn_recurrence_backward(d, x, a, b, A_log, dt_bias, cu_seqlens, initial_state, chunk_states, grad_out, grad_final,
                            dx, da, db, dA_log, ddt_bias, dinitial_state, workspace, workspace_bytes, stream=None,
                            check=True) -> int:
    rc = load().gdn_recurrence_backward(ctypes.byref(d), _ptr(x), _ptr(a), _ptr(b), _ptr(A_log), _ptr(dt_bias),
                                        _ptr(cu_seqlens), _ptr(initial_state), _ptr(chunk_states), _ptr(grad_out),
                                        _ptr(grad_final), _ptr(dx), _ptr(da), _ptr(db), _ptr(dA_log), _ptr(ddt_bias),
                                        _ptr(dinitial_state), _ptr(workspace), int(workspace_bytes), _stream(stream))
    if check:
        _check(rc, "gdn_recurrence_backward")
    return rc


def gdn_recurrence_step(d, x, a, b, A_log, dt_bias, state, out, stream=None, check=True) -> int:
    rc = load().gdn_recurrence_step(ctypes.byref(d), _ptr(x), _ptr(a), _ptr(b), _ptr(A_log), _ptr(dt_bias),
                                    _ptr(state), _ptr(out), _stream(stream))
    if check:
        _check(rc, "gdn_recurrence_step")
    return rc


def gdn_rotary_desc_init(B, T, packed, Hq, Hk, d, dtype) -> gdn_rotary_desc:
    r = gdn_rotary_desc()
    _check(load().gdn_rotary_desc_init(ctypes.byref(r), B, T, packed, Hq, Hk, d, dtype), "gdn_rotary_desc_init")
    return r


def gdn_rotary_table(rot, theta, scaling, factor, low, high, original, turns) -> None:
    """Fill ``turns``, a HOST int64 tensor of rot/2 entries (the bits of the uint64 table)."""
    if turns.device.type != "cpu" or turns.dtype != torch.int64 or not turns.is_contiguous() or turns.numel() < rot // 2:
        raise ValueError("turns: a contiguous host int64 tensor of rot/2 entries")
    _check(load().gdn_rotary_table(int(rot), float(theta), int(scaling), float(factor), float(low), float(high),
                                   float(original), _ptr(turns)), "gdn_rotary_table")


def gdn_rotary_workspace_bytes(d) -> int:
    return _query("gdn_rotary_workspace_bytes", d)


def gdn_rotary(d, q, k, turns, positions, cu_seqlens, offsets, q_out, k_out, workspace, workspace_bytes, stream=None,
               check=True) -> int:
    rc = load().gdn_rotary(ctypes.byref(d), _ptr(q), _ptr(k), _ptr(turns), _ptr(positions), _ptr(cu_seqlens),
                           _ptr(offsets), _ptr(q_out), _ptr(k_out), _ptr(workspace), int(workspace_bytes),
                           _stream(stream))
    if check:
        _check(rc, "gdn_rotary")
    return rc


def gdn_group_norm_desc_init(N, L, C, G, dtype) -> gdn_group_norm_desc:
    d = gdn_group_norm_desc()
    _check(load().gdn_group_norm_desc_init(ctypes.byref(d), N, L, C, G, dtype), "gdn_group_norm_desc_init")
    return d


def gdn_group_norm_workspace_bytes(d) -> int:
    return _query("gdn_group_norm_workspace_bytes", d)


def gdn_group_norm_backward_workspace_bytes(d) -> int:
    return _query("gdn_group_norm_backward_workspace_bytes", d)


def gdn_group_norm_forward(d, x, weight, bias, out, mean, rstd, workspace, workspace_bytes, stream=None,
                           check=True) -> int:
    rc = load().gdn_group_norm_forward(ctypes.byref(d), _ptr(x), _ptr(weight), _ptr(bias), _ptr(out), _ptr(mean),
                                       _ptr(rstd), _ptr(workspace), int(workspace_bytes), _stream(stream))
    if check:
        _check(rc, "gdn_group_norm_forward")
    return rc


def gdn_group_norm_backward(d, x, weight, bias, mean, rstd, grad_out, dx, dweight, dbias, workspace, workspace_bytes,
                            stream=None, check=True) -> int:
    rc = load().gdn_group_norm_backward(ctypes.byref(d), _ptr(x), _ptr(weight), _ptr(bias), _ptr(mean), _ptr(rstd),
                                        _ptr(grad_out), _ptr(dx), _ptr(dweight), _ptr(dbias), _ptr(workspace),
                                        int(workspace_bytes), _stream(stream))
    if check:
        _check(rc, "gdn_group_norm_backward")
    return rc


# --------------------------------------------------- tensors -> descriptor
def desc_for(q_raw, k_raw, v_raw, a, b, gate, norm_w, *, Hk, Hv, dk, dv,
             cu_seqlens=None, l2_eps=1e-6, norm_eps=1e-5, scale=1.0) -> gdn_desc:
    """Descriptor for [B, T, C] views (channel stride 1) of the given tensors."""
    B, T = q_raw.shape[0], q_raw.shape[1]
    N = (cu_seqlens.numel() - 1) if cu_seqlens is not None else 0
    d = gdn_desc_init(B, T, N, Hk, Hv, dk, dv, DTYPE_CODES[q_raw.dtype])
    for name, t in (("q", q_raw), ("k", k_raw), ("v", v_raw), ("a", a), ("b", b), ("gate", gate)):
        if t.shape[-1] > 1 and t.stride(2) != 1:
            raise ValueError(f"{name}: channel dimension must be contiguous")
        setattr(d, f"{name}_stride_b", t.stride(0))
        setattr(d, f"{name}_stride_t", t.stride(1))
    d.gate_dtype = DTYPE_CODES[gate.dtype]
    d.norm_w_dtype = DTYPE_CODES[norm_w.dtype]
    d.l2_eps, d.norm_eps, d.scale = l2_eps, norm_eps, scale
    return d


@dataclass
class Buffers:
    desc: gdn_desc
    out: torch.Tensor
    final_state: Optional[torch.Tensor]
    workspace: torch.Tensor

    @property
    def ws_bytes(self) -> int:
        return self.workspace.numel()

    def ws_view(self, name: str) -> torch.Tensor:
        """Typed view of one intermediate of the workspace (see gdn_workspace_offsets)."""
        d = self.desc
        lay = gdn_workspace_offsets(d)
        ntok = d.B * d.T
        # intermediates: fp16 for bf16/fp16 activations, fp32 for fp32; the
        # cumulative decay is fp64 for fp32 activations
        st = torch.float32 if d.dtype == GDN_F32 else torch.float16
        gt = torch.float64 if d.dtype == GDN_F32 else torch.float32
        qk = (d.Hk, ntok, d.dk) if d.dtype == GDN_F32 else (2, d.Hk, ntok, d.dk)  # hi, lo planes
        shapes = {"q": (qk, st), "k": (qk, st),
                  "v": ((d.Hv, ntok, d.dv), st), "beta": ((d.Hv, ntok), torch.float32),
                  "gamma": ((d.Hv, ntok), gt), "o": ((ntok, d.Hv, d.dv), st),
                  "status": ((1,), torch.int32), "chunk_off": ((d.N + 1,), torch.int32)}
        shape, dt = shapes[name]
        off = getattr(lay, name)
        n = 1
        for s in shape:
            n *= s
        nbytes = n * torch.empty((), dtype=dt).element_size()
        return self.workspace[off:off + nbytes].view(dt).view(shape)


def alloc(desc: gdn_desc, device, want_final_state=True) -> Buffers:
    """Allocate out, final_state and the workspace for ``desc`` with torch."""
    act = ACT_TORCH[desc.dtype]
    out = torch.empty((desc.B, desc.T, desc.Hv, desc.dv), dtype=act, device=device)
    fin = (torch.empty((desc.N, desc.Hv, desc.dk, desc.dv), dtype=torch.float32, device=device)
           if want_final_state else None)
    ws = torch.empty(gdn_workspace_bytes(desc), dtype=torch.uint8, device=device)
    return Buffers(desc, out, fin, ws)


def make_desc(inp) -> gdn_desc:
    w = inp.w
    return desc_for(inp.q_raw, inp.k_raw, inp.v_raw, inp.a, inp.b, inp.gate, inp.norm_w,
                    Hk=w.Hk, Hv=w.Hv, dk=w.dk, dv=w.dv, cu_seqlens=inp.cu_seqlens)


def forward(inp, bufs: Optional[Buffers] = None, stream=None, want_final_state=True) -> Buffers:
    """Run the core forward on an ``Inputs``-like object whose tensors live on
    the GPU (see ``workloads.Inputs``)."""
    if bufs is None:
        bufs = alloc(make_desc(inp), inp.q_raw.device, want_final_state)
    gdn_forward(bufs.desc, inp.q_raw, inp.k_raw, inp.v_raw, inp.a, inp.b, inp.gate, inp.conv_w,
                inp.A_log, inp.dt_bias, inp.norm_w, inp.cu_seqlens, inp.initial_state,
                bufs.out, bufs.final_state, bufs.workspace, bufs.ws_bytes, stream)
    return bufs


@dataclass
class Grads:
    dq_raw: torch.Tensor
    dk_raw: torch.Tensor
    dv_raw: torch.Tensor
    da: torch.Tensor
    db: torch.Tensor
    dgate: torch.Tensor
    dconv_w: torch.Tensor
    dA_log: torch.Tensor
    ddt_bias: torch.Tensor
    dnorm_w: torch.Tensor
    dinitial_state: Optional[torch.Tensor]
    workspace: torch.Tensor


def alloc_grads(desc: gdn_desc, device, want_dinitial=True) -> Grads:
    """Gradient buffers (dense, see gdn_backward in include/gdn.h) and the workspace."""
    act = ACT_TORCH[desc.dtype]
    ntok = desc.B * desc.T
    ch_qk, ch_v = desc.Hk * desc.dk, desc.Hv * desc.dv
    f32 = dict(dtype=torch.float32, device=device)
    return Grads(
        dq_raw=torch.empty((ntok, ch_qk), dtype=act, device=device),
        dk_raw=torch.empty((ntok, ch_qk), dtype=act, device=device),
        dv_raw=torch.empty((ntok, ch_v), dtype=act, device=device),
        da=torch.empty((ntok, desc.Hv), dtype=act, device=device),
        db=torch.empty((ntok, desc.Hv), dtype=act, device=device),
        dgate=torch.empty((ntok, ch_v), dtype=ACT_TORCH[desc.gate_dtype], device=device),
        dconv_w=torch.empty((2 * ch_qk + ch_v, 4), **f32), dA_log=torch.empty(desc.Hv, **f32),
        ddt_bias=torch.empty(desc.Hv, **f32), dnorm_w=torch.empty(desc.dv, **f32),
        dinitial_state=torch.empty((desc.N, desc.Hv, desc.dk, desc.dv), **f32) if want_dinitial else None,
        workspace=torch.empty(gdn_backward_workspace_bytes(desc), dtype=torch.uint8, device=device))


def backward(inp, grad_out, grad_final=None, grads: Optional[Grads] = None, stream=None) -> Grads:
    """Gradients of sum(grad_out * out) + sum(grad_final * final_state) for an
    ``Inputs``-like object on the GPU (grad_out [B, T, Hv, dv] act dtype,
    contiguous; grad_final [N, Hv, dk, dv] fp32 or None)."""
    d = make_desc(inp)
    if grads is None:
        grads = alloc_grads(d, inp.q_raw.device)
    gdn_backward(d, inp.q_raw, inp.k_raw, inp.v_raw, inp.a, inp.b, inp.gate, inp.conv_w, inp.A_log,
                 inp.dt_bias, inp.norm_w, inp.cu_seqlens, inp.initial_state, grad_out, grad_final,
                 grads.dq_raw, grads.dk_raw, grads.dv_raw, grads.da, grads.db, grads.dgate, grads.dconv_w,
                 grads.dA_log, grads.ddt_bias, grads.dnorm_w, grads.dinitial_state, grads.workspace,
                 grads.workspace.numel(), stream)
    return grads


# ------------------------- operators beside the gated delta rule, on tensors
def _expect(t, name, shape, dtype, device, contiguous=True):
    """One tensor argument of the functions below: what a kernel would take on trust is checked here."""
    if t is None:
        return
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype != dtype:
        raise ValueError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if t.device != device:
        raise ValueError(f"{name}: on {t.device}, expected {device}")
    if contiguous and not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")


def _strides(t, name):
    """(batch, token) element strides of a [B, T, C] view. A dimension of one element has no
    stride of its own, whatever torch reports for it."""
    if t.dim() != 3 or (t.shape[2] > 1 and t.stride(2) != 1):
        raise ValueError(f"{name}: a [B, T, C] view with contiguous channels")
    st = t.stride(1) if t.shape[1] > 1 else t.shape[2]
    return t.stride(0) if t.shape[0] > 1 else st * t.shape[1], st


def _on_current(t):
    """The library launches on the current device: a tensor elsewhere is refused."""
    if t.device.type != "cuda" or t.device.index != torch.cuda.current_device():
        raise ValueError(f"tensors on {t.device}, but the current device is cuda:{torch.cuda.current_device()}")


def _allocating(stream):
    """Where a function below allocates: on the stream that it launches on, whose order then also guards the
    memory's former and next use."""
    if stream is None:
        return contextlib.nullcontext()
    return torch.cuda.stream(torch.cuda.ExternalStream(stream) if isinstance(stream, int) else stream)


def _expect_workspace(t, device):
    _expect(t, "workspace", (t.numel(),), torch.uint8, device)


def recurrence_desc_for(x, a, b, cu_seqlens=None) -> gdn_recurrence_desc:
    """Descriptor of the gated linear recurrence over [B, T, D] views x, a, b."""
    B, T, D = x.shape
    for t, name in ((a, "a"), (b, "b")):
        _expect(t, name, x.shape, x.dtype, x.device, contiguous=False)
    d = gdn_recurrence_desc_init(B, T, 0 if cu_seqlens is None else cu_seqlens.numel() - 1, D, DTYPE_CODES[x.dtype])
    for name, t in (("x", x), ("a", a), ("b", b)):
        sb, st = _strides(t, name)
        setattr(d, f"{name}_stride_b", sb)
        setattr(d, f"{name}_stride_t", st)
    return d


@dataclass
class RecurrenceBuffers:
    desc: gdn_recurrence_desc
    out: torch.Tensor
    final_state: Optional[torch.Tensor]
    chunk_states: Optional[torch.Tensor]
    workspace: torch.Tensor

    @property
    def ws_bytes(self) -> int:
        return self.workspace.numel()


def alloc_recurrence(desc, device, want_final_state=True, want_chunk_states=False) -> RecurrenceBuffers:
    """Output buffers of gdn_recurrence_forward; chunk_states are what its backward reads."""
    f32 = dict(dtype=torch.float32, device=device)
    chunks = -(-desc.T // GDN_RECURRENCE_CHUNK)
    return RecurrenceBuffers(
        desc, torch.empty((desc.B, desc.T, desc.D), dtype=ACT_TORCH[desc.dtype], device=device),
        torch.empty((desc.N, desc.D), **f32) if want_final_state else None,
        torch.empty((desc.B, chunks, desc.D), **f32) if want_chunk_states else None,
        torch.empty(gdn_recurrence_workspace_bytes(desc), dtype=torch.uint8, device=device))


@dataclass
class RecurrenceGrads:
    dx: torch.Tensor
    da: torch.Tensor
    db: torch.Tensor
    dA_log: torch.Tensor
    ddt_bias: torch.Tensor
    dinitial_state: Optional[torch.Tensor]
    workspace: torch.Tensor

    @property
    def ws_bytes(self) -> int:
        return self.workspace.numel()


def alloc_recurrence_grads(desc, device, want_dinitial=True) -> RecurrenceGrads:
    """Gradient buffers and workspace of gdn_recurrence_backward."""
    f32 = dict(dtype=torch.float32, device=device)
    tok = lambda: torch.empty((desc.B, desc.T, desc.D), dtype=ACT_TORCH[desc.dtype], device=device)  # noqa: E731
    return RecurrenceGrads(tok(), tok(), tok(), torch.empty(desc.D, **f32), torch.empty(desc.D, **f32),
                           torch.empty((desc.N, desc.D), **f32) if want_dinitial else None,
                           torch.empty(gdn_recurrence_backward_workspace_bytes(desc), dtype=torch.uint8, device=device))


def _check_recurrence(d, x, A_log, dt_bias, cu_seqlens, initial_state):
    _on_current(x)
    for t, name in ((A_log, "A_log"), (dt_bias, "dt_bias")):
        _expect(t, name, (d.D,), torch.float32, x.device)
    _expect(cu_seqlens, "cu_seqlens", (d.N + 1,), torch.int32, x.device)
    _expect(initial_state, "initial_state", (d.N, d.D), torch.float32, x.device)


def recurrence_forward(x, a, b, A_log, dt_bias, cu_seqlens=None, initial_state=None, want_final_state=True,
                       want_chunk_states=False, bufs: Optional[RecurrenceBuffers] = None,
                       stream=None) -> RecurrenceBuffers:
    """Gated linear recurrence (see gdn_recurrence_forward in include/gdn.h) of [B, T, D] views on the
    GPU; packed sequences with cu_seqlens (int32 [N+1], B = 1). want_chunk_states keeps what
    ``recurrence_backward`` can use."""
    d = recurrence_desc_for(x, a, b, cu_seqlens)
    _check_recurrence(d, x, A_log, dt_bias, cu_seqlens, initial_state)
    if bufs is None:
        with _allocating(stream):
            bufs = alloc_recurrence(d, x.device, want_final_state, want_chunk_states)
    else:
        _expect(bufs.out, "bufs.out", (d.B, d.T, d.D), x.dtype, x.device)
        _expect(bufs.final_state, "bufs.final_state", (d.N, d.D), torch.float32, x.device)
        _expect(bufs.chunk_states, "bufs.chunk_states", (d.B, -(-d.T // GDN_RECURRENCE_CHUNK), d.D), torch.float32,
                x.device)
        _expect_workspace(bufs.workspace, x.device)
        bufs.desc = d
    gdn_recurrence_forward(d, x, a, b, A_log, dt_bias, cu_seqlens, initial_state, bufs.out, bufs.final_state,
                           bufs.chunk_states, bufs.workspace, bufs.ws_bytes, stream)
    return bufs


def recurrence_backward(x, a, b, A_log, dt_bias, grad_out, grad_final=None, chunk_states=None, cu_seqlens=None,
                        initial_state=None, grads: Optional[RecurrenceGrads] = None, stream=None) -> RecurrenceGrads:
    """Gradients of sum(grad_out * out) + sum(grad_final * final_state). chunk_states: the forward's of
    the same inputs, or None (recomputed)."""
    d = recurrence_desc_for(x, a, b, cu_seqlens)
    _check_recurrence(d, x, A_log, dt_bias, cu_seqlens, initial_state)
    _expect(grad_out, "grad_out", (d.B, d.T, d.D), x.dtype, x.device)
    _expect(grad_final, "grad_final", (d.N, d.D), torch.float32, x.device)
    _expect(chunk_states, "chunk_states", (d.B, -(-d.T // GDN_RECURRENCE_CHUNK), d.D), torch.float32, x.device)
    if grads is None:
        with _allocating(stream):
            grads = alloc_recurrence_grads(d, x.device)
    else:
        for name in ("dx", "da", "db"):
            _expect(getattr(grads, name), f"grads.{name}", (d.B, d.T, d.D), x.dtype, x.device)
        for name in ("dA_log", "ddt_bias"):
            _expect(getattr(grads, name), f"grads.{name}", (d.D,), torch.float32, x.device)
        _expect(grads.dinitial_state, "grads.dinitial_state", (d.N, d.D), torch.float32, x.device)
        _expect_workspace(grads.workspace, x.device)
    gdn_recurrence_backward(d, x, a, b, A_log, dt_bias, cu_seqlens, initial_state, chunk_states, grad_out, grad_final,
                            grads.dx, grads.da, grads.db, grads.dA_log, grads.ddt_bias, grads.dinitial_state,
                            grads.workspace, grads.ws_bytes, stream)
    return grads


def recurrence_step(x, a, b, A_log, dt_bias, state, out=None, stream=None) -> torch.Tensor:
    """One more token of each sequence: x, a, b [B, 1, D] views, state fp32 [B, D] updated in place."""
    d = recurrence_desc_for(x, a, b)
    _check_recurrence(d, x, A_log, dt_bias, None, None)
    _expect(state, "state", (d.B, d.D), torch.float32, x.device)
    if out is None:
        with _allocating(stream):
            out = torch.empty((d.B, d.T, d.D), dtype=x.dtype, device=x.device)
    _expect(out, "out", (d.B, 1, d.D), x.dtype, x.device)
    gdn_recurrence_step(d, x, a, b, A_log, dt_bias, state, out, stream)
    return out


def rotary_table(rot, theta=10000.0, scaling="plain", factor=1.0, low=1.0, high=4.0, original=8192, device="cuda"):
    """The table of turns for ``rotary`` on ``device``: int64 [rot/2] holding the bits of the uint64
    entries (see gdn_rotary_table and gdn_rotary_scaling in include/gdn.h)."""
    if scaling not in ROTARY_SCALINGS:
        raise ValueError(f"scaling: one of {sorted(ROTARY_SCALINGS)}, not {scaling!r}")
    turns = torch.empty(max(int(rot) // 2, 0), dtype=torch.int64)
    gdn_rotary_table(rot, theta, ROTARY_SCALINGS[scaling], factor, low, high, original, turns)
    return turns.to(device)


def rotary_desc_for(q, k, q_out, k_out, *, d, rot=None, layout="half", inverse=False, scale=1.0,
                    cu_seqlens=None) -> gdn_rotary_desc:
    """Descriptor of ``rotary`` for [B, T, H*d] views (k and k_out None: no k)."""
    if layout not in ROTARY_LAYOUTS:
        raise ValueError(f"layout: one of {sorted(ROTARY_LAYOUTS)}, not {layout!r}")
    if (k is None) != (k_out is None):
        raise ValueError("k and k_out: both or neither")
    B, T = q.shape[:2]
    for name, t, like in (("q_out", q_out, q), ("k_out", k_out, k)):
        if like is not None:
            _expect(t, name, like.shape, q.dtype, q.device, contiguous=False)
    if k is not None:
        _expect(k, "k", (B, T, k.shape[-1]), q.dtype, q.device, contiguous=False)
    heads = []
    for name, t in (("q", q), ("k", k)):
        if t is not None and t.shape[-1] % d:
            raise ValueError(f"{name}: {t.shape[-1]} channels, not a multiple of the head's {d}")
        heads.append(0 if t is None else t.shape[-1] // d)
    r = gdn_rotary_desc_init(B, T, 0 if cu_seqlens is None else cu_seqlens.numel() - 1, heads[0], heads[1], d,
                             DTYPE_CODES[q.dtype])
    for name, t in (("q", q), ("k", k), ("q_out", q_out), ("k_out", k_out)):
        if t is not None:
            sb, st = _strides(t, name)
            setattr(r, f"{name}_stride_b", sb)
            setattr(r, f"{name}_stride_t", st)
    r.rot = d if rot is None else rot
    r.layout, r.inverse, r.scale = ROTARY_LAYOUTS[layout], int(bool(inverse)), scale
    return r


def rotary(q, k, table, *, d, rot=None, layout="half", inverse=False, scale=1.0, positions=None, cu_seqlens=None,
           offsets=None, q_out=None, k_out=None, workspace=None, stream=None):
    """Rotary positions of q and k (k may be None): (q_out, k_out), new tensors unless given; pass q and
    k themselves to rotate in place. inverse=True is the gradient. positions int32 [B, T], or offsets
    int32 [N] added to the positions counted from each sequence's start."""
    _on_current(q)
    with _allocating(stream):
        if q_out is None:
            q_out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        if k is not None and k_out is None:
            k_out = torch.empty(k.shape, dtype=k.dtype, device=k.device)
    r = rotary_desc_for(q, k, q_out, k_out, d=d, rot=rot, layout=layout, inverse=inverse, scale=scale,
                        cu_seqlens=cu_seqlens)
    _expect(table, "table", (r.rot // 2,), torch.int64, q.device)
    _expect(positions, "positions", (r.B, r.T), torch.int32, q.device)
    _expect(cu_seqlens, "cu_seqlens", (r.N + 1,), torch.int32, q.device)
    _expect(offsets, "offsets", (r.N,), torch.int32, q.device)
    if workspace is None:
        with _allocating(stream):
            workspace = torch.empty(gdn_rotary_workspace_bytes(r), dtype=torch.uint8, device=q.device)
    _expect_workspace(workspace, q.device)
    gdn_rotary(r, q, k, table, positions, cu_seqlens, offsets, q_out, k_out, workspace, workspace.numel(), stream)
    return q_out, k_out


def group_norm_desc_for(x, weight=None, *, groups, act="silu", eps=1e-5) -> gdn_group_norm_desc:
    """Descriptor of the group norm of a [N, L, C] view."""
    if act not in ACTIVATIONS:
        raise ValueError(f"act: one of {sorted(ACTIVATIONS)}, not {act!r}")
    N, L, C = x.shape
    d = gdn_group_norm_desc_init(N, L, C, groups, DTYPE_CODES[x.dtype])
    d.x_stride_n, d.x_stride_l = _strides(x, "x")
    if weight is not None:
        d.weight_dtype = DTYPE_CODES[weight.dtype]
    d.act, d.eps = ACTIVATIONS[act], eps
    return d


@dataclass
class GroupNormBuffers:
    desc: gdn_group_norm_desc
    out: torch.Tensor
    mean: Optional[torch.Tensor]
    rstd: Optional[torch.Tensor]
    workspace: torch.Tensor

    @property
    def ws_bytes(self) -> int:
        return self.workspace.numel()


def alloc_group_norm(desc, device) -> GroupNormBuffers:
    f32 = dict(dtype=torch.float32, device=device)
    return GroupNormBuffers(
        desc, torch.empty((desc.N, desc.L, desc.C), dtype=ACT_TORCH[desc.dtype], device=device),
        torch.empty((desc.N, desc.G), **f32), torch.empty((desc.N, desc.G), **f32),
        torch.empty(gdn_group_norm_workspace_bytes(desc), dtype=torch.uint8, device=device))


@dataclass
class GroupNormGrads:
    dx: torch.Tensor
    dweight: Optional[torch.Tensor]
    dbias: Optional[torch.Tensor]
    workspace: torch.Tensor

    @property
    def ws_bytes(self) -> int:
        return self.workspace.numel()


def alloc_group_norm_grads(desc, device) -> GroupNormGrads:
    f32 = dict(dtype=torch.float32, device=device)
    return GroupNormGrads(torch.empty((desc.N, desc.L, desc.C), dtype=ACT_TORCH[desc.dtype], device=device),
                          torch.empty(desc.C, **f32), torch.empty(desc.C, **f32),
                          torch.empty(gdn_group_norm_backward_workspace_bytes(desc), dtype=torch.uint8, device=device))


def _check_group_norm(d, x, weight, bias):
    _on_current(x)
    for t, name in ((weight, "weight"), (bias, "bias")):
        _expect(t, name, (d.C,), ACT_TORCH[d.weight_dtype], x.device)


def group_norm_forward(x, weight=None, bias=None, *, groups, act="silu", eps=1e-5,
                       bufs: Optional[GroupNormBuffers] = None, stream=None) -> GroupNormBuffers:
    """Group norm with an activation of a [N, L, C] view (see gdn_group_norm_forward in include/gdn.h);
    mean and rstd are kept for ``group_norm_backward``."""
    d = group_norm_desc_for(x, weight if weight is not None else bias, groups=groups, act=act, eps=eps)
    _check_group_norm(d, x, weight, bias)
    if bufs is None:
        with _allocating(stream):
            bufs = alloc_group_norm(d, x.device)
    else:
        _expect(bufs.out, "bufs.out", x.shape, x.dtype, x.device)
        for name in ("mean", "rstd"):
            _expect(getattr(bufs, name), f"bufs.{name}", (d.N, d.G), torch.float32, x.device)
        _expect_workspace(bufs.workspace, x.device)
        bufs.desc = d
    gdn_group_norm_forward(d, x, weight, bias, bufs.out, bufs.mean, bufs.rstd, bufs.workspace, bufs.ws_bytes, stream)
    return bufs


def group_norm_backward(x, weight, bias, mean, rstd, grad_out, *, groups, act="silu", eps=1e-5,
                        grads: Optional[GroupNormGrads] = None, stream=None) -> GroupNormGrads:
    """Gradients of sum(grad_out * out) with the forward's mean and rstd."""
    d = group_norm_desc_for(x, weight if weight is not None else bias, groups=groups, act=act, eps=eps)
    _check_group_norm(d, x, weight, bias)
    _expect(grad_out, "grad_out", x.shape, x.dtype, x.device)
    for t, name in ((mean, "mean"), (rstd, "rstd")):
        _expect(t, name, (d.N, d.G), torch.float32, x.device)
    if grads is None:
        with _allocating(stream):
            grads = alloc_group_norm_grads(d, x.device)
    else:
        _expect(grads.dx, "grads.dx", x.shape, x.dtype, x.device)
        for name in ("dweight", "dbias"):
            _expect(getattr(grads, name), f"grads.{name}", (d.C,), torch.float32, x.device)
        _expect_workspace(grads.workspace, x.device)
    gdn_group_norm_backward(d, x, weight, bias, mean, rstd, grad_out, grads.dx, grads.dweight, grads.dbias,
                            grads.workspace, grads.ws_bytes, stream)
    return grads
