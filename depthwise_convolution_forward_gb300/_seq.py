"""ctypes binding of the sequence operators (``include/gconv_seq.h``):
causal depthwise convolution, gated linear recurrence, residual + RMS norm to
8 bits and the 8-bit matrix product.  Argument marshalling only, in the manner
of ``_binding``; names match the C ABI.

Tensors are torch tensors (or device addresses as ints); ``None`` is NULL.
Problem records are made once for a shape and kept by the caller.
"""
from __future__ import annotations

import ctypes
from typing import Optional, Sequence

from . import _binding as B

ACT_NONE, ACT_SILU = 0, 1
GCONV_SEQ_MAX_D = (1 << 31) - 128
GCONV_CONV1D_MAX_K = 8
GCONV_SCAN_CHUNK = 8
GCONV_NORM_MAX_D = 32768
GCONV_MATMUL_Q8_MAX_K = 65536
GCONV_MATMUL_Q8_MAX_N = 1 << 21


class gconv_conv1d_problem(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int64), ("T", ctypes.c_int64), ("D", ctypes.c_int32), ("K", ctypes.c_int32),
                ("act", ctypes.c_int32), ("reserved", ctypes.c_int32), ("x_stride", ctypes.c_int64 * 2),
                ("y_stride", ctypes.c_int64 * 2)]


class gconv_scan_problem(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int64), ("T", ctypes.c_int64), ("D", ctypes.c_int32), ("decay", ctypes.c_float),
                ("x_stride", ctypes.c_int64 * 2), ("r_stride", ctypes.c_int64 * 2), ("i_stride", ctypes.c_int64 * 2),
                ("y_stride", ctypes.c_int64 * 2)]


class gconv_norm_problem(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("D", ctypes.c_int32), ("eps", ctypes.c_float),
                ("x_stride", ctypes.c_int64), ("residual_stride", ctypes.c_int64), ("y_stride", ctypes.c_int64),
                ("reserved", ctypes.c_int64)]


class gconv_matmul_q8_problem(ctypes.Structure):
    _fields_ = [("M", ctypes.c_int64), ("N", ctypes.c_int32), ("K", ctypes.c_int32), ("y_stride", ctypes.c_int64),
                ("reserved", ctypes.c_int64)]


_fn = None  # the C functions, in the order of declare()


def declare(lib) -> None:
    """Argument types of the sequence operators (called by load_library)."""
    vp, i32, i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
    conv_p, scan_p = ctypes.POINTER(gconv_conv1d_problem), ctypes.POINTER(gconv_scan_problem)
    norm_p, mm_p, n_p = ctypes.POINTER(gconv_norm_problem), ctypes.POINTER(gconv_matmul_q8_problem), ctypes.POINTER(i64)
    for name, args in {
        "gconv_causal_conv1d_fwd": [vp] * 7 + [conv_p, i32, vp],
        "gconv_causal_conv1d_bwd": [vp] * 11 + [conv_p, i32, vp, i64, vp],
        "gconv_causal_conv1d_bwd_workspace_size": [conv_p, i32, n_p],
        "gconv_gated_scan_fwd": [vp] * 9 + [scan_p, i32, vp],
        "gconv_gated_scan_bwd": [vp] * 13 + [scan_p, i32, vp, i64, vp],
        "gconv_gated_scan_saved_size": [scan_p, i32, n_p],
        "gconv_gated_scan_bwd_workspace_size": [scan_p, i32, n_p],
        "gconv_rms_norm_q8": [vp] * 7 + [norm_p, i32, vp],
        "gconv_quantize_rows_q8": [vp] * 3 + [norm_p, i32, vp],
        "gconv_matmul_q8": [vp] * 6 + [mm_p, i32, vp],
    }.items():
        f = getattr(lib, name)
        f.restype, f.argtypes = i32, args
    global _fn
    _fn = (lib.gconv_causal_conv1d_fwd, lib.gconv_causal_conv1d_bwd, lib.gconv_gated_scan_fwd, lib.gconv_gated_scan_bwd,
           lib.gconv_rms_norm_q8, lib.gconv_quantize_rows_q8, lib.gconv_matmul_q8)


def _load():
    B.load_library()
    return _fn


def _pair(stride: Optional[Sequence[int]]):
    return (ctypes.c_int64 * 2)(*(stride or (0, 0)))


def make_conv1d_problem(b: int, t: int, d: int, k: int, act: int = ACT_NONE, x_stride=None,
                        y_stride=None) -> gconv_conv1d_problem:
    """Record of a causal convolution; strides are (batch, token) in elements,
    None for packed [B, T, D]."""
    return gconv_conv1d_problem(b, t, d, k, act, 0, _pair(x_stride), _pair(y_stride))


def make_scan_problem(b: int, t: int, d: int, decay: float = 8.0, x_stride=None, r_stride=None, i_stride=None,
                      y_stride=None) -> gconv_scan_problem:
    """Record of a gated scan; strides are (batch, token) in elements, None for
    packed [B, T, D]."""
    return gconv_scan_problem(b, t, d, decay, _pair(x_stride), _pair(r_stride), _pair(i_stride), _pair(y_stride))


def make_norm_problem(rows: int, d: int, eps: float = 1e-6, x_stride: int = 0, residual_stride: int = 0,
                      y_stride: int = 0) -> gconv_norm_problem:
    """Record of the norm and of the row quantiser; row strides in elements, 0
    for packed."""
    return gconv_norm_problem(rows, d, eps, x_stride, residual_stride, y_stride, 0)


def make_matmul_q8_problem(m: int, n: int, k: int, y_stride: int = 0) -> gconv_matmul_q8_problem:
    """Record of an 8-bit product [m, k] x [n, k]^T; y_stride 0 for packed."""
    return gconv_matmul_q8_problem(m, n, k, y_stride, 0)


def _size(fn, p, dtype: int) -> int:
    n = ctypes.c_int64(0)
    B._check(fn(p, dtype, ctypes.byref(n)))
    return n.value


def _bytes(workspace, workspace_bytes: int) -> int:
    if workspace is not None and not isinstance(workspace, int) and not workspace_bytes:
        return workspace.numel() * workspace.element_size()
    return workspace_bytes


# A call of a few microseconds on the GPU is over before Python has marshalled
# the next one's arguments, so these functions do as little as they can: the C
# functions are looked up once, and a record is passed by reference by its type.
def _a(t):
    if t is None:
        return None
    try:
        return t.data_ptr()
    except AttributeError:
        return t  # a device address


def _s(stream):
    try:
        return stream.cuda_stream
    except AttributeError:
        return stream  # a stream's address, or None


def gconv_causal_conv1d_fwd(x, w, bias, state_in, lens, y, state_out, p: gconv_conv1d_problem, dtype: int,
                            stream=None) -> None:
    """Causal depthwise convolution with carried state (see gconv_seq.h)."""
    st = (_fn or _load())[0](_a(x), _a(w), _a(bias), _a(state_in), _a(lens), _a(y), _a(state_out), p, dtype, _s(stream))
    if st:
        B._check(st)


def gconv_causal_conv1d_bwd_workspace_size(p: gconv_conv1d_problem, dtype: int) -> int:
    """Device workspace bytes gconv_causal_conv1d_bwd needs."""
    return _size(B.load_library().gconv_causal_conv1d_bwd_workspace_size, p, dtype)


def gconv_causal_conv1d_bwd(dy, dstate_out, x, w, bias, state_in, lens, dx, dw, dbias, dstate_in,
                            p: gconv_conv1d_problem, dtype: int, workspace=None, workspace_bytes: int = 0,
                            stream=None) -> None:
    """Gradients of the causal depthwise convolution (see gconv_seq.h)."""
    st = (_fn or _load())[1](_a(dy), _a(dstate_out), _a(x), _a(w), _a(bias), _a(state_in), _a(lens), _a(dx), _a(dw),
                             _a(dbias), _a(dstate_in), p, dtype, _a(workspace), _bytes(workspace, workspace_bytes),
                             _s(stream))
    if st:
        B._check(st)


def gconv_gated_scan_saved_size(p: gconv_scan_problem, dtype: int) -> int:
    """Bytes of the states the forward pass saves for the backward pass."""
    return _size(B.load_library().gconv_gated_scan_saved_size, p, dtype)


def gconv_gated_scan_bwd_workspace_size(p: gconv_scan_problem, dtype: int) -> int:
    """Device workspace bytes gconv_gated_scan_bwd needs."""
    return _size(B.load_library().gconv_gated_scan_bwd_workspace_size, p, dtype)


def gconv_gated_scan_fwd(x, r, i, lam, h0, lens, y, hT, saved, p: gconv_scan_problem, dtype: int,
                         stream=None) -> None:
    """Gated linear recurrence (see gconv_seq.h)."""
    st = (_fn or _load())[2](_a(x), _a(r), _a(i), _a(lam), _a(h0), _a(lens), _a(y), _a(hT), _a(saved), p, dtype, _s(stream))
    if st:
        B._check(st)


def gconv_gated_scan_bwd(dy, dhT, x, r, i, lam, lens, saved, dx, dr, di, dlam, dh0, p: gconv_scan_problem, dtype: int,
                         workspace=None, workspace_bytes: int = 0, stream=None) -> None:
    """Gradients of the gated linear recurrence (see gconv_seq.h)."""
    st = (_fn or _load())[3](_a(dy), _a(dhT), _a(x), _a(r), _a(i), _a(lam), _a(lens), _a(saved), _a(dx), _a(dr), _a(di),
                             _a(dlam), _a(dh0), p, dtype, _a(workspace), _bytes(workspace, workspace_bytes), _s(stream))
    if st:
        B._check(st)


def gconv_rms_norm_q8(x, residual, weight, residual_out, y, q, scale, p: gconv_norm_problem, dtype: int,
                      stream=None) -> None:
    """Residual addition + RMS norm with an 8-bit output (see gconv_seq.h)."""
    st = (_fn or _load())[4](_a(x), _a(residual), _a(weight), _a(residual_out), _a(y), _a(q), _a(scale), p, dtype, _s(stream))
    if st:
        B._check(st)


def gconv_quantize_rows_q8(x, q, scale, p: gconv_norm_problem, dtype: int, stream=None) -> None:
    """Rows to 8 bits with a scale each (see gconv_seq.h)."""
    st = (_fn or _load())[5](_a(x), _a(q), _a(scale), p, dtype, _s(stream))
    if st:
        B._check(st)


def gconv_matmul_q8(xq, x_scale, wq, w_scale, bias, y, p: gconv_matmul_q8_problem, dtype: int, stream=None) -> None:
    """8-bit matrix product with row scales on both sides (see gconv_seq.h)."""
    st = (_fn or _load())[6](_a(xq), _a(x_scale), _a(wq), _a(w_scale), _a(bias), _a(y), p, dtype, _s(stream))
    if st:
        B._check(st)
