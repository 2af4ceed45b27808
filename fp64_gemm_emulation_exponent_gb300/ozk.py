"""Python binding of libozk (ctypes): argument marshalling only.

Every function here forwards to the C-ABI entry point of the same name in
``include/ozk.h``; all computation runs in the library's CUDA kernels.  The
library must have been built (``fp64_gemm_emulation_exponent_gb300.build``);
loading fails loudly otherwise, and there is no CPU fallback.
"""
from __future__ import annotations

import ctypes
import os

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libozk.so")

OZK_OK = 0
OZK_ERR_INVALID_ARG = 1
OZK_ERR_UNSUPPORTED = 2
OZK_ERR_WORKSPACE = 3
OZK_ERR_CUDA = 4
OZK_ERR_TIMEOUT = 5
OZK_ERR_DEVICE = 6
OZK_MAX_MODULI = 20
OZK_MAX_K = 4194304
OZK_SPLIT_MAX_K = 131008
OZK_SCALE_NONFINITE = -(2**31)
OZK_LIMBS = 8
OZK_SCALE_NOALLOC_MAX = 262144
OZK_MAX_GROUPS = 1024
OZK_BF16, OZK_F16, OZK_F32, OZK_F64 = 0, 1, 2, 3
OZK_NVFP4, OZK_MXFP4 = 0, 1
OZK_SILU, OZK_GELU, OZK_GELU_TANH = 0, 1, 2

_i64, _i32, _vp, _sz = ctypes.c_int64, ctypes.c_int, ctypes.c_void_p, ctypes.c_size_t
_f32 = ctypes.c_float

# name -> (restype, argtypes), mirroring include/ozk.h
SIGNATURES = {
    "ozk_status_string": (ctypes.c_char_p, [_i32]),
    "ozk_moduli": (_i32, [_i32, _vp]),
    "ozk_beta": (_i32, [_i64, _i32]),
    "ozk_kpad": (_i64, [_i64]),
    "ozk_gamma": (_i32, [_i64, _i32]),
    "ozk_dgemm_norm": (_i32, [_i64, _i64, _i64, _vp, _i64, _vp, _i64, _vp, _i64, _i32, _vp]),
    "ozk_dgemm_norm_ws": (_i32, [_i64, _i64, _i64, _vp, _i64, _vp, _i64, _vp, _i64, _i32, _vp, _sz, _vp]),
    "ozk_dgemm_norm_ws_timed": (_i32, [_i64, _i64, _i64, _vp, _i64, _vp, _i64, _vp, _i64, _i32, _vp, _sz, _vp, _vp]),
    "ozk_scale_norm": (_i32, [_i64, _i64, _i64, _vp, _i64, _vp, _i64, _i32, _vp, _vp, _vp, _vp]),
    "ozk_moduli_for_bits": (_i32, [_i64, _i32]),
    "ozk_dgemm_bits": (_i32, [_i64, _i64, _i64, _vp, _i64, _vp, _i64, _vp, _i64, _i32, _vp]),
    "ozk_workspace_size": (_sz, [_i64, _i64, _i64, _i32]),
    "ozk_workspace_layout": (_i32, [_i64, _i64, _i64, _i32, _vp]),
    "ozk_dgemm": (_i32, [_i64, _i64, _i64, _vp, _i64, _vp, _i64, _vp, _i64, _i32, _vp]),
    "ozk_dgemm_ws": (_i32, [_i64, _i64, _i64, _vp, _i64, _vp, _i64, _vp, _i64, _i32, _vp, _sz, _vp]),
    "ozk_dgemm_ws_timed": (_i32, [_i64, _i64, _i64, _vp, _i64, _vp, _i64, _vp, _i64, _i32, _vp, _sz, _vp, _vp]),
    "ozk_dgemm_host": (_i32, [_i64, _i64, _i64, _vp, _i64, _vp, _i64, _vp, _i64, _i32, _vp]),
    "ozk_dgemm_host_async": (_i32, [_i64, _i64, _i64, _vp, _i64, _vp, _i64, _vp, _i64, _i32, _vp]),
    "ozk_stream_status": (_i32, [_vp]),
    "ozk_release_cached": (_i32, []),
    "ozk_scale": (_i32, [_i64, _i64, _i64, _vp, _i64, _vp, _i64, _i32, _vp, _vp, _vp, _vp]),
    "ozk_scale_noalloc": (_i32, [_i64, _i64, _i64, _vp, _i64, _vp, _i64, _i32, _vp, _vp, _vp]),
    "ozk_quantize_a": (_i32, [_i64, _i64, _vp, _i64, _vp, _i32, _vp, _vp]),
    "ozk_quantize_b": (_i32, [_i64, _i64, _vp, _i64, _vp, _i32, _vp, _vp]),
    "ozk_residue_gemm": (_i32, [_i64, _i64, _i64, _vp, _vp, _i32, _i32, _vp, _i64, _i32, _vp]),
    "ozk_residue_gemm_withheld": (_i32, [_i64, _i64, _i64, _vp, _vp, _i32, _vp, _i64, _i32, ctypes.c_uint32, _vp]),
    "ozk_crt_combine": (_i32, [_i64, _i64, _i32, _vp, _i32, _i64, _i32, _vp, _vp, _vp, _i64, _vp]),
    "ozk_crt_lift": (_i32, [_i64, _i64, _i32, _vp, _i32, _i64, _i32, _vp, _vp]),
    "ozk_mx4_scale_bytes": (_sz, [_i64, _i64, _i32, _i32]),
    "ozk_mx4_quantize": (_i32, [_i64, _i64, _vp, _i64, _i32, _i32, _f32, _vp, _i32, _vp, _vp, _vp]),
    "ozk_mx4_dequantize": (_i32, [_i64, _i64, _vp, _vp, _i32, _vp, _i32, _vp, _i64, _i32, _vp]),
    "ozk_mx4_gemm": (_i32, [_i64, _i64, _i64, _vp, _vp, _vp, _vp, _i32, _f32, _vp, _i64, _i32, _vp]),
    "ozk_mx4_grouped_gemm": (_i32, [_i64, _i64, _i64, _i32, _vp, _vp, _vp, _vp, _vp, _i32, _f32, _vp, _i64, _i32,
                                    _vp]),
    "ozk_grouped_gemm": (_i32, [_i64, _i64, _i64, _i32, _vp, _vp, _i64, _vp, _i64, _i64, _i32, _vp, _i64, _i32, _vp]),
    "ozk_grouped_gemm_dx": (_i32, [_i64, _i64, _i64, _i32, _vp, _vp, _i64, _vp, _i64, _i64, _i32, _vp, _i64, _i32,
                                   _vp]),
    "ozk_grouped_gemm_dw": (_i32, [_i64, _i64, _i64, _i32, _vp, _vp, _i64, _vp, _i64, _i32, _vp, _i64, _i64, _i32,
                                   _vp]),
    "ozk_mx4_gemv": (_i32, [_i64, _i64, _i64, _i32, _vp, _vp, _i64, _i32, _vp, _vp, _i32, _f32, _vp, _i64, _i32, _vp]),
    "ozk_mx4_gated_gemv": (_i32, [_i64, _i64, _i64, _i32, _vp, _vp, _i64, _i32, _vp, _vp, _i32, _f32, _i32, _vp, _i64,
                                  _i32, _vp]),
    "ozk_grouped_gated_gemm": (_i32, [_i64, _i64, _i64, _i32, _vp, _vp, _i64, _vp, _i64, _i64, _i32, _i32, _vp, _i64, _vp,
                                      _i64, _i64, _vp]),
    "ozk_grouped_gated_gemm_grad": (_i32, [_i64, _i64, _i64, _i32, _vp, _vp, _i64, _vp, _i64, _i64, _vp, _i64, _vp, _i64,
                                           _i64, _i32, _vp, _i64, _vp, _i64, _vp, _i64, _i64, _vp]),
    "ozk_gated_grad": (_i32, [_i64, _i64, _i32, _vp, _vp, _i64, _vp, _i64, _i64, _i32, _vp, _i64, _vp]),
    "ozk_withhold_next_product": (_i32, [_i32, _i32, _i32, ctypes.c_uint32]),
    "ozk_event_create": (_i32, [_vp]),
    "ozk_event_destroy": (_i32, [_vp]),
    "ozk_event_record": (_i32, [_vp, _vp]),
    "ozk_event_elapsed": (_i32, [_vp, _vp, _vp]),
    "ozk_device_sm_count": (_i32, []),
}

class WorkspaceInfo(ctypes.Structure):
    """ozk_workspace_info of include/ozk.h."""
    _fields_ = [("total_bytes", ctypes.c_size_t), ("maxima_offset", ctypes.c_size_t),
                ("s_offset", ctypes.c_size_t), ("t_offset", ctypes.c_size_t),
                ("a_slices_offset", ctypes.c_size_t), ("b_slices_offset", ctypes.c_size_t),
                ("planes_offset", ctypes.c_size_t), ("kpad", ctypes.c_int64), ("a_plane", ctypes.c_int64),
                ("b_plane", ctypes.c_int64), ("planes_kind", ctypes.c_int), ("planes_ld", ctypes.c_int64),
                ("planes_plane", ctypes.c_int64), ("splits", ctypes.c_int)]


_lib = None


class OzkError(RuntimeError):
    def __init__(self, name, status):
        self.status = status
        super().__init__(f"{name} returned {status}: {status_string(status)}")


def lib() -> ctypes.CDLL:
    """The loaded libozk.so.  Raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(
                f"{LIB_PATH} is missing: build it with `python -c 'import __graft_entry__ as g; g.build()'`"
            )
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _lib = L
    return _lib


def status_string(status: int) -> str:
    return lib().ozk_status_string(status).decode()


def _call(name, *args):
    rc = getattr(lib(), name)(*args)
    if rc != OZK_OK:
        raise OzkError(name, rc)
    return rc


# ---------------------------------------------------------------- host helpers
def ozk_moduli(n_moduli: int):
    out = (ctypes.c_int32 * n_moduli)()
    _call("ozk_moduli", n_moduli, ctypes.cast(out, _vp))
    return list(out)


def ozk_beta(K: int, n_moduli: int) -> int:
    return lib().ozk_beta(K, n_moduli)


def ozk_kpad(K: int) -> int:
    return lib().ozk_kpad(K)


def ozk_moduli_for_bits(K: int, target_bits: int) -> int:
    return lib().ozk_moduli_for_bits(K, target_bits)


def ozk_workspace_size(M: int, N: int, K: int, n_moduli: int) -> int:
    return lib().ozk_workspace_size(M, N, K, n_moduli)


# ---------------------------------------------------------------- torch helpers
_DTYPES = {}
_torch = _current_device = _current_stream = _forward_ad = None


def _load_torch():
    global _torch, _current_device, _current_stream, _forward_ad
    import torch
    from torch.autograd import forward_ad

    _DTYPES.update({torch.bfloat16: OZK_BF16, torch.float16: OZK_F16, torch.float32: OZK_F32,
                    torch.float64: OZK_F64})
    lib()
    _current_device, _current_stream = torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream
    _torch, _forward_ad = torch, forward_ad
    return torch


def _stream_at(index, stream):
    """Handle of the given stream, or of the current one, of a device."""
    if stream is None:
        return _current_stream(index)
    if stream.device_index != index:
        raise ValueError(f"operands on cuda:{index}, a stream of cuda:{stream.device_index}")
    return stream.cuda_stream


def _run(name, stream, *args, after=()):
    """The entry point `name` on the device that the tensors among args share
    (its SMs, kernels and status word are the current device's; their addresses
    are passed) and on the given stream or that device's current one; host
    tensors alone: on the stream's device, or the current one.  The stream's
    handle follows args, `after` the handle."""
    torch = _torch or _load_torch()
    index, values = None, []
    for a in args:
        if hasattr(a, "data_ptr"):
            at = a.get_device()
            if at >= 0 and index is None:
                index = at
            elif at >= 0 and at != index:
                raise ValueError(f"{name}: operands on cuda:{index} and cuda:{at}")
            a = a.data_ptr()
        values.append(a)
    if index is None:
        index = torch.cuda.current_device() if stream is None else stream.device_index
    handle = _stream_at(index, stream)
    if _current_device() == index:
        return _call(name, *values, handle, *after)
    with torch.cuda.device(index):
        return _call(name, *values, handle, *after)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    import torch

    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _ld(t):
    """Leading dimension (elements) of a row-major 2-D tensor with unit column stride."""
    if t.dim() != 2 or (t.stride(1) != 1 and t.size(1) > 1):
        raise ValueError("expected a 2-D row-major tensor with unit column stride")
    return max(t.stride(0), t.size(1), 1)


# ---------------------------------------------------------------- the GEMM
def ozk_dgemm(M, N, K, A, lda, B, ldb, C, ldc, n_moduli, stream=None):
    """C-ABI ozk_dgemm on device tensors (A, B, C are torch.float64 CUDA tensors)."""
    return _run("ozk_dgemm", stream, M, N, K, A, lda, B, ldb, C, ldc, n_moduli)


def ozk_dgemm_ws(M, N, K, A, lda, B, ldb, C, ldc, n_moduli, workspace, workspace_bytes, stream=None):
    return _run("ozk_dgemm_ws", stream, M, N, K, A, lda, B, ldb, C, ldc, n_moduli, workspace, workspace_bytes)


def ozk_dgemm_ws_timed(M, N, K, A, lda, B, ldb, C, ldc, n_moduli, workspace, workspace_bytes, events,
                       stream=None):
    ev = (ctypes.c_void_p * 5)(*[e.value for e in events]) if events is not None else None
    return _run("ozk_dgemm_ws_timed", stream, M, N, K, A, lda, B, ldb, C, ldc, n_moduli, workspace, workspace_bytes,
                after=(ctypes.cast(ev, _vp) if ev else None,))


def ozk_dgemm_norm_ws_timed(M, N, K, A, lda, B, ldb, C, ldc, n_moduli, workspace, workspace_bytes, events,
                            stream=None):
    ev = (ctypes.c_void_p * 5)(*[e.value for e in events]) if events is not None else None
    return _run("ozk_dgemm_norm_ws_timed", stream, M, N, K, A, lda, B, ldb, C, ldc, n_moduli, workspace, workspace_bytes,
                after=(ctypes.cast(ev, _vp) if ev else None,))


def ozk_dgemm_host(M, N, K, A, lda, B, ldb, C, ldc, n_moduli, stream=None):
    """Host (CPU, ideally pinned) float64 tensors in and out; synchronous."""
    return _run("ozk_dgemm_host", stream, M, N, K, A, lda, B, ldb, C, ldc, n_moduli)


def ozk_dgemm_host_async(M, N, K, A, lda, B, ldb, C, ldc, n_moduli, stream=None):
    """Host (pinned) float64 tensors; returns once enqueued, C is complete when the stream gets there."""
    return _run("ozk_dgemm_host_async", stream, M, N, K, A, lda, B, ldb, C, ldc, n_moduli)


def ozk_stream_status(stream=None):
    """Status of the given stream and its device, or of the current ones."""
    torch = _torch or _load_torch()
    if stream is None or stream.device_index == _current_device():
        return lib().ozk_stream_status(_stream(stream))
    with torch.cuda.device(stream.device_index):
        return lib().ozk_stream_status(_stream(stream))


def ozk_release_cached():
    return _call("ozk_release_cached")


def dgemm(A, B, n_moduli: int = 14, out=None, stream=None, target_bits=None, scaling="max"):
    """C = A @ B for float64 CUDA tensors through ozk_dgemm (or ozk_dgemm_bits
    when target_bits is given: the moduli count then follows from K; or
    ozk_dgemm_norm with scaling="norm": scales from the rows' 2-norms)."""
    if _torch is None:
        _load_torch()
    M, K = A.shape
    K2, N = B.shape
    if K != K2:
        raise ValueError("inner dimensions differ")
    if out is None:
        out = _empty((M, N), _torch.float64, A.device, stream)
    if scaling == "norm":
        if target_bits is not None:
            raise ValueError("target_bits picks the count of the largest-entry rule")
        ozk_dgemm_norm(M, N, K, A, _ld(A), B, _ld(B), out, _ld(out), n_moduli, stream)
    elif scaling != "max":
        raise ValueError(f"unknown scaling {scaling!r}")
    elif target_bits is None:
        ozk_dgemm(M, N, K, A, _ld(A), B, _ld(B), out, _ld(out), n_moduli, stream)
    else:
        _run("ozk_dgemm_bits", stream, M, N, K, A, _ld(A), B, _ld(B), out, _ld(out), target_bits)
    return out


# ---------------------------------------------------------------- stages
def ozk_scale(M, N, K, A, lda, B, ldb, n_moduli, s, t, scratch, stream=None):
    return _run("ozk_scale", stream, M, N, K, A, lda, B, ldb, n_moduli, s, t, scratch)


def ozk_workspace_layout(M: int, N: int, K: int, n_moduli: int) -> WorkspaceInfo:
    info = WorkspaceInfo()
    _call("ozk_workspace_layout", M, N, K, n_moduli, ctypes.cast(ctypes.pointer(info), _vp))
    return info


def ozk_gamma(K: int, n_moduli: int) -> int:
    return lib().ozk_gamma(K, n_moduli)


def ozk_dgemm_norm(M, N, K, A, lda, B, ldb, C, ldc, n_moduli, stream=None):
    return _run("ozk_dgemm_norm", stream, M, N, K, A, lda, B, ldb, C, ldc, n_moduli)


def ozk_dgemm_norm_ws(M, N, K, A, lda, B, ldb, C, ldc, n_moduli, workspace, workspace_bytes, stream=None):
    return _run("ozk_dgemm_norm_ws", stream, M, N, K, A, lda, B, ldb, C, ldc, n_moduli, workspace, workspace_bytes)


def ozk_scale_norm(M, N, K, A, lda, B, ldb, n_moduli, s, t, scratch, stream=None):
    return _run("ozk_scale_norm", stream, M, N, K, A, lda, B, ldb, n_moduli, s, t, scratch)


def ozk_scale_noalloc(M, N, K, A, lda, B, ldb, n_moduli, s, t, stream=None):
    return _run("ozk_scale_noalloc", stream, M, N, K, A, lda, B, ldb, n_moduli, s, t)


def ozk_quantize_a(M, K, A, lda, s, n_moduli, a_slices, stream=None):
    return _run("ozk_quantize_a", stream, M, K, A, lda, s, n_moduli, a_slices)


def ozk_quantize_b(K, N, B, ldb, t, n_moduli, b_slices, stream=None):
    return _run("ozk_quantize_b", stream, K, N, B, ldb, t, n_moduli, b_slices)


def ozk_residue_gemm(M, N, K, a_slices, b_slices, n_moduli, out_kind, out, ldo, splits, stream=None):
    return _run("ozk_residue_gemm", stream, M, N, K, a_slices, b_slices, n_moduli, out_kind, out, ldo, splits)


def ozk_residue_gemm_withheld(M, N, K, a_slices, b_slices, n_moduli, out, ldo, withhold_kb, timeout_us,
                              stream=None):
    return _run("ozk_residue_gemm_withheld", stream, M, N, K, a_slices, b_slices, n_moduli, out, ldo, withhold_kb,
                timeout_us)


def ozk_withhold_next_product(pairs, cta, kblock, timeout_us):
    return _call("ozk_withhold_next_product", pairs, cta, kblock, timeout_us)


def ozk_crt_combine(M, N, n_moduli, inp, in_kind, ldi, splits, s, t, C, ldc, stream=None):
    return _run("ozk_crt_combine", stream, M, N, n_moduli, inp, in_kind, ldi, splits, s, t, C, ldc)


def ozk_crt_lift(M, N, n_moduli, inp, in_kind, ldi, splits, X, stream=None):
    return _run("ozk_crt_lift", stream, M, N, n_moduli, inp, in_kind, ldi, splits, X)


# ---------------------------------------------------------------- 4-bit matrices and grouped products
# A small call takes a few microseconds on the GPU, so these wrappers do no
# more than check and marshal: pointers go as plain integers, the stream comes
# from the device index, sizes are computed here rather than by another call.
# Every call runs on the device that holds its operands, whichever is current.
_FORMATS = {"nvfp4": OZK_NVFP4, "mxfp4": OZK_MXFP4}
_WORD_COLUMNS = {"nvfp4": 64, "mxfp4": 128}  # columns one word of four scale bytes covers


def _dtype(t):
    """The ozk_dtype of a torch dtype."""
    try:
        return _DTYPES[t]
    except KeyError:
        raise TypeError(f"no ozk_dtype for {t}") from None


def _format(fmt):
    try:
        return _FORMATS[fmt]
    except KeyError:
        raise ValueError(f"unknown 4-bit format {fmt!r} (nvfp4, mxfp4)") from None


def _empty(shape, dtype, device, stream):
    """A new tensor whose memory belongs to the stream that writes it."""
    if stream is None:
        return _torch.empty(shape, dtype=dtype, device=device)
    with _torch.cuda.stream(stream):
        return _torch.empty(shape, dtype=dtype, device=device)


def _result(out, rows, cols, dtype, device, stream):
    """(tensor, leading dimension, ozk_dtype) of a rows x cols result: out, or a new tensor; dtype None: out's own."""
    if out is None:
        kind = _DTYPES.get(dtype)
        if kind is None:
            _dtype(dtype)  # raises
        if stream is None:
            return _torch.empty((rows, cols), dtype=dtype, device=device), cols or 1, kind
        return _empty((rows, cols), dtype, device, stream), cols or 1, kind
    if out.shape != (rows, cols):
        raise ValueError(f"out has shape {tuple(out.shape)}, the result ({rows}, {cols})")
    if dtype is not None and out.dtype != dtype:
        raise TypeError(f"out is {out.dtype}, the result {dtype}")
    if out.device != device:
        raise ValueError(f"out is on {out.device}, the operands on {device}")
    return out, _rows(out)[2], _dtype(out.dtype)


def _device_index(t):
    index = t.get_device()
    if index < 0:
        raise ValueError("expected CUDA tensors")
    return index


def _same_device(index, *tensors):
    for t in tensors:
        if t.get_device() != index:
            raise ValueError(f"operands on cuda:{index} and {t.device}")


def _offsets(offsets, index):
    """The number of groups that offsets, a device vector, has."""
    shape = offsets.shape
    if len(shape) != 1 or shape[0] < 2 or offsets.dtype != _torch.int32 or not offsets.is_contiguous():
        raise TypeError("offsets: a contiguous int32 vector of groups + 1 entries is expected")
    if offsets.get_device() != index:
        raise ValueError(f"operands on cuda:{index} and {offsets.device}")
    return shape[0] - 1


def _one_row(columns):
    """Leading dimension of a single row: nothing is addressed by it, whatever
    the tensor's own stride, and bulk copies want it a multiple of 8."""
    return -(-columns // 8) * 8 or 8


def _rows(t):
    """(rows, columns, leading dimension) of a matrix with unit column stride and rows that do not overlap."""
    shape, stride = t.shape, t.stride()
    if len(shape) != 2:
        raise ValueError("expected a 2-D row-major tensor with unit column stride")
    (r, c), (sr, sc) = shape, stride
    if sc != 1 and c > 1 or r > 1 and sr < c:
        raise ValueError("expected a 2-D row-major tensor with unit column stride, its rows apart (not an expanded one)")
    if r == 1:
        return r, c, _one_row(c)
    return r, c, sr if r > 1 and sr > c else c or 1


def _groups(t):
    """(groups, rows, columns, leading dimension, group stride) of a [groups, rows, columns] tensor with unit column
    stride, rows and groups that do not overlap."""
    shape, stride = t.shape, t.stride()
    if len(shape) != 3:
        raise ValueError("expected a [groups, rows, columns] tensor with unit column stride")
    (g, r, c), (sg, sr, sc) = shape, stride
    if sc != 1 and c > 1:
        raise ValueError("expected a [groups, rows, columns] tensor with unit column stride")
    ld = _one_row(c) if r == 1 else sr if r > 1 and sr > c else c or 1
    if r > 1 and sr < c or g > 1 and sg < (r - 1) * ld + c:
        raise ValueError("rows or groups that overlap")
    return g, r, c, ld, sg if g > 1 else r * ld


class Mx4:
    """A microscaled 4-bit matrix: ``rows`` x ``K`` in ``groups`` groups, its
    ``codes`` and ``scales`` as ozk_mx4_quantize stores them (uint8 tensors),
    ``fmt`` "nvfp4" or "mxfp4"; ``offsets`` where the groups are ragged."""

    __slots__ = ("rows", "K", "fmt", "groups", "offsets", "device", "_memory", "_index", "_codes", "_scales")

    def __init__(self, codes, scales, rows, K, fmt, groups=1, offsets=None):
        if _torch is None:
            _load_torch()
        index = _device_index(codes)
        if offsets is not None:
            groups = _offsets(offsets, index)
        if codes.dtype != _torch.uint8 or scales.dtype != _torch.uint8:
            raise TypeError("codes and scales: uint8 tensors are expected")
        if codes.numel() != rows * (-(-K // 64) * 32) or not codes.is_contiguous():
            raise ValueError("codes: rows x kpad / 2 contiguous bytes are expected")
        if scales.numel() < mx4_scale_bytes(rows, K, fmt, groups) or not scales.is_contiguous():
            raise ValueError("scales: too few bytes, or not contiguous")
        if offsets is None and groups != 1 and rows % groups:
            raise ValueError(f"{rows} rows in {groups} equal groups")
        _same_device(index, scales)
        self.rows, self.K, self.fmt, self.groups, self.offsets = rows, K, fmt, groups, offsets
        self._memory, self._index, self.device = (codes, scales), index, codes.device
        self._codes, self._scales = codes.data_ptr(), scales.data_ptr()

    @property
    def codes(self):
        if isinstance(self._memory, tuple):
            return self._memory[0]
        half = -(-self.K // 64) * 32
        return self._memory[: self.rows * half].view(self.rows, half)

    @property
    def scales(self):
        if isinstance(self._memory, tuple):
            return self._memory[1]
        return self._memory[self._scales - self._codes:]


_new_mx4 = object.__new__


def mx4_scale_bytes(rows: int, K: int, fmt: str = "nvfp4", groups: int = 1) -> int:
    """ozk_mx4_scale_bytes, without the limits on its arguments."""
    if fmt not in _WORD_COLUMNS:
        _format(fmt)
    return (rows // 128 + groups) * -(-(-(-K // 64) * 64) // _WORD_COLUMNS[fmt]) * 512


def mx4_quantize(x, fmt: str = "nvfp4", offsets=None, prescale: float = 1.0, stream=None) -> Mx4:
    """x as a microscaled 4-bit matrix (ozk_mx4_quantize).  x: [rows, K] with
    unit column stride, its rows in ragged groups where offsets (int32, on the
    device) is given; or [groups, rows, K], one group per matrix."""
    torch = _torch or _load_torch()
    groups, f, index, at = 1, _format(fmt), _device_index(x), None
    if offsets is not None:
        groups = _offsets(offsets, index)
        at = offsets.data_ptr()
    if index != _current_device():
        with _torch.cuda.device(index):
            return mx4_quantize(x, fmt, offsets, prescale, stream)
    if len(x.shape) == 3:
        if offsets is not None:
            raise ValueError("offsets are for the rows of a 2-D matrix")
        groups = x.size(0)
        if groups == 0:
            raise ValueError("no groups")
        if x.is_contiguous():
            x = x.view(groups * x.size(1), x.size(2))
        else:  # copied where the call runs
            with torch.cuda.stream(stream):
                x = x.reshape(groups * x.size(1), x.size(2))
    rows, K, ld = _rows(x)
    # codes, then scales, in one allocation
    code_bytes = -(-rows * (-(-K // 64) * 32) // 256) * 256
    size, device = code_bytes + mx4_scale_bytes(rows, K, fmt, groups), x.device
    if stream is None:
        memory = torch.empty(size, dtype=torch.uint8, device=device)
    else:
        memory = _empty(size, torch.uint8, device, stream)
    codes = memory.data_ptr()
    rc = _lib.ozk_mx4_quantize(rows, K, x.data_ptr(), ld, _dtype(x.dtype), f, prescale, at, groups, codes,
                               codes + code_bytes, _stream_at(index, stream))
    if rc:
        raise OzkError("ozk_mx4_quantize", rc)
    q = _new_mx4(Mx4)
    q.rows, q.K, q.fmt, q.groups, q.offsets, q.device = rows, K, fmt, groups, offsets, device
    q._memory, q._index, q._codes, q._scales = memory, index, codes, codes + code_bytes
    return q


def mx4_dequantize(q: Mx4, dtype=None, out=None, stream=None):
    """The values q stands for, [rows, K] of dtype (default float32).  Rows in
    no group are not written."""
    if q._index != _current_device():
        with _torch.cuda.device(q._index):
            return mx4_dequantize(q, dtype, out, stream)
    if dtype is None and out is None:
        dtype = _torch.float32
    out, ld, kind = _result(out, q.rows, q.K, dtype, q.device, stream)
    rc = _lib.ozk_mx4_dequantize(q.rows, q.K, q._codes, q._scales, _FORMATS[q.fmt],
                                 None if q.offsets is None else q.offsets.data_ptr(), q.groups, out.data_ptr(), ld,
                                 kind, _stream_at(q._index, stream))
    if rc:
        raise OzkError("ozk_mx4_dequantize", rc)
    return out


def _no_tangents(name, *tensors):
    """Refuses forward-mode tangents, which would be dropped (with gradients off too: no_grad is for reverse mode alone)."""
    if _forward_ad is None or _forward_ad._current_level < 0:
        return
    for t in tensors:
        if _forward_ad.unpack_dual(t)[1] is not None:
            raise NotImplementedError(f"{name} has no forward-mode derivative, and an operand carries a tangent "
                                      "(forward_ad.unpack_dual(x).primal is without it)")


def _pair_of(a, b):
    if a.fmt != b.fmt or a.K != b.K:
        raise ValueError(f"operands differ: {a.fmt}, K = {a.K} and {b.fmt}, K = {b.K}")
    if a._index != b._index:
        raise ValueError(f"operands on cuda:{a._index} and cuda:{b._index}")


def mx4_gemm(a: Mx4, b: Mx4, alpha: float = 1.0, out_dtype=None, out=None, stream=None):
    """alpha * A @ B^T of two 4-bit matrices of one group each (ozk_mx4_gemm):
    [a.rows, b.rows] of out_dtype (default bfloat16)."""
    _pair_of(a, b)
    if a._index != _current_device():
        with _torch.cuda.device(a._index):
            return mx4_gemm(a, b, alpha, out_dtype, out, stream)
    if a.groups != 1 or b.groups != 1 or a.offsets is not None or b.offsets is not None:
        raise ValueError("matrices of one group are expected; mx4_grouped_gemm takes grouped ones")
    if out_dtype is None and out is None:
        out_dtype = _torch.bfloat16
    out, ld, kind = _result(out, a.rows, b.rows, out_dtype, a.device, stream)
    rc = _lib.ozk_mx4_gemm(a.rows, b.rows, a.K, a._codes, a._scales, b._codes, b._scales, _FORMATS[a.fmt], alpha,
                           out.data_ptr(), ld, kind, _stream_at(a._index, stream))
    if rc:
        raise OzkError("ozk_mx4_gemm", rc)
    return out


def mx4_grouped_gemm(x: Mx4, w: Mx4, alpha: float = 1.0, out_dtype=None, out=None, stream=None):
    """alpha * x_t @ w_g(t)^T (ozk_mx4_grouped_gemm): x quantised with offsets,
    w from a [groups, N, K] tensor; [x.rows, N] of out_dtype (default
    bfloat16).  Rows in no group are not written."""
    _pair_of(x, w)
    if x._index != _current_device():
        with _torch.cuda.device(x._index):
            return mx4_grouped_gemm(x, w, alpha, out_dtype, out, stream)
    if x.offsets is None or w.offsets is not None or x.groups != w.groups:
        raise ValueError("rows quantised with offsets and weights of as many equal groups are expected")
    if out_dtype is None and out is None:
        out_dtype = _torch.bfloat16
    N = w.rows // w.groups
    out, ld, kind = _result(out, x.rows, N, out_dtype, x.device, stream)
    rc = _lib.ozk_mx4_grouped_gemm(x.rows, N, x.K, x.groups, x.offsets.data_ptr(), x._codes, x._scales, w._codes,
                                   w._scales, _FORMATS[x.fmt], alpha, out.data_ptr(), ld, kind,
                                   _stream_at(x._index, stream))
    if rc:
        raise OzkError("ozk_mx4_grouped_gemm", rc)
    return out


_ACTIVATIONS = {"silu": OZK_SILU, "gelu": OZK_GELU, "gelu_tanh": OZK_GELU_TANH}


def _activation(name):
    try:
        return _ACTIVATIONS[name]
    except KeyError:
        raise ValueError(f"unknown activation {name!r} (silu, gelu, gelu_tanh)") from None


def _few_rows(x, w, offsets, act, alpha, out_dtype, out, stream):
    """mx4_gemv and, where act is given, mx4_gated_gemv, which has two rows of w to an output column."""
    if x.requires_grad and out is None and _torch.is_grad_enabled():
        raise NotImplementedError("products with 4-bit weights record no gradient, and x asks for one: "
                                  "x.detach(), no_grad or out says that none is wanted")
    _no_tangents("a product with 4-bit weights", x)
    index, groups, at, per = w._index, w.groups, None, 1 if act is None else 2
    if x.get_device() != index:
        raise ValueError(f"operands on {x.device} and cuda:{index}")
    if w.offsets is not None:
        raise ValueError("weights in equal groups are expected")
    if offsets is not None:
        if _offsets(offsets, index) != groups:
            raise ValueError(f"offsets of {offsets.shape[0] - 1} groups, weights of {groups}")
        at = offsets.data_ptr()
    elif groups != 1:
        raise ValueError(f"offsets are needed for weights of {groups} groups")
    if x.is_contiguous() and len(x.shape) == 2:
        T, K = x.shape
        ldx = K or 1
    else:
        T, K, ldx = _rows(x)
    rows, dtype = w.rows, x.dtype
    N = rows // (groups * per)
    if K != w.K or N * per * groups != rows:
        raise ValueError(f"x is {tuple(x.shape)}, the weights {rows} x {w.K} in {groups} groups")
    kind_x = _DTYPES.get(dtype)
    if kind_x is None:
        _dtype(dtype)  # raises
    if out is None:
        ld, kind = N or 1, kind_x
        if out_dtype is None:
            out_dtype = dtype
        elif out_dtype is not dtype:
            kind = _dtype(out_dtype)
        if stream is None:
            out = _torch.empty((T, N), dtype=out_dtype, device=w.device)
        else:
            out = _empty((T, N), out_dtype, w.device, stream)
    else:
        out, ld, kind = _result(out, T, N, out_dtype, w.device, stream)
    handle = _current_stream(index) if stream is None else _stream_at(index, stream)
    if act is None:
        rc = _lib.ozk_mx4_gemv(T, N, K, groups, at, x.data_ptr(), ldx, kind_x, w._codes, w._scales, _FORMATS[w.fmt], alpha,
                               out.data_ptr(), ld, kind, handle)
    else:
        rc = _lib.ozk_mx4_gated_gemv(T, N, K, groups, at, x.data_ptr(), ldx, kind_x, w._codes, w._scales, _FORMATS[w.fmt],
                                     alpha, act, out.data_ptr(), ld, kind, handle)
    if rc:
        raise OzkError("ozk_mx4_gemv" if act is None else "ozk_mx4_gated_gemv", rc)
    return out


def mx4_gemv(x, w: Mx4, offsets=None, alpha: float = 1.0, out_dtype=None, out=None, stream=None):
    """alpha * x_t @ w_g(t)^T for a few rows of 16-bit x, not quantised
    (ozk_mx4_gemv): x [T, K] bf16 or fp16, w a matrix of one group, or from a
    [groups, N, K] tensor with offsets for the rows of x; [T, N] of out_dtype
    (default x's).  Rows in no group are not written.  No graph is
    recorded: where x asks for a gradient the call is refused, unless under
    no_grad or with out given; so are forward-mode tangents."""
    if w._index != _current_device():
        with _torch.cuda.device(w._index):
            return mx4_gemv(x, w, offsets, alpha, out_dtype, out, stream)
    return _few_rows(x, w, offsets, None, alpha, out_dtype, out, stream)


def mx4_gated_gemv(x, w: Mx4, offsets=None, activation: str = "silu", alpha: float = 1.0, out_dtype=None, out=None,
                   stream=None):
    """act(g) * u for a few rows of 16-bit x (ozk_mx4_gated_gemv): w holds 2 H
    rows per group, the gate's first, g = alpha * x_t @ w_g(t)[:H]^T and u the
    same with w_g(t)[H:]; activation "silu", "gelu" or "gelu_tanh"; [T, H].
    Otherwise as mx4_gemv."""
    if w._index != _current_device():
        with _torch.cuda.device(w._index):
            return mx4_gated_gemv(x, w, offsets, activation, alpha, out_dtype, out, stream)
    return _few_rows(x, w, offsets, _activation(activation), alpha, out_dtype, out, stream)


def _grouped(first, second, offsets, groups):
    """(groups, ozk_dtype, device index) that the operands of a grouped product share."""
    if _torch is None:
        _load_torch()
    kind = first.dtype
    if kind != second.dtype:
        raise TypeError(f"operands of different types: {kind} and {second.dtype}")
    index = _device_index(first)
    if second.get_device() != index:
        raise ValueError(f"operands on cuda:{index} and {second.device}")
    n = _offsets(offsets, index)
    if groups is not None and n != groups:
        raise ValueError(f"offsets of {n} groups, weights of {groups}")
    return n, _dtype(kind), index


def grouped_gemm(x, w, offsets, out_dtype=None, out=None, stream=None):
    """y[t] = x[t] @ w[g(t)]^T (ozk_grouped_gemm): x [T, K], w [groups, N, K] of
    one 16-bit type, offsets int32 [groups + 1] on the device; [T, N] of their
    type or float32.  Rows in no group are not written.

    Autograd records it where x or w asks for a gradient (grouped_gemm_dx and
    grouped_gemm_dw, each only where asked for; zeros for rows in no group; a
    float32 result's gradient is rounded to the operands' type), once: there is
    no second derivative, and forward-mode tangents are refused.  With out
    given, and in every other call here, no graph is recorded."""
    groups, N, K, ldw, stride = _groups(w)
    _, kind, index = _grouped(x, w, offsets, groups)
    if index != _current_device():
        with _torch.cuda.device(index):
            return grouped_gemm(x, w, offsets, out_dtype, out, stream)
    _no_tangents("grouped_gemm", x, w)
    if out is None and (x.requires_grad or w.requires_grad) and _torch.is_grad_enabled():
        with _torch.cuda.stream(stream):
            return (_GroupedGemm or _load_function()).apply(x, w, offsets, out_dtype)
    T, k, ldx = _rows(x)
    if k != K:
        raise ValueError(f"x is {tuple(x.shape)}, the weights {tuple(w.shape)}")
    out, ld, out_kind = _result(out, T, N, out_dtype or (x.dtype if out is None else None), x.device, stream)
    rc = _lib.ozk_grouped_gemm(T, N, K, groups, offsets.data_ptr(), x.data_ptr(), ldx, w.data_ptr(), ldw, stride,
                               kind, out.data_ptr(), ld, out_kind, _stream_at(index, stream))
    if rc:
        raise OzkError("ozk_grouped_gemm", rc)
    return out


def _bulk_rows(t):
    """t, or a copy of it, with rows that bulk copies can read."""
    rows, cols = t.shape
    if t.stride(1) == 1 and t.stride(0) >= cols and t.stride(0) % 8 == 0 and t.data_ptr() % 16 == 0:
        return t
    copy = _torch.empty((rows, -(-cols // 8) * 8), dtype=t.dtype, device=t.device)[:, :cols]
    return copy.copy_(t)


_GroupedGemm = None


def _load_function():
    """The autograd function of grouped_gemm (torch is loaded by now)."""
    global _GroupedGemm

    class GroupedGemm(_torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, w, offsets, out_dtype):
            ctx.save_for_backward(x, w, offsets)
            return grouped_gemm(x, w, offsets, out_dtype)

        @staticmethod
        @_torch.autograd.function.once_differentiable
        def backward(ctx, dy):
            x, w, offsets = ctx.saved_tensors
            dy = _bulk_rows(dy.to(x.dtype))
            dx = dw = None
            if ctx.needs_input_grad[0]:
                dx = grouped_gemm_dx(dy, w, offsets, out=_torch.zeros(x.shape, dtype=x.dtype, device=x.device))
            if ctx.needs_input_grad[1]:
                dw = grouped_gemm_dw(dy, x, offsets)
            return dx, dw, None, None

    _GroupedGemm = GroupedGemm
    return GroupedGemm


def grouped_gemm_dx(dy, w, offsets, out_dtype=None, out=None, stream=None):
    """The gradient of grouped_gemm with respect to x: dx[t] = dy[t] @ w[g(t)], [T, K]."""
    groups, N, K, ldw, stride = _groups(w)
    _, kind, index = _grouped(dy, w, offsets, groups)
    if index != _current_device():
        with _torch.cuda.device(index):
            return grouped_gemm_dx(dy, w, offsets, out_dtype, out, stream)
    T, n, lddy = _rows(dy)
    if n != N:
        raise ValueError(f"dy is {tuple(dy.shape)}, the weights {tuple(w.shape)}")
    out, ld, out_kind = _result(out, T, K, out_dtype or (dy.dtype if out is None else None), dy.device, stream)
    rc = _lib.ozk_grouped_gemm_dx(T, N, K, groups, offsets.data_ptr(), dy.data_ptr(), lddy, w.data_ptr(), ldw,
                                  stride, kind, out.data_ptr(), ld, out_kind, _stream_at(index, stream))
    if rc:
        raise OzkError("ozk_grouped_gemm_dx", rc)
    return out


def grouped_gemm_dw(dy, x, offsets, out_dtype=None, out=None, stream=None):
    """The gradient with respect to w: dw[g] = the sum of dy[t]^T x[t] over the
    rows of group g, [groups, N, K] (zeros for a group without rows)."""
    groups, kind, index = _grouped(dy, x, offsets, None)
    if index != _current_device():
        with _torch.cuda.device(index):
            return grouped_gemm_dw(dy, x, offsets, out_dtype, out, stream)
    (T, N, lddy), (t, K, ldx) = _rows(dy), _rows(x)
    if t != T:
        raise ValueError(f"dy is {tuple(dy.shape)}, x {tuple(x.shape)}")
    if out is None:
        if out_dtype is not None:
            _dtype(out_dtype)
        out = _empty((groups, N, K), out_dtype or x.dtype, x.device, stream)
        ld, stride = K or 1, N * (K or 1)
    else:
        if out.shape != (groups, N, K):
            raise ValueError(f"out has shape {tuple(out.shape)}, the result ({groups}, {N}, {K})")
        if out_dtype is not None and out.dtype != out_dtype:
            raise TypeError(f"out is {out.dtype}, the result {out_dtype}")
        _same_device(index, out)
        ld, stride = _groups(out)[3:]
    rc = _lib.ozk_grouped_gemm_dw(T, N, K, groups, offsets.data_ptr(), dy.data_ptr(), lddy, x.data_ptr(), ldx, kind,
                                  out.data_ptr(), ld, stride, _dtype(out.dtype), _stream_at(index, stream))
    if rc:
        raise OzkError("ozk_grouped_gemm_dw", rc)
    return out


_GatedGemm = None


def _load_gated():
    """The autograd function of grouped_gated_gemm (torch is loaded by now)."""
    global _GatedGemm

    class GatedGemm(_torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, w, offsets, args):
            T, H = args[:2]
            room = -(-H // 4) * 4
            slopes = _torch.empty((2, T, room), dtype=_torch.float32, device=x.device)
            h = _torch.empty((T, H), dtype=x.dtype, device=x.device)
            _gated(args, h.data_ptr(), H or 1, slopes.data_ptr(), room, T * room)
            ctx.save_for_backward(x, w, offsets, slopes if room == H else slopes[:, :, :H])
            return h

        @staticmethod
        @_torch.autograd.function.once_differentiable
        def backward(ctx, dh):
            x, w, offsets, slopes = ctx.saved_tensors
            dx, dw = grouped_gated_gemm_grad(dh, x, w, offsets, slopes, *ctx.needs_input_grad[:2])
            return dx, dw, None, None

    _GatedGemm = GatedGemm
    return GatedGemm


def grouped_gated_gemm(x, w, offsets, activation: str = "silu", out=None, slopes=None, stream=None):
    """h[t] = act(x[t] @ w[g(t)][:H]^T) * (x[t] @ w[g(t)][H:]^T)
    (ozk_grouped_gated_gemm): x [T, K], w [groups, 2 H, K] of one 16-bit type,
    the gate's rows first; activation "silu", "gelu" or "gelu_tanh"; [T, H] of
    their type.  Rows in no group are not written.  slopes, a [2, T, H] float32
    tensor, takes dh/dgate and dh/dup, which gated_grad multiplies a gradient of
    h by.

    Autograd records it where x or w asks for a gradient
    (grouped_gated_gemm_grad), once: there is no second derivative, and
    forward-mode tangents are refused.  With out or slopes given no graph is
    recorded.  Between the passes the slopes are kept, 8 bytes for an element of
    h.  Both passes can be captured into a CUDA graph, together, and only
    while no result of an eager pass from the same leaves is alive: autograd
    would take their gradients to that pass's stream, which ends the capture with
    an error, whatever the function."""
    groups, N, K, ldw, stride = _groups(w)
    _, kind, index = _grouped(x, w, offsets, groups)
    act = _activation(activation)
    if index != _current_device():
        with _torch.cuda.device(index):
            return grouped_gated_gemm(x, w, offsets, activation, out, slopes, stream)
    _no_tangents("grouped_gated_gemm", x, w)
    T, k, ldx = _rows(x)
    if k != K or N % 2:
        raise ValueError(f"x is {tuple(x.shape)}, the weights {tuple(w.shape)}")
    args = (T, N // 2, K, groups, offsets.data_ptr(), x.data_ptr(), ldx, w.data_ptr(), ldw, stride, kind, act,
            _stream_at(index, stream))
    if out is None and slopes is None and (x.requires_grad or w.requires_grad) and _torch.is_grad_enabled():
        function = _GatedGemm or _load_gated()
        if stream is None:
            return function.apply(x, w, offsets, args)
        with _torch.cuda.stream(stream):
            return function.apply(x, w, offsets, args)
    out, ld, _ = _result(out, T, N // 2, x.dtype, x.device, stream)
    at, lds, plane = (None, 0, 0) if slopes is None else _slopes(slopes, T, N // 2, index)
    _gated(args, out.data_ptr(), ld, at, lds, plane)
    return out


def _gated(args, out, ld, slopes, lds, plane):
    rc = _lib.ozk_grouped_gated_gemm(*args[:-1], out, ld, slopes, lds, plane, args[-1])
    if rc:
        raise OzkError("ozk_grouped_gated_gemm", rc)


def _slopes(slopes, T, H, index):
    """(address, leading dimension, stride between the two) of a gated product's slopes."""
    if slopes.shape != (2, T, H):
        raise ValueError(f"slopes have shape {tuple(slopes.shape)}, (2, {T}, {H}) is expected")
    if slopes.dtype != _torch.float32:
        raise TypeError(f"slopes are {slopes.dtype}, float32 is expected")
    _same_device(index, slopes)
    return (slopes.data_ptr(), *_groups(slopes)[3:])


def _plain_rows(t, dtype, stream):
    """(t, leading dimension), t rounded to dtype and laid out in rows where it is not (an expanded gradient)."""
    (rows, cols), (sr, sc) = t.shape, t.stride()
    if t.dtype != dtype or sc != 1 and cols > 1 or sr < cols and rows > 1:
        with _torch.cuda.stream(stream):
            t = t.to(dtype).contiguous()
        return t, cols or 1
    return t, sr if rows > 1 else _one_row(cols)


def gated_grad(dh, slopes, offsets=None, out=None, stream=None):
    """The gradient with respect to a gated product's two projections
    (ozk_gated_grad): dh [T, H], bf16 or fp16, times each of slopes [2, T, H],
    side by side, [T, 2 H] of dh's type.  With it as dy, grouped_gemm_dx and
    grouped_gemm_dw give the gradients of x and w.  With offsets, rows in no
    group are not written."""
    if _torch is None:
        _load_torch()
    index = _device_index(slopes)
    _same_device(index, dh)
    if index != _current_device():
        with _torch.cuda.device(index):
            return gated_grad(dh, slopes, offsets, out, stream)
    groups = 1 if offsets is None else _offsets(offsets, index)
    if len(dh.shape) != 2:
        raise ValueError("expected a 2-D gradient")
    T, H = dh.shape
    at, lds, plane = _slopes(slopes, T, H, index)
    handle = _stream_at(index, stream)
    out, ld, kind = _result(out, T, 2 * H, dh.dtype, slopes.device, stream)
    dh, lddh = _plain_rows(dh, dh.dtype, stream)
    rc = _lib.ozk_gated_grad(T, H, groups, None if offsets is None else offsets.data_ptr(), dh.data_ptr(), lddh, at, lds, plane,
                             kind, out.data_ptr(), ld, handle)
    if rc:
        raise OzkError("ozk_gated_grad", rc)
    return out


def grouped_gated_gemm_grad(dh, x, w, offsets, slopes, need_dx: bool = True, need_dw: bool = True, stream=None):
    """(dx, dw) of grouped_gated_gemm from the gradient of its result and the
    slopes that it kept (ozk_grouped_gated_gemm_grad), both of x's type (dh of
    another type is rounded to it); None for one that is not asked for.  dx is
    zero in rows of no group, dw [groups, 2 H, K] for groups without rows."""
    groups, N, K, ldw, stride = _groups(w)
    _, kind, index = _grouped(x, w, offsets, groups)
    if index != _current_device():
        with _torch.cuda.device(index):
            return grouped_gated_gemm_grad(dh, x, w, offsets, slopes, need_dx, need_dw, stream)
    T, k, ldx = _rows(x)
    if k != K or N % 2:
        raise ValueError(f"x is {tuple(x.shape)}, the weights {tuple(w.shape)}")
    if dh.shape != (T, N // 2):
        raise ValueError(f"the gradient has shape {tuple(dh.shape)}, the result ({T}, {N // 2})")
    _same_device(index, dh)
    at, lds, plane = _slopes(slopes, T, N // 2, index)
    handle, dtype, device = _stream_at(index, stream), x.dtype, x.device
    dh, lddh = _plain_rows(dh, dtype, stream)
    ldp = -(-N // 8) * 8  # rows that bulk copies can read
    dpre = _empty((T, ldp), dtype, device, stream)
    dx = _empty((T, K), dtype, device, stream) if need_dx else None
    dw = _empty((groups, N, K), dtype, device, stream) if need_dw else None
    rc = _lib.ozk_grouped_gated_gemm_grad(
        T, N // 2, K, groups, offsets.data_ptr(), dh.data_ptr(), lddh, at, lds, plane, x.data_ptr(), ldx, w.data_ptr(), ldw,
        stride, kind, dpre.data_ptr(), ldp, dx.data_ptr() if need_dx else None, K or 1, dw.data_ptr() if need_dw else None,
        K or 1, N * (K or 1), handle)
    if rc:
        raise OzkError("ozk_grouped_gated_gemm_grad", rc)
    return dx, dw


# ---------------------------------------------------------------- events
class Event:
    """A CUDA event created by the library (for stage timing)."""

    def __init__(self):
        self.handle = ctypes.c_void_p()
        _call("ozk_event_create", ctypes.byref(self.handle))

    @property
    def value(self):
        return self.handle.value

    def record(self, stream=None):
        _run("ozk_event_record", stream, self.handle)

    def elapsed_ms(self, end: "Event") -> float:
        ms = ctypes.c_float()
        _call("ozk_event_elapsed", self.handle, end.handle, ctypes.byref(ms))
        return ms.value

    def __del__(self):
        try:
            if self.handle and _lib is not None:
                _lib.ozk_event_destroy(self.handle)
        except Exception:
            pass


def sm_count() -> int:
    return lib().ozk_device_sm_count()
