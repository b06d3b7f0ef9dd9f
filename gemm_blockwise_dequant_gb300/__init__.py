"""Python binding of libqgemm.so (include/qgemm.h): argument marshalling only.

Every function here has the name of a C entry point, takes torch tensors that
live on the current CUDA device, passes their data pointers and sizes through
ctypes and raises ``QGError`` when the library returns a non-zero status.  All
arithmetic runs in the library's CUDA kernels; there is no fallback.  If the
library has not been built, importing the binding works but the first call
raises ``QGLibraryMissing`` (build it with ``gemm_blockwise_dequant_gb300.build``).

PyTorch provides device memory and streams only.  Workspaces the library asks
for are allocated here, by torch, when the caller does not pass one.
"""
from __future__ import annotations

import ctypes
import os
import threading

__all__ = [
    "QG_OK", "QG_ERR_INVALID_ARG", "QG_ERR_UNSUPPORTED", "QG_ERR_CUDA", "QG_ERR_WORKSPACE_TOO_SMALL",
    "QG_F32", "QG_F16", "QG_BF16", "QGError", "QGLibraryMissing", "lib", "library_path",
    "qgemm_nbits", "qgemm_nbits_uniform_zp", "qgemm_codebook4", "qgemm_workspace_bytes",
    "qmoe_decode_fused", "qmoe_decode_fused_dp4a", "qmoe_decode_fused_noalloc", "qmoe_decode_workspace_bytes", "QG_QMOE_NOALLOC_SCRATCH_BYTES",
    "qg_fp16_uniform_value", "qg_dequant_nbits",
    "qg_dequant_nbits_uniform_zp", "qg_dequant_codebook4", "qg_read_device_fault", "qg_status_string",
    "qgemm_codebook4_nested", "qgemm_codebook4_nested_workspace_bytes", "qmoe_ragged_mm",
    "qmoe_ragged_mm_workspace_bytes", "qg_gather_block_quantized", "QG_WF_U2", "QG_WF_U4", "QG_WF_U8", "QG_WF_E4M3",
    "qgemm_nbits_packed_zp", "qgemm_nbits_packed_zp_workspace_bytes", "qg_test_bounded_wait",
    "qg_test_gemv_plan", "qg_test_cluster_limit", "qmoe_ragged_mm_device_offsets", "qmoe_ragged_mm_device_offsets_workspace_bytes",
    "qg_lora_apply", "qg_lora_apply_workspace_bytes", "qg_lora_grad", "qg_lora_grad_workspace_bytes",
    "qgemm_nbits_dgrad", "qgemm_nbits_uniform_zp_dgrad", "qgemm_codebook4_dgrad", "qgemm_dgrad_workspace_bytes",
    "QGGradList", "qg_clip_grad_norm", "qg_clip_grad_norm_workspace_bytes",
]

QG_OK, QG_ERR_INVALID_ARG, QG_ERR_UNSUPPORTED, QG_ERR_CUDA, QG_ERR_WORKSPACE_TOO_SMALL = 0, 1, 2, 3, 4
QG_F32, QG_F16, QG_BF16 = 0, 1, 2
QG_QMOE_NOALLOC_SCRATCH_BYTES = 1 << 20
QG_WF_U2, QG_WF_U4, QG_WF_U8, QG_WF_E4M3 = 0, 1, 2, 3

_HERE = os.path.dirname(os.path.abspath(__file__))
library_path = os.path.join(_HERE, "libqgemm.so")
_lib = None
_lock = threading.Lock()


class QGError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__("%s returned %s" % (where, _status_name(status)))


class QGLibraryMissing(ImportError):
    pass


def _status_name(s):
    return {0: "QG_OK", 1: "QG_ERR_INVALID_ARG", 2: "QG_ERR_UNSUPPORTED", 3: "QG_ERR_CUDA",
            4: "QG_ERR_WORKSPACE_TOO_SMALL"}.get(s, "status %d" % s)


_P, _I, _SZ, _F, _L = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_float, ctypes.c_int64
_SIGS = {
    "qgemm_nbits": ([_P, _I, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _P, _SZ, _P], _I),
    "qgemm_nbits_uniform_zp": ([_P, _I, _P, _P, _F, _P, _I, _I, _I, _I, _I, _I, _P, _SZ, _P], _I),
    "qgemm_codebook4": ([_P, _I, _P, _P, _P, _P, _I, _I, _I, _I, _I, _P, _SZ, _P], _I),
    "qgemm_workspace_bytes": ([_I, _I, _I, _I, _I, _I], _SZ),
    "qmoe_decode_fused": ([_P, _P, _P, _I, _I, _P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _P, _P, _P, _SZ,
                           _P], _I),
    "qmoe_decode_fused_dp4a": ([_P, _P, _P, _I, _I, _P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _P, _P, _P,
                                _SZ, _P], _I),
    "qmoe_decode_workspace_bytes": ([_I, _I, _I], _SZ),
    "qmoe_decode_fused_noalloc": ([_P, _P, _P, _I, _I, _P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _P, _P,
                                   _P], _I),
    "qg_fp16_uniform_value": ([_P, _SZ, _P, _P, _P, _SZ, _P], _I),
    "qg_dequant_nbits": ([_P, _P, _P, _P, _I, _I, _I, _I, _P], _I),
    "qg_dequant_nbits_uniform_zp": ([_P, _P, _F, _P, _I, _I, _I, _I, _P], _I),
    "qg_dequant_codebook4": ([_P, _P, _P, _P, _I, _I, _I, _P], _I),
    "qg_gather_block_quantized": ([_P, ctypes.c_int64, _P, _I, _P, _P, ctypes.c_int64, _I, _I, _P, _I, _P, _P], _I),
    "qgemm_codebook4_nested": ([_P, _I, _P, _P, _P, _P, _P, _F, _I, _P, _I, _I, _I, _I, _I, _P, _SZ, _P], _I),
    "qgemm_codebook4_nested_workspace_bytes": ([_I, _I, _I, _I, _I], _SZ),
    "qgemm_nbits_packed_zp": ([_P, _I, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _P, _SZ, _P], _I),
    "qgemm_nbits_packed_zp_workspace_bytes": ([_I, _I, _I, _I, _I, _I], _SZ),
    "qmoe_ragged_mm": ([_P, _I, _P, _I, _P, _P, _P, _P, _I, _I, _I, _I, _I, _P, _SZ, _P], _I),
    "qmoe_ragged_mm_workspace_bytes": ([_I, _P, _I, _I, _I, _I, _I], _SZ),
    "qmoe_ragged_mm_device_offsets": ([_P, _I, _P, _I, _I, _P, _P, _P, _P, _I, _I, _I, _I, _I, _P, _SZ, _P, _P], _I),
    "qmoe_ragged_mm_device_offsets_workspace_bytes": ([_I], _SZ),
    "qg_lora_apply_workspace_bytes": ([_I, _I, _I, _I, _I], _SZ),
    "qg_lora_apply": ([_P, _I, _L, _P, _P, _I, _P, _P, _I, _P, _I, _I, _P, _I, _L, _P, _I, _L, _P, _I, _I, _I, _P, _P,
                       _SZ, _P], _I),
    "qg_lora_grad_workspace_bytes": ([_I, _I, _I, _I, _I, _I], _SZ),
    "qg_lora_grad": ([_P, _I, _L, _P, _L, _P, _P, _P, _I, _P, _P, _I, _P, _I, _I, _P, _P, _L, _P, _P, _I, _I, _I, _I,
                      _I, _P, _P, _SZ, _P], _I),
    "qgemm_dgrad_workspace_bytes": ([_I, _I, _I, _I, _I], _SZ),
    "qgemm_nbits_dgrad": ([_P, _I, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _P, _SZ, _P], _I),
    "qgemm_nbits_uniform_zp_dgrad": ([_P, _I, _P, _P, _F, _P, _I, _I, _I, _I, _I, _I, _P, _SZ, _P], _I),
    "qgemm_codebook4_dgrad": ([_P, _I, _P, _P, _P, _P, _I, _I, _I, _I, _I, _P, _SZ, _P], _I),
    "qg_grad_list_init": ([_P, _I, _P], _I),
    "qg_clip_grad_norm_workspace_bytes": ([_L], _SZ),
    "qg_clip_grad_norm": ([_P, _I, _L, _F, _F, _P, _P, _SZ, _P], _I),
    "qg_read_device_fault": ([_P], _I),
    "qg_test_bounded_wait": ([_I, ctypes.c_uint, _P, _P], _I),
    "qg_test_gemv_plan": ([_I, _I, _I, _I, _I, _P], _I),
    "qg_test_cluster_limit": ([_I], _I),
    "qg_status_string": ([_I], ctypes.c_char_p),
}


def lib():
    """The loaded libqgemm.so (raises QGLibraryMissing if it was not built)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(library_path):
                raise QGLibraryMissing("libqgemm.so not built; run gemm_blockwise_dequant_gb300.build.build()")
            L = ctypes.CDLL(library_path)
            for name, (args, res) in _SIGS.items():
                f = getattr(L, name)
                f.argtypes = args
                f.restype = res
            _lib = L
    return _lib


# ---------------------------------------------------------------- marshalling
_TORCH = None


def _torch():
    global _TORCH
    if _TORCH is None:
        import torch

        _TORCH = torch
    return _TORCH


_DTYPE_CODES = None


def _dtype_code(t):
    global _DTYPE_CODES
    if _DTYPE_CODES is None:
        torch = _torch()
        _DTYPE_CODES = {torch.float32: QG_F32, torch.float16: QG_F16, torch.bfloat16: QG_BF16}
    return _DTYPE_CODES[t.dtype]


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    torch = _torch()
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _check(status, where):
    if status != QG_OK:
        raise QGError(status, where)
    return status


def _empty_for(nbytes, device, stream):
    """Scratch memory for one call on `stream` (None: the current one).  Memory of the stream's own: what it held before
    is done with, and whoever gets it next comes later, in that stream's order -- no other stream's."""
    torch = _torch()
    if stream is None:
        return torch.empty(nbytes, dtype=torch.uint8, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(nbytes, dtype=torch.uint8, device=device)


def _workspace(need, workspace, device, stream):
    """(workspace, its size in bytes): the caller's, else a new one of need()
    bytes (None when the call needs none); the library checks the size."""
    if workspace is not None:
        return workspace, workspace.numel() * workspace.element_size()
    nbytes = need()
    if nbytes == 0:
        return None, 0
    return _empty_for(nbytes, device, stream), nbytes


def qgemm_workspace_bytes(a_dtype: int, M: int, N: int, K: int, bits: int, block_size: int) -> int:
    return lib().qgemm_workspace_bytes(a_dtype, M, N, K, bits, block_size)


def qgemm_nbits(A, W, scales, zero_points, Y, *, bits, block_size, workspace=None, stream=None, raw=False):
    """Y[M,N] = A[M,K] . dequant(W)^T with fp16 scales and fp16 zero points (or None).

    A: [M, K] float32/float16/bfloat16; W: [N, K*bits/8] uint8; scales and
    zero_points: [N, K/block_size] float16; Y: [M, N] float32/float16/bfloat16.
    """
    M, K = A.shape
    N = W.shape[0]
    ws, wsb = _workspace(lambda: qgemm_workspace_bytes(_dtype_code(A), M, N, K, bits, block_size), workspace, A.device, stream)
    s = lib().qgemm_nbits(_ptr(A), _dtype_code(A), _ptr(W), _ptr(scales), _ptr(zero_points), _ptr(Y),
                          _dtype_code(Y), M, N, K, bits, block_size, _ptr(ws), wsb, _stream(stream))
    return s if raw else _check(s, "qgemm_nbits")


def qgemm_nbits_uniform_zp(A, W, scales, uniform_zp, Y, *, bits, block_size, workspace=None, stream=None,
                           raw=False):
    """As qgemm_nbits with every zero point equal to the scalar uniform_zp."""
    M, K = A.shape
    N = W.shape[0]
    ws, wsb = _workspace(lambda: qgemm_workspace_bytes(_dtype_code(A), M, N, K, bits, block_size), workspace, A.device, stream)
    s = lib().qgemm_nbits_uniform_zp(_ptr(A), _dtype_code(A), _ptr(W), _ptr(scales), float(uniform_zp), _ptr(Y),
                                     _dtype_code(Y), M, N, K, bits, block_size, _ptr(ws), wsb, _stream(stream))
    return s if raw else _check(s, "qgemm_nbits_uniform_zp")


def qgemm_codebook4(A, W, codebook, absmax, Y, *, block_size, workspace=None, stream=None, raw=False):
    """Y = A . (codebook[q] * absmax)^T; codebook [16] float32, absmax [N, K/block_size] float32."""
    M, K = A.shape
    N = W.shape[0]
    ws, wsb = _workspace(lambda: qgemm_workspace_bytes(_dtype_code(A), M, N, K, 4, block_size), workspace, A.device, stream)
    s = lib().qgemm_codebook4(_ptr(A), _dtype_code(A), _ptr(W), _ptr(codebook), _ptr(absmax), _ptr(Y),
                              _dtype_code(Y), M, N, K, block_size, _ptr(ws), wsb, _stream(stream))
    return s if raw else _check(s, "qgemm_codebook4")


def qmoe_decode_workspace_bytes(k: int, hidden: int, inter: int) -> int:
    return lib().qmoe_decode_workspace_bytes(k, hidden, inter)


def qmoe_decode_fused(x, expert_ids, expert_weights, *, num_experts, fc1_w, fc1_scales, fc1_zp, fc1_bias, fc2_w,
                      fc2_scales, fc2_zp, fc2_bias, bits, block_size, y, swiglu_interleaved=0, status=None,
                      workspace=None, stream=None, raw=False):
    """One-token fused QMoE decode (fc1 -> SwiGLU -> fc2, weighted over the k slots); y [hidden] float16."""
    hidden = x.shape[-1]
    inter = fc2_w.shape[-1] * 8 // bits
    k = expert_ids.numel()
    ws, wsb = _workspace(lambda: qmoe_decode_workspace_bytes(k, hidden, inter), workspace, x.device, stream)
    s = lib().qmoe_decode_fused(_ptr(x), _ptr(expert_ids), _ptr(expert_weights), k, num_experts, _ptr(fc1_w),
                                _ptr(fc1_scales), _ptr(fc1_zp), _ptr(fc1_bias), _ptr(fc2_w), _ptr(fc2_scales),
                                _ptr(fc2_zp), _ptr(fc2_bias), hidden, inter, bits, block_size,
                                int(swiglu_interleaved), _ptr(y), _ptr(status), _ptr(ws), wsb, _stream(stream))
    return s if raw else _check(s, "qmoe_decode_fused")


def qmoe_decode_fused_dp4a(x, expert_ids, expert_weights, *, num_experts, fc1_w, fc1_scales, fc1_zp, fc1_bias,
                           fc2_w, fc2_scales, fc2_zp, fc2_bias, bits, block_size, y, swiglu_interleaved=0,
                           status=None, workspace=None, stream=None, raw=False):
    """qmoe_decode_fused with int8 activations (per-block symmetric quantization, dp4a dot products)."""
    hidden = x.shape[-1]
    inter = fc2_w.shape[-1] * 8 // bits
    k = expert_ids.numel()
    ws, wsb = _workspace(lambda: qmoe_decode_workspace_bytes(k, hidden, inter), workspace, x.device, stream)
    s = lib().qmoe_decode_fused_dp4a(_ptr(x), _ptr(expert_ids), _ptr(expert_weights), k, num_experts, _ptr(fc1_w),
                                     _ptr(fc1_scales), _ptr(fc1_zp), _ptr(fc1_bias), _ptr(fc2_w), _ptr(fc2_scales),
                                     _ptr(fc2_zp), _ptr(fc2_bias), hidden, inter, bits, block_size,
                                     int(swiglu_interleaved), _ptr(y), _ptr(status), _ptr(ws), wsb, _stream(stream))
    return s if raw else _check(s, "qmoe_decode_fused_dp4a")


def qmoe_decode_fused_noalloc(x, expert_ids, expert_weights, *, num_experts, fc1_w, fc1_scales, fc1_zp, fc1_bias,
                              fc2_w, fc2_scales, fc2_zp, fc2_bias, bits, block_size, y, swiglu_interleaved=0,
                              status=None, stream=None, raw=False):
    """qmoe_decode_fused without a workspace: the library's fixed device scratch is used
    (callers that cannot allocate; shapes beyond QG_QMOE_NOALLOC_SCRATCH_BYTES are refused)."""
    hidden = x.shape[-1]
    inter = fc2_w.shape[-1] * 8 // bits
    k = expert_ids.numel()
    s = lib().qmoe_decode_fused_noalloc(_ptr(x), _ptr(expert_ids), _ptr(expert_weights), k, num_experts,
                                        _ptr(fc1_w), _ptr(fc1_scales), _ptr(fc1_zp), _ptr(fc1_bias), _ptr(fc2_w),
                                        _ptr(fc2_scales), _ptr(fc2_zp), _ptr(fc2_bias), hidden, inter, bits,
                                        block_size, int(swiglu_interleaved), _ptr(y), _ptr(status), _stream(stream))
    return s if raw else _check(s, "qmoe_decode_fused_noalloc")


def qg_fp16_uniform_value(t, workspace=None, stream=None):
    """(is_uniform, value) for an fp16 tensor (bitwise equality of all elements)."""
    if workspace is None:
        workspace = _empty_for(16, t.device, stream)
    u = ctypes.c_int(0)
    v = ctypes.c_float(0.0)
    _check(lib().qg_fp16_uniform_value(_ptr(t), t.numel(), ctypes.byref(u), ctypes.byref(v), _ptr(workspace),
                                       workspace.numel(), _stream(stream)), "qg_fp16_uniform_value")
    return bool(u.value), (float(v.value) if u.value else None)


def qg_dequant_nbits(W, scales, zero_points, out, *, bits, block_size, stream=None, raw=False):
    N, K = out.shape
    s = lib().qg_dequant_nbits(_ptr(W), _ptr(scales), _ptr(zero_points), _ptr(out), N, K, bits, block_size,
                               _stream(stream))
    return s if raw else _check(s, "qg_dequant_nbits")


def qg_dequant_nbits_uniform_zp(W, scales, uniform_zp, out, *, bits, block_size, stream=None, raw=False):
    N, K = out.shape
    s = lib().qg_dequant_nbits_uniform_zp(_ptr(W), _ptr(scales), float(uniform_zp), _ptr(out), N, K, bits,
                                          block_size, _stream(stream))
    return s if raw else _check(s, "qg_dequant_nbits_uniform_zp")


def qg_dequant_codebook4(W, codebook, absmax, out, *, block_size, stream=None, raw=False):
    N, K = out.shape
    s = lib().qg_dequant_codebook4(_ptr(W), _ptr(codebook), _ptr(absmax), _ptr(out), N, K, block_size,
                                   _stream(stream))
    return s if raw else _check(s, "qg_dequant_codebook4")


def qgemm_codebook4_nested_workspace_bytes(a_dtype: int, M: int, N: int, K: int, block_size: int) -> int:
    return lib().qgemm_codebook4_nested_workspace_bytes(a_dtype, M, N, K, block_size)


def qgemm_codebook4_nested(A, W, codebook, absmax_q, absmax_table, absmax2, absmax_offset, Y, *, block_size,
                           nested_block=256, workspace=None, stream=None, raw=False):
    """qgemm_codebook4 with a nested absmax: absmax = table[absmax_q] * absmax2[i // nested_block] + offset
    (absmax_q [N, K/block_size] uint8, absmax_table [256] float32, absmax2 float32)."""
    M, K = A.shape
    N = W.shape[0]
    ws, wsb = _workspace(lambda: qgemm_codebook4_nested_workspace_bytes(_dtype_code(A), M, N, K, block_size), workspace,
                         A.device, stream)
    s = lib().qgemm_codebook4_nested(_ptr(A), _dtype_code(A), _ptr(W), _ptr(codebook), _ptr(absmax_q),
                                     _ptr(absmax_table), _ptr(absmax2), float(absmax_offset), nested_block, _ptr(Y),
                                     _dtype_code(Y), M, N, K, block_size, _ptr(ws), wsb, _stream(stream))
    return s if raw else _check(s, "qgemm_codebook4_nested")


def qgemm_nbits_packed_zp_workspace_bytes(a_dtype: int, M: int, N: int, K: int, bits: int, block_size: int) -> int:
    return lib().qgemm_nbits_packed_zp_workspace_bytes(a_dtype, M, N, K, bits, block_size)


def qgemm_nbits_packed_zp(A, W, scales, zero_points_packed, Y, *, bits, block_size, workspace=None, stream=None,
                          raw=False):
    """qgemm_nbits with unsigned integer zero points packed like the codes:
    zero_points_packed [N, ceil((K/block_size)*bits/8)] uint8, field b of a row
    at bit b*bits, least significant bit first."""
    M, K = A.shape
    N = W.shape[0]
    ws, wsb = _workspace(lambda: qgemm_nbits_packed_zp_workspace_bytes(_dtype_code(A), M, N, K, bits, block_size),
                         workspace, A.device, stream)
    s = lib().qgemm_nbits_packed_zp(_ptr(A), _dtype_code(A), _ptr(W), _ptr(scales), _ptr(zero_points_packed),
                                    _ptr(Y), _dtype_code(Y), M, N, K, bits, block_size, _ptr(ws), wsb,
                                    _stream(stream))
    return s if raw else _check(s, "qgemm_nbits_packed_zp")


def _host_offsets(offsets):
    import numpy as np

    off = np.ascontiguousarray(np.asarray(offsets.cpu() if hasattr(offsets, "cpu") else offsets, dtype=np.int64))
    return off, off.ctypes.data_as(ctypes.c_void_p)


def qmoe_ragged_mm_workspace_bytes(x_dtype: int, offsets, N: int, K: int, bits: int, block_size: int) -> int:
    off, p = _host_offsets(offsets)
    return lib().qmoe_ragged_mm_workspace_bytes(x_dtype, p, off.size - 1, N, K, bits, block_size)


def qmoe_ragged_mm(X, offsets, W, scales, zero_points, Y, *, bits, block_size, workspace=None, stream=None,
                   raw=False):
    """Y[r] = X[r] . dequant(W[e])^T for the rows r of expert e (offsets[e] <= r < offsets[e+1]).

    X: [T, K] float32/float16/bfloat16; offsets: host sequence (or CPU tensor) of E+1 ints;
    W: [E, N, K*bits/8] uint8; scales / zero_points: [E, N, K/block_size] float16 (zero_points None
    for the midpoint); Y: [T, N] float32/float16/bfloat16.
    """
    off, p = _host_offsets(offsets)
    E, N = W.shape[0], W.shape[1]
    K = X.shape[1]
    ws, wsb = _workspace(lambda: lib().qmoe_ragged_mm_workspace_bytes(_dtype_code(X), p, E, N, K, bits, block_size),
                         workspace, X.device, stream)
    s = lib().qmoe_ragged_mm(_ptr(X), _dtype_code(X), p, E, _ptr(W), _ptr(scales), _ptr(zero_points), _ptr(Y),
                             _dtype_code(Y), N, K, bits, block_size, _ptr(ws), wsb, _stream(stream))
    return s if raw else _check(s, "qmoe_ragged_mm")


def qmoe_ragged_mm_device_offsets_workspace_bytes(num_experts: int) -> int:
    return lib().qmoe_ragged_mm_device_offsets_workspace_bytes(int(num_experts))


def qmoe_ragged_mm_device_offsets(X, offsets_dev, W, scales, zero_points, Y, *, bits, block_size, status=None,
                                  workspace=None, stream=None, raw=False):
    """qmoe_ragged_mm with the E+1 expert offsets in a device int64 tensor (no host copy).

    X: [max_rows, K] float16/bfloat16 (max_rows >= offsets[E]); Y: [max_rows, N]; rows of Y at or
    past offsets[E] are left untouched; status: a device int32 set to 1 for refused offsets, or None.
    """
    E, N = W.shape[0], W.shape[1]
    max_rows, K = X.shape
    ws, wsb = _workspace(lambda: lib().qmoe_ragged_mm_device_offsets_workspace_bytes(E), workspace, X.device, stream)
    s = lib().qmoe_ragged_mm_device_offsets(_ptr(X), _dtype_code(X), _ptr(offsets_dev), E, max_rows, _ptr(W),
                                            _ptr(scales), _ptr(zero_points), _ptr(Y), _dtype_code(Y), N, K, bits,
                                            block_size, _ptr(ws), wsb, _ptr(status), _stream(stream))
    return s if raw else _check(s, "qmoe_ragged_mm_device_offsets")


def qg_gather_block_quantized(indices, W, scales, zero_points, Y, *, w_format, block_size, status=None, stream=None,
                              raw=False):
    """Y[i] = dequant(table row indices[i]) for a block-quantized [vocab, D] table.

    indices: int64 (any shape; Y is [indices.numel(), D]); W: [vocab, D*bits/8] uint8 codes or
    [vocab, D] E4M3 bytes; scales / zero_points: [vocab, D/block_size] float16 (zero_points None
    for the midpoint, and for E4M3); Y: float32/float16/bfloat16; status: a device int32 or None.
    """
    n, D = Y.shape
    s = lib().qg_gather_block_quantized(_ptr(indices), n, _ptr(W), int(w_format), _ptr(scales), _ptr(zero_points),
                                        W.shape[0], D, block_size, _ptr(Y), _dtype_code(Y), _ptr(status),
                                        _stream(stream))
    return s if raw else _check(s, "qg_gather_block_quantized")


# ---------------------------------------------------------------- adapters and fine-tuning
# These calls take tens of arguments and a few microseconds on the device, so their marshalling is kept short: plain
# integers for addresses (ctypes converts them) and no call of PyTorch's that is not needed.
def _addr(t):
    return None if t is None else t.data_ptr()


def _stream_and_workspace(need, workspace, t, stream):
    """(raw stream, workspace address, its bytes, the workspace): on `stream`, or on the device's current one."""
    raw = _torch()._C._cuda_getCurrentRawStream(t.get_device()) if stream is None else stream.cuda_stream
    if workspace is not None:
        return raw, workspace.data_ptr(), workspace.numel() * workspace.element_size(), workspace
    if not need:
        return raw, None, 0, None
    workspace = _empty_for(need, t.device, stream)
    return raw, workspace.data_ptr(), need, workspace


def _rows2d(t, rows, cols, what):
    """The distance between the rows of a 2-D tensor whose rows are contiguous (the C calls take no other)."""
    ld, step = t.stride() if t.dim() == 2 else (0, 0)
    if t.shape != (rows, cols) or (step != 1 and cols > 1):
        raise ValueError("%s: a tensor of %d rows of %d contiguous values is wanted" % (what, rows, cols))
    return ld if rows > 1 else cols  # the stride of a single row says nothing


def _adapter_sizes(A, B, scaling, seg_offsets, seg_adapter, status):
    torch = _torch()
    if status is not None and (status.dtype != torch.int32 or status.numel() < 1):
        raise ValueError("status: an int32 is wanted")
    na, r, K = A.shape
    N = B.shape[1]
    if B.shape != (na, N, r) or A.dtype != B.dtype or not A.is_contiguous() or not B.is_contiguous():
        raise ValueError("A [adapters, rank, K] and B [adapters, N, rank] of one type, contiguous, are wanted")
    if scaling is not None and (scaling.dtype != torch.float32 or scaling.shape != (na,) or not scaling.is_contiguous()):
        raise ValueError("scaling: [adapters] float32 is wanted")
    S = seg_adapter.numel()
    if seg_offsets.numel() != S + 1 or seg_offsets.dtype != torch.int64 or seg_adapter.dtype != torch.int32 \
            or not seg_offsets.is_contiguous() or not seg_adapter.is_contiguous():
        raise ValueError("seg_offsets [requests + 1] int64 and seg_adapter [requests] int32 are wanted")
    return na, r, K, N, S


def qg_lora_apply_workspace_bytes(rows: int, num_segments: int, rank: int, N: int, K: int) -> int:
    return lib().qg_lora_apply_workspace_bytes(rows, num_segments, rank, N, K)


def qg_lora_apply(X, seg_offsets, seg_adapter, A, B, scaling, Y_in, Y, *, V=None, status=None, workspace=None,
                  stream=None, raw=False):
    """Y[t] = Y_in[t] + scaling[a] (X[t] A[a]^T) B[a]^T for the rows t of each request, a the request's adapter.

    X: [T, K]; seg_offsets: [S + 1] int64 and seg_adapter: [S] int32, both on the device (request i owns rows
    seg_offsets[i] .. seg_offsets[i+1]-1; a negative adapter means none); A: [adapters, rank, K]; B: [adapters, N,
    rank]; scaling: [adapters] float32 or None (1); Y_in: [T, N] in float32 or Y's type, None (zeros) or Y itself;
    Y: [T, N]; V: [T, rank] float32 that receives X A^T for qg_lora_grad, or None; status: a device int32 or None.
    X, Y_in and Y may be column slices (rows apart, values contiguous).
    """
    na, r, K, N, S = _adapter_sizes(A, B, scaling, seg_offsets, seg_adapter, status)
    T = X.shape[0]
    ldx, ldy = _rows2d(X, T, K, "X"), _rows2d(Y, T, N, "Y")
    yin = (None, 0, 0) if Y_in is None else (Y_in.data_ptr(), _dtype_code(Y_in), _rows2d(Y_in, T, N, "Y_in"))
    if V is not None and (V.shape != (T, r) or V.dtype != _torch().float32 or not V.is_contiguous()):
        raise ValueError("V: [rows, rank] float32 is wanted")
    L = lib()
    need = L.qg_lora_apply_workspace_bytes(T, S, r, N, K) if workspace is None else 0
    st, wp, wb, _ = _stream_and_workspace(need, workspace, X, stream)
    s = L.qg_lora_apply(X.data_ptr(), _dtype_code(X), ldx, seg_offsets.data_ptr(), seg_adapter.data_ptr(), S, A.data_ptr(),
                        B.data_ptr(), _dtype_code(A), _addr(scaling), na, r, yin[0], yin[1], yin[2], Y.data_ptr(),
                        _dtype_code(Y), ldy, _addr(V), T, N, K, _addr(status), wp, wb, st)
    return s if raw else _check(s, "qg_lora_apply")


def qg_lora_grad_workspace_bytes(rows: int, num_segments: int, num_adapters: int, rank: int, N: int, K: int) -> int:
    return lib().qg_lora_grad_workspace_bytes(rows, num_segments, num_adapters, rank, N, K)


def qg_lora_grad(dY, X, V, seg_offsets, seg_adapter, A, B, scaling, dX_in, dX, dA, dB, *, accumulate=False, status=None,
                 workspace=None, stream=None, raw=False):
    """The backward pass of qg_lora_apply: dX = dX_in + G A with G = scaling dY B, dA = G^T X, dB = scaling dY^T V.

    dY: [T, N] and X: [T, K] of one type; V: [T, rank] float32 from qg_lora_apply; dX_in and dX: [T, K] in X's type
    (dX_in None for zeros or dX itself; dX None when no gradient of X is wanted); dA and dB: shapes of A and B, in
    their type or float32, zero for adapters without rows (accumulate: added to what they hold).
    """
    na, r, K, N, S = _adapter_sizes(A, B, scaling, seg_offsets, seg_adapter, status)
    T = X.shape[0]
    xt = X.dtype
    if dY.dtype != xt or V.shape != (T, r) or V.dtype != _torch().float32 or not V.is_contiguous():
        raise ValueError("dY of X's type and V [rows, rank] float32 are wanted")
    if dA.shape != A.shape or dB.shape != B.shape or dA.dtype != dB.dtype or not dA.is_contiguous() or not dB.is_contiguous():
        raise ValueError("dA and dB: the shapes of A and B, contiguous and of one type, are wanted")
    lddy, ldx, lddx = _rows2d(dY, T, N, "dY"), _rows2d(X, T, K, "X"), 0
    if dX is not None:
        lddx = _rows2d(dX, T, K, "dX")
        if dX.dtype != xt or (dX_in is not None and (dX_in.dtype != xt or _rows2d(dX_in, T, K, "dX_in") != lddx)):
            raise ValueError("dX_in and dX: X's type, and one distance between rows, are wanted")
    L = lib()
    need = L.qg_lora_grad_workspace_bytes(T, S, na, r, N, K) if workspace is None else 0
    st, wp, wb, _ = _stream_and_workspace(need, workspace, X, stream)
    s = L.qg_lora_grad(dY.data_ptr(), _dtype_code(X), lddy, X.data_ptr(), ldx, V.data_ptr(), seg_offsets.data_ptr(),
                       seg_adapter.data_ptr(), S, A.data_ptr(), B.data_ptr(), _dtype_code(A), _addr(scaling), na, r,
                       _addr(dX_in), _addr(dX), lddx, dA.data_ptr(), dB.data_ptr(), _dtype_code(dA), 1 if accumulate else 0,
                       T, N, K, _addr(status), wp, wb, st)
    return s if raw else _check(s, "qg_lora_grad")


def qgemm_dgrad_workspace_bytes(dy_dtype: int, M: int, N: int, K: int, bits: int) -> int:
    return lib().qgemm_dgrad_workspace_bytes(dy_dtype, M, N, K, bits)


def _dgrad_sizes(dY, W, params, table, dX, bits, block_size, codebook=False):
    """M, N, K; table: the zero points [N, K/block_size] or None, or the codebook [16]."""
    torch = _torch()
    (M, N), (mx, K), (nw, wb), (np, nb) = dY.shape, dX.shape, W.shape, params.shape
    if mx != M or nw != N or np != N or wb != K * bits // 8 or (block_size > 0 and nb != K // block_size) or not dY.is_contiguous() \
            or not dX.is_contiguous() or not W.is_contiguous() or not params.is_contiguous():
        raise ValueError("dY [M, N], W [N, K*bits/8], parameters [N, K/block_size] and dX [M, K], contiguous, are wanted")
    wanted = torch.float32 if codebook else torch.float16
    if W.dtype != torch.uint8 or params.dtype != wanted:
        raise ValueError("W in uint8 and %s are wanted" % ("absmax in float32" if codebook else "scales in float16"))
    if table is not None and (table.dtype != wanted or not table.is_contiguous() or (table.numel() != 16 if codebook else table.shape != (N, nb))):
        raise ValueError("the codebook [16] in float32, or zero points in the scales' shape and type, contiguous, are wanted")
    return M, N, K


def qgemm_nbits_dgrad(dY, W, scales, zero_points, dX, *, bits, block_size, workspace=None, stream=None, raw=False):
    """dX[M,K] = dY[M,N] . dequant(W)[N,K]: the gradient of the activations through the frozen weight of qgemm_nbits."""
    M, N, K = _dgrad_sizes(dY, W, scales, zero_points, dX, bits, block_size)
    L = lib()
    need = L.qgemm_dgrad_workspace_bytes(_dtype_code(dY), M, N, K, bits) if workspace is None else 0
    st, wp, wb, _ = _stream_and_workspace(need, workspace, dY, stream)
    s = L.qgemm_nbits_dgrad(_addr(dY), _dtype_code(dY), _addr(W), _addr(scales), _addr(zero_points), _addr(dX),
                            _dtype_code(dX), M, N, K, bits, block_size, wp, wb, st)
    return s if raw else _check(s, "qgemm_nbits_dgrad")


def qgemm_nbits_uniform_zp_dgrad(dY, W, scales, uniform_zp, dX, *, bits, block_size, workspace=None, stream=None, raw=False):
    """As qgemm_nbits_dgrad with every zero point equal to the scalar uniform_zp."""
    M, N, K = _dgrad_sizes(dY, W, scales, None, dX, bits, block_size)
    L = lib()
    need = L.qgemm_dgrad_workspace_bytes(_dtype_code(dY), M, N, K, bits) if workspace is None else 0
    st, wp, wb, _ = _stream_and_workspace(need, workspace, dY, stream)
    s = L.qgemm_nbits_uniform_zp_dgrad(_addr(dY), _dtype_code(dY), _addr(W), _addr(scales), float(uniform_zp), _addr(dX),
                                       _dtype_code(dX), M, N, K, bits, block_size, wp, wb, st)
    return s if raw else _check(s, "qgemm_nbits_uniform_zp_dgrad")


def qgemm_codebook4_dgrad(dY, W, codebook, absmax, dX, *, block_size, workspace=None, stream=None, raw=False):
    """dX = dY . (codebook[q] * absmax): the gradient of the activations through the frozen weight of qgemm_codebook4."""
    M, N, K = _dgrad_sizes(dY, W, absmax, codebook, dX, 4, block_size, codebook=True)
    L = lib()
    need = L.qgemm_dgrad_workspace_bytes(_dtype_code(dY), M, N, K, 4) if workspace is None else 0
    st, wp, wb, _ = _stream_and_workspace(need, workspace, dY, stream)
    s = L.qgemm_codebook4_dgrad(_addr(dY), _dtype_code(dY), _addr(W), _addr(codebook), _addr(absmax), _addr(dX),
                                _dtype_code(dX), M, N, K, block_size, wp, wb, st)
    return s if raw else _check(s, "qgemm_codebook4_dgrad")


class _GradTensor(ctypes.Structure):
    _fields_ = [("grad", _P), ("out", _P), ("numel", _L), ("first_chunk", _L), ("dtype", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


class QGGradList:
    """The gradient tensors of a step, for qg_clip_grad_norm: made once, used every step.

    It holds the tensors, their addresses on the device and a workspace, so it is for buffers that stay where they
    are from step to step, and for one step at a time.  outs: where the clipped gradients go, each of its gradient's size and type (default: in place).
    """

    def __init__(self, grads, outs=None):
        torch = _torch()
        grads = list(grads)
        outs = grads if outs is None else list(outs)
        if len(outs) != len(grads):
            raise ValueError("outs: one for each gradient is wanted")
        host = (_GradTensor * max(1, len(grads)))()
        for h, g, o in zip(host, grads, outs):
            if not g.is_cuda or not o.is_cuda:
                raise ValueError("gradients and outs: tensors of a GPU are wanted")
            if not g.is_contiguous() or not o.is_contiguous() or g.numel() != o.numel() or g.dtype != o.dtype:
                raise ValueError("gradients and outs: contiguous tensors of one size and type are wanted")
            h.grad, h.out, h.numel, h.dtype = g.data_ptr(), o.data_ptr(), g.numel(), _dtype_code(g)
        chunks = ctypes.c_int64(0)
        _check(lib().qg_grad_list_init(host, len(grads), ctypes.byref(chunks)), "qg_grad_list_init")
        self.grads, self.outs, self.count, self.chunks = grads, outs, len(grads), chunks.value
        device = grads[0].device if grads else torch.device("cuda", torch.cuda.current_device())
        self.table = torch.frombuffer(bytearray(host), dtype=torch.uint8).to(device)
        self.workspace = torch.empty(lib().qg_clip_grad_norm_workspace_bytes(self.chunks), dtype=torch.uint8, device=device)


def qg_clip_grad_norm_workspace_bytes(chunks: int) -> int:
    return lib().qg_clip_grad_norm_workspace_bytes(chunks)


def qg_clip_grad_norm(grads, max_norm, norm, *, eps=1e-6, workspace=None, stream=None, raw=False):
    """norm = the 2-norm over all gradients; each out = its gradient * min(1, max_norm / (norm + eps)).

    grads: a QGGradList, or a sequence of tensors (clipped in place; the list is then laid out in every call);
    norm: a float32 device tensor of one value.
    """
    if norm.dtype != _torch().float32 or norm.numel() != 1 or not norm.is_cuda:
        raise ValueError("norm: one float32 value of a GPU is wanted")
    if not isinstance(grads, QGGradList):
        grads = QGGradList(grads)
    st, wp, wb, _ = _stream_and_workspace(0, grads.workspace if workspace is None else workspace, grads.table, stream)
    if stream is not None:
        grads.table.record_stream(stream)
        grads.workspace.record_stream(stream)
    s = lib().qg_clip_grad_norm(_addr(grads.table), grads.count, grads.chunks, float(max_norm), float(eps), _addr(norm), wp,
                                wb, st)
    return s if raw else _check(s, "qg_clip_grad_norm")


def qg_read_device_fault() -> int:
    v = ctypes.c_uint(0)
    _check(lib().qg_read_device_fault(ctypes.byref(v)), "qg_read_device_fault")
    return int(v.value)


def qg_test_bounded_wait(fill: bool, limit_us: int, out, stream=None, raw=False):
    """Test hook (include/qgemm_testing.h): the library's bounded pipeline wait
    in a one-CTA kernel whose producer fills the stage only if `fill`; out is a
    device int32 tensor of 3 (1: that consumer warp's wait completed, 0: it
    gave up)."""
    s = lib().qg_test_bounded_wait(1 if fill else 0, int(limit_us), _ptr(out), _stream(stream))
    return s if raw else _check(s, "qg_test_bounded_wait")


def qg_test_gemv_plan(M: int, N: int, K: int, a_dtype: int = QG_F32, zp_mode: int = 2):
    """Test hook (include/qgemm_testing.h): the launch plan of the 2-bit
    tensor-core GEMV for this shape -- a dict of rows_per_tile, warps (consumer
    warps), ctas, stages -- or None when the shape takes another path."""
    out = (ctypes.c_int * 4)()
    s = lib().qg_test_gemv_plan(int(M), int(N), int(K), int(a_dtype), int(zp_mode), ctypes.cast(out, ctypes.c_void_p))
    if s == QG_ERR_UNSUPPORTED:
        return None
    _check(s, "qg_test_gemv_plan")
    return dict(zip(("rows_per_tile", "warps", "ctas", "stages"), list(out)))


def qg_test_cluster_limit(widest: int) -> int:
    """Test hook (include/qgemm_testing.h): the widest cluster of the adapter and activation-gradient launches of few
    rows (1, 2, 4, 8 or 16) from now on; returns the limit before."""
    before = lib().qg_test_cluster_limit(int(widest))
    if before == 0:
        raise ValueError("a power of two up to 16 is wanted")
    return before


def qg_status_string(status: int) -> str:
    return lib().qg_status_string(status).decode()
