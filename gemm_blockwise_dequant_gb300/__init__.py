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
    "QGAdamWList", "qg_adamw_step", "qg_adamw_step_workspace_bytes", "QG_STATE_F32", "QG_STATE_E4M3", "QG_STATE_BLOCK",
    "qg_token_logprobs", "qg_token_logprobs_grad", "qmoe_route_topk", "qmoe_tokens_fused", "qmoe_tokens_workspace_bytes",
]

QG_OK, QG_ERR_INVALID_ARG, QG_ERR_UNSUPPORTED, QG_ERR_CUDA, QG_ERR_WORKSPACE_TOO_SMALL = 0, 1, 2, 3, 4
QG_F32, QG_F16, QG_BF16 = 0, 1, 2
QG_QMOE_NOALLOC_SCRATCH_BYTES = 1 << 20
QG_WF_U2, QG_WF_U4, QG_WF_U8, QG_WF_E4M3 = 0, 1, 2, 3
QG_STATE_F32, QG_STATE_E4M3, QG_STATE_BLOCK = 0, 1, 256

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


_P, _I, _SZ, _F, _L, _D = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_float, ctypes.c_int64, ctypes.c_double
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
    "qg_adamw_list_init": ([_P, _I, _P], _I),
    "qg_adamw_step_workspace_bytes": ([_L], _SZ),
    "qg_adamw_step": ([_P, _I, _L, _D, _P, _D, _D, _D, _L, _P, _F, _F, _P, _P, _SZ, _P], _I),
    "qg_token_logprobs": ([_P, _I, _L, _P, _I, _I, _F, _P, _P, _P, _I, _P, _P, _P, _P], _I),
    "qg_token_logprobs_grad": ([_P, _I, _L, _P, _P, _P, _P, _P, _F, _P, _L, _I, _I, _P], _I),
    "qmoe_route_topk": ([_P, _I, _L, _I, _I, _I, _I, _P, _P, _P], _I),
    "qmoe_tokens_workspace_bytes": ([_I, _I, _I, _I], _SZ),
    "qmoe_tokens_fused": ([_P, _I, _P, _P, _I, _I, _I, _P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _P, _I, _P, _P, _SZ, _P], _I),
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


def _on_gpu(*tensors):
    """The library takes addresses and works on the current device: one of the host, or of another device, would go unnoticed until a kernel follows it."""
    here = -1
    for t in tensors:
        if t is not None:
            at = t.get_device()
            if at < 0:
                raise ValueError("tensors of a GPU are wanted")
            if at != here:
                if here >= 0:
                    raise ValueError("tensors of one GPU are wanted")
                here = at
    if here >= 0 and here != _torch()._C._cuda_getDevice():
        raise ValueError("tensors of the current device are wanted")


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


class _AdamWTensor(ctypes.Structure):
    _fields_ = [("param", _P), ("grad", _P), ("master", _P), ("exp_avg", _P), ("exp_avg_sq", _P), ("exp_avg_scale", _P),
                ("exp_avg_sq_scale", _P), ("numel", _L), ("first_chunk", _L), ("weight_decay", _F), ("param_dtype", ctypes.c_int32),
                ("grad_dtype", ctypes.c_int32), ("state", ctypes.c_int32)]


class QGAdamWList:
    """The tensors of an optimizer step, for qg_adamw_step: made once, used every step.

    params and grads: one gradient of its size for each parameter, float32/float16/bfloat16 each.  master: float32 copies of
    the parameters, or None (a sequence may hold None for some).  weight_decay: a number, or one for each tensor.

    States: with exp_avg None they are made here, all zero, as `state` says ("f32", or "e4m3": 8 bits and a scale for
    every QG_STATE_BLOCK values; or one of the two for each tensor).  Else the caller's: exp_avg in float32 with
    exp_avg_sq, or in float8_e4m3fn with exp_avg_rms (the root of the second moment) and the float32 scales of both.
    They are attributes of those names afterwards, for saving: lists with None where a tensor has none.

    It holds the tensors, their addresses on the device and a workspace, so it is for buffers that stay where they are
    from step to step, and for one step at a time.
    """

    def __init__(self, params, grads, *, master=None, weight_decay=0.0, state="f32", exp_avg=None, exp_avg_sq=None, exp_avg_scale=None,
                 exp_avg_rms=None, exp_avg_rms_scale=None):
        torch = _torch()
        params = list(params)
        n = len(params)
        each = lambda v, what: [None] * n if v is None else _as_many(list(v), n, what)
        grads, master = _as_many(list(grads), n, "grads"), each(master, "master")
        decay = [float(weight_decay)] * n if isinstance(weight_decay, (int, float)) else _as_many([float(d) for d in weight_decay], n, "weight_decay")
        if exp_avg is None:
            if not (exp_avg_sq is None and exp_avg_scale is None and exp_avg_rms is None and exp_avg_rms_scale is None):
                raise ValueError("states: exp_avg is wanted with them")
            kinds = [state] * n if isinstance(state, str) else _as_many(list(state), n, "state")
            if any(k not in ("f32", "e4m3") for k in kinds):
                raise ValueError("state: f32 or e4m3 is wanted")
            zeros = lambda p, k, dtype, per=1: None if k else torch.zeros(-(-p.numel() // per), dtype=dtype, device=p.device)
            eight = [k == "e4m3" for k in kinds]
            exp_avg = [zeros(p, False, torch.float8_e4m3fn if k else torch.float32) for p, k in zip(params, eight)]
            exp_avg_sq = [zeros(p, k, torch.float32) for p, k in zip(params, eight)]
            exp_avg_rms = [zeros(p, not k, torch.float8_e4m3fn) for p, k in zip(params, eight)]
            exp_avg_scale, exp_avg_rms_scale = ([zeros(p, not k, torch.float32, QG_STATE_BLOCK) for p, k in zip(params, eight)] for _ in range(2))
        exp_avg = _as_many(list(exp_avg), n, "exp_avg")
        exp_avg_sq, exp_avg_rms = each(exp_avg_sq, "exp_avg_sq"), each(exp_avg_rms, "exp_avg_rms")
        exp_avg_scale, exp_avg_rms_scale = each(exp_avg_scale, "exp_avg_scale"), each(exp_avg_rms_scale, "exp_avg_rms_scale")
        host = (_AdamWTensor * max(1, n))()
        for i, (h, p) in enumerate(zip(host, params)):
            m = exp_avg[i]
            eight = m is not None and m.dtype == torch.float8_e4m3fn
            second = exp_avg_rms[i] if eight else exp_avg_sq[i]
            blocks = -(-p.numel() // QG_STATE_BLOCK)
            wanted = [(grads[i], None, p.numel()), (m, torch.float8_e4m3fn if eight else torch.float32, p.numel()),
                      (second, torch.float8_e4m3fn if eight else torch.float32, p.numel())]
            if eight:
                wanted += [(exp_avg_scale[i], torch.float32, blocks), (exp_avg_rms_scale[i], torch.float32, blocks)]
            if master[i] is not None:
                wanted.append((master[i], torch.float32, p.numel()))
            for t, dtype, numel in [(p, None, p.numel())] + wanted:
                if t is None or not t.is_cuda or t.device != params[0].device:
                    raise ValueError("parameters, gradients and states: tensors of one GPU are wanted")
                if not t.is_contiguous() or t.numel() != numel or (dtype is not None and t.dtype != dtype):
                    raise ValueError("gradients, states and master copies: contiguous tensors of the parameter's size are wanted (states in "
                                     "float32, or in float8_e4m3fn with float32 scales)")
            h.param, h.grad, h.master, h.exp_avg, h.exp_avg_sq = p.data_ptr(), grads[i].data_ptr(), _addr(master[i]), m.data_ptr(), second.data_ptr()
            h.exp_avg_scale, h.exp_avg_sq_scale = (_addr(exp_avg_scale[i]), _addr(exp_avg_rms_scale[i])) if eight else (None, None)
            h.numel, h.weight_decay, h.param_dtype, h.grad_dtype = p.numel(), decay[i], _dtype_code(p), _dtype_code(grads[i])
            h.state = QG_STATE_E4M3 if eight else QG_STATE_F32
        chunks = ctypes.c_int64(0)
        _check(lib().qg_adamw_list_init(host, n, ctypes.byref(chunks)), "qg_adamw_list_init")
        self.params, self.grads, self.master, self.count, self.chunks = params, grads, master, n, chunks.value
        self.exp_avg, self.exp_avg_sq, self.exp_avg_scale = exp_avg, exp_avg_sq, exp_avg_scale
        self.exp_avg_rms, self.exp_avg_rms_scale = exp_avg_rms, exp_avg_rms_scale
        device = params[0].device if n else torch.device("cuda", torch.cuda.current_device())
        self.table = torch.frombuffer(bytearray(host), dtype=torch.uint8).to(device)
        self.workspace = torch.empty(lib().qg_adamw_step_workspace_bytes(self.chunks), dtype=torch.uint8, device=device)


def _as_many(v, n, what):
    if len(v) != n:
        raise ValueError("%s: one for each parameter is wanted" % what)
    return v


def qg_adamw_step_workspace_bytes(chunks: int) -> int:
    return lib().qg_adamw_step_workspace_bytes(chunks)


def _device_scalar(t, dtype, what):
    if t.dtype != dtype or t.numel() != 1 or not t.is_cuda:
        raise ValueError("%s: one %s value of a GPU is wanted" % (what, str(dtype).replace("torch.", "")))
    return t.data_ptr()


def qg_adamw_step(tensors, *, lr, step, betas=(0.9, 0.999), eps=1e-8, max_norm=None, norm_eps=1e-6, norm=None, workspace=None, stream=None,
                  raw=False):
    """One AdamW step over the parameters of a QGAdamWList, in place.

    lr: a number or a float32 device tensor of one value; step: 1 for the first one, a number or an int64 device tensor
    of one value (a captured call reads both anew).  max_norm: the gradients enter scaled by min(1, max_norm / (their
    2-norm + norm_eps)), None for no clipping; norm: a float32 device tensor of one value that receives the 2-norm (with
    max_norm), or None.  A norm that is infinite or NaN leaves every tensor as it was.
    """
    torch = _torch()
    if not isinstance(tensors, QGAdamWList):
        raise ValueError("tensors: a QGAdamWList is wanted")
    lr_dev = _device_scalar(lr, torch.float32, "lr") if isinstance(lr, torch.Tensor) else None
    step_dev = _device_scalar(step, torch.int64, "step") if isinstance(step, torch.Tensor) else None
    norm_dev = None if norm is None else _device_scalar(norm, torch.float32, "norm")
    if max_norm is not None and not max_norm >= 0:
        raise ValueError("max_norm: a number that is not negative, or None, is wanted")
    _on_gpu(tensors.table, None if lr_dev is None else lr, None if step_dev is None else step, norm, workspace)
    st, wp, wb, _ = _stream_and_workspace(0, tensors.workspace if workspace is None else workspace, tensors.table, stream)
    if stream is not None:
        tensors.table.record_stream(stream)
        tensors.workspace.record_stream(stream)
    s = lib().qg_adamw_step(tensors.table.data_ptr(), tensors.count, tensors.chunks, 0.0 if lr_dev else float(lr), lr_dev, betas[0], betas[1],
                            eps, 1 if step_dev else int(step), step_dev, -1.0 if max_norm is None else float(max_norm), float(norm_eps),
                            norm_dev, wp, wb, st)
    return s if raw else _check(s, "qg_adamw_step")


# ---------------------------------------------------------------- log probabilities of tokens
def _logits_args(X, targets):
    """rows, vocab, the distance between rows, and the tokens' address."""
    if X.dim() != 2:
        raise ValueError("X: logits [rows, vocab] are wanted")
    T, V = X.shape
    if targets is not None and (targets.dtype != _torch().int64 or targets.shape != (T,) or not targets.is_contiguous()):
        raise ValueError("targets: [rows] int64 is wanted")
    return T, V, _rows2d(X, T, V, "X"), _addr(targets)


def _per_row(t, T, what):
    if t is None:
        return None
    if t.dtype != _torch().float32 or t.shape != (T,) or not t.is_contiguous():
        raise ValueError("%s: [rows] float32 is wanted" % what)
    return t.data_ptr()


def qg_token_logprobs(X, targets, logprob, *, entropy=None, lse=None, top_ids=None, top_logprobs=None, inv_temperature=1.0, status=None,
                      stream=None, raw=False):
    """logprob[t] = log softmax(X[t] * inv_temperature)[targets[t]], with the entropy and log-sum-exp of each row and the
    most probable tokens.

    X: [T, V] float32/float16/bfloat16 logits (rows may lie apart); targets: [T] int64 or None (a negative one: none given
    there, logprob 0); logprob, entropy, lse: [T] float32 or None; top_ids [T, k] int64 and top_logprobs [T, k] float32
    (k up to 64): the k largest logits of each row, the lower index first among equals; status: a device int32 set to 1 by
    a target at or past V, or None.
    """
    T, V, ldx, tp = _logits_args(X, targets)
    torch = _torch()
    k = 0
    if (top_ids is None) != (top_logprobs is None):
        raise ValueError("top_ids and top_logprobs: both or none are wanted")
    if top_ids is not None:
        if top_ids.dim() != 2 or top_ids.shape[0] != T or top_ids.dtype != torch.int64 or top_logprobs.shape != top_ids.shape \
                or top_logprobs.dtype != torch.float32 or not top_ids.is_contiguous() or not top_logprobs.is_contiguous():
            raise ValueError("top_ids [rows, k] int64 and top_logprobs [rows, k] float32 are wanted")
        k = top_ids.shape[1]
    if status is not None and (status.dtype != torch.int32 or status.numel() < 1):
        raise ValueError("status: an int32 is wanted")
    _on_gpu(X, targets, logprob, entropy, lse, top_ids, top_logprobs, status)
    st = torch._C._cuda_getCurrentRawStream(X.get_device()) if stream is None else stream.cuda_stream
    s = lib().qg_token_logprobs(X.data_ptr(), _dtype_code(X), ldx, tp, T, V, inv_temperature, _per_row(logprob, T, "logprob"),
                                _per_row(entropy, T, "entropy"), _per_row(lse, T, "lse"), k, _addr(top_ids), _addr(top_logprobs), _addr(status), st)
    return s if raw else _check(s, "qg_token_logprobs")


def qg_token_logprobs_grad(X, targets, lse, d_logprob, dX, *, entropy=None, d_entropy=None, inv_temperature=1.0, stream=None, raw=False):
    """The gradient of the logits from d_logprob [T] and d_entropy [T] (None: zeros) of qg_token_logprobs, with its lse and
    (beside d_entropy) entropy; dX: [T, V] in X's type, or X itself."""
    T, V, ldx, tp = _logits_args(X, targets)
    lddx = _rows2d(dX, T, V, "dX")
    if dX.dtype != X.dtype:
        raise ValueError("dX: X's type is wanted")
    _on_gpu(X, targets, lse, d_logprob, dX, entropy, d_entropy)
    st = _torch()._C._cuda_getCurrentRawStream(X.get_device()) if stream is None else stream.cuda_stream
    s = lib().qg_token_logprobs_grad(X.data_ptr(), _dtype_code(X), ldx, tp, _per_row(lse, T, "lse"), _per_row(entropy, T, "entropy"),
                                     _per_row(d_logprob, T, "d_logprob"), _per_row(d_entropy, T, "d_entropy"), inv_temperature, dX.data_ptr(), lddx, T, V, st)
    return s if raw else _check(s, "qg_token_logprobs_grad")


# ---------------------------------------------------------------- mixture of experts over a few tokens
def qmoe_route_topk(logits, expert_ids, expert_weights, *, renormalize=True, stream=None, raw=False):
    """The k experts of each token with the largest router logits (the lower index first among equals), and their softmax
    weights over the k (renormalize) or over all experts.

    logits: [T, E] float32/float16/bfloat16 (rows may lie apart); expert_ids: [T, k] int32; expert_weights: [T, k] float32.
    """
    torch = _torch()
    if logits.dim() != 2:
        raise ValueError("logits: [tokens, experts] are wanted")
    T, E = logits.shape
    if expert_ids.dim() != 2 or expert_ids.shape[0] != T or expert_ids.dtype != torch.int32 or expert_weights.shape != expert_ids.shape \
            or expert_weights.dtype != torch.float32 or not expert_ids.is_contiguous() or not expert_weights.is_contiguous():
        raise ValueError("expert_ids [tokens, k] int32 and expert_weights [tokens, k] float32 are wanted")
    _on_gpu(logits, expert_ids, expert_weights)
    st = torch._C._cuda_getCurrentRawStream(logits.get_device()) if stream is None else stream.cuda_stream
    s = lib().qmoe_route_topk(logits.data_ptr(), _dtype_code(logits), _rows2d(logits, T, E, "logits"), T, E, expert_ids.shape[1],
                              1 if renormalize else 0, expert_ids.data_ptr(), expert_weights.data_ptr(), st)
    return s if raw else _check(s, "qmoe_route_topk")


def qmoe_tokens_workspace_bytes(tokens: int, k: int, hidden: int, inter: int) -> int:
    return lib().qmoe_tokens_workspace_bytes(tokens, k, hidden, inter)


def _expert_sizes(w, scales, zp, bias, N, K, bits, block_size, what):
    """The number of experts of a projection [E, N, K]."""
    torch = _torch()
    half = torch.float16
    E = w.shape[0]
    blocks = (E, N, K // block_size if block_size > 0 else 0)
    if w.dtype != torch.uint8 or w.shape != (E, N, K * bits // 8) or not w.is_contiguous():
        raise ValueError("%s_w: [experts, %d, %d] uint8, contiguous, is wanted" % (what, N, K * bits // 8))
    if scales.dtype != half or scales.shape != blocks or not scales.is_contiguous() \
            or zp is not None and (zp.dtype != half or zp.shape != blocks or not zp.is_contiguous()) \
            or bias is not None and (bias.dtype != half or bias.shape != (E, N) or not bias.is_contiguous()):
        raise ValueError("%s: scales and zero points [experts, %d, %d] and biases [experts, %d] in float16, contiguous, are wanted" % (what, N, blocks[2], N))
    return E


def qmoe_tokens_fused(x, expert_ids, expert_weights, *, fc1_w, fc1_scales, fc1_zp, fc1_bias, fc2_w, fc2_scales, fc2_zp, fc2_bias, bits,
                      block_size, y, swiglu_interleaved=0, status=None, workspace=None, stream=None, raw=False):
    """The layer of qmoe_decode_fused over a few tokens, each with k experts of its own; every chosen expert's weights are read once.

    x: [T, hidden] float16/bfloat16; expert_ids [T, k] int32 and expert_weights [T, k] float32 (T * k up to 1024); weights,
    scales, zero points and biases as in qmoe_decode_fused; y: [T, hidden] float32/float16/bfloat16; status: a device int32
    set to 1 by an id that is no expert, or None.
    """
    torch = _torch()
    if x.dim() != 2 or y.shape != x.shape or not x.is_contiguous() or not y.is_contiguous():
        raise ValueError("x and y: [tokens, hidden], contiguous, are wanted")
    T, hidden = x.shape
    if expert_ids.dim() != 2 or expert_ids.shape[0] != T or expert_ids.dtype != torch.int32 or expert_weights.shape != expert_ids.shape \
            or expert_weights.dtype != torch.float32 or not expert_ids.is_contiguous() or not expert_weights.is_contiguous():
        raise ValueError("expert_ids [tokens, k] int32 and expert_weights [tokens, k] float32 are wanted")
    if status is not None and (status.dtype != torch.int32 or status.numel() < 1):
        raise ValueError("status: an int32 is wanted")
    k = expert_ids.shape[1]
    if bits not in (2, 4, 8):
        raise ValueError("bits: 2, 4 or 8 is wanted")
    inter = fc2_w.shape[-1] * 8 // bits
    E = _expert_sizes(fc1_w, fc1_scales, fc1_zp, fc1_bias, 2 * inter, hidden, bits, block_size, "fc1")
    if _expert_sizes(fc2_w, fc2_scales, fc2_zp, fc2_bias, hidden, inter, bits, block_size, "fc2") != E:
        raise ValueError("fc1 and fc2: as many experts in both are wanted")
    _on_gpu(x, expert_ids, expert_weights, y, status, fc1_w, fc1_scales, fc1_zp, fc1_bias, fc2_w, fc2_scales, fc2_zp, fc2_bias, workspace)
    L = lib()
    need = L.qmoe_tokens_workspace_bytes(T, k, hidden, inter) if workspace is None else 0
    st, wp, wb, _ = _stream_and_workspace(need, workspace, x, stream)
    s = L.qmoe_tokens_fused(x.data_ptr(), _dtype_code(x), expert_ids.data_ptr(), expert_weights.data_ptr(), T, k, E, fc1_w.data_ptr(),
                            fc1_scales.data_ptr(), _addr(fc1_zp), _addr(fc1_bias), fc2_w.data_ptr(), fc2_scales.data_ptr(), _addr(fc2_zp),
                            _addr(fc2_bias), hidden, inter, bits, block_size, 1 if swiglu_interleaved else 0, y.data_ptr(), _dtype_code(y), _addr(status), wp, wb, st)
    return s if raw else _check(s, "qmoe_tokens_fused")


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
