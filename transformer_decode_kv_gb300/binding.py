"""Thin ctypes binding of libllm (include/llm.h): argument marshalling only.

Every step of the decode path runs inside the library's CUDA kernels; this module only converts
Python/numpy/torch arguments into the C structs and pointers the C ABI takes. Importing it when
libllm.so has not been built raises an error: there is no fallback implementation.
"""
from __future__ import annotations

import ctypes as C
import os
from typing import Iterable, Optional, Sequence

import numpy as np

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libllm.so")

F32, F16, BF16, Q8_0, F8_E4M3, F4_E2M1 = 0, 1, 2, 8, 100, 101
CTX_HOST_ONLY = 1
CTX_FUSED_STEP = 2
CTX_KV_SPLIT = 4


class HParams(C.Structure):
    _fields_ = [("n_layer", C.c_int32), ("n_embd", C.c_int32), ("n_head", C.c_int32),
                ("n_head_kv", C.c_int32), ("head_dim", C.c_int32), ("n_ff", C.c_int32),
                ("n_vocab", C.c_int32), ("rope_freq_base", C.c_float), ("rms_eps", C.c_float),
                ("rope_type", C.c_int32)]


class CParams(C.Structure):
    _fields_ = [("n_ctx", C.c_uint32), ("n_seq_max", C.c_uint32), ("n_batch", C.c_uint32),
                ("n_ubatch", C.c_uint32), ("type_k", C.c_int32), ("type_v", C.c_int32),
                ("stream", C.c_void_p), ("flags", C.c_uint32)]


class Batch(C.Structure):
    _fields_ = [("n_tokens", C.c_int32), ("token", C.POINTER(C.c_int32)),
                ("pos", C.POINTER(C.c_int32)), ("n_seq_id", C.POINTER(C.c_int32)),
                ("seq_id", C.POINTER(C.POINTER(C.c_int32))), ("logits", C.POINTER(C.c_int8))]


class SamplerParams(C.Structure):
    _fields_ = [("top_k", C.c_int32), ("top_p", C.c_float), ("min_p", C.c_float),
                ("temperature", C.c_float), ("repeat_penalty", C.c_float),
                ("penalty_tokens", C.POINTER(C.c_int32)), ("n_penalty_tokens", C.c_int32)]


class KvPagesDesc(C.Structure):
    _fields_ = [("type", C.c_int32), ("n_head_kv", C.c_int32), ("head_dim", C.c_int32),
                ("page_size", C.c_int32), ("n_pages", C.c_int32),
                ("k", C.c_void_p), ("v", C.c_void_p),
                ("stride_page", C.c_int64), ("stride_cell", C.c_int64), ("stride_head", C.c_int64),
                ("k_scale", C.c_void_p), ("v_scale", C.c_void_p),
                ("sstride_page", C.c_int64), ("sstride_cell", C.c_int64),
                ("sstride_head", C.c_int64), ("k_block", C.c_void_p), ("v_block", C.c_void_p),
                ("bstride_page", C.c_int64), ("bstride_cell", C.c_int64),
                ("bstride_head", C.c_int64)]


class SeqPagesDesc(C.Structure):
    _fields_ = [("n_seq", C.c_int32), ("page_size", C.c_int32), ("n_pages", C.c_int32),
                ("ld_table", C.c_int32), ("max_free", C.c_int32),
                ("table", C.c_void_p), ("n_kv", C.c_void_p), ("free_pages", C.c_void_p),
                ("n_free", C.c_void_p)]


class AttnShape(C.Structure):
    _fields_ = [("type", C.c_int32), ("n_head", C.c_int32), ("scale", C.c_float),
                ("window", C.c_int32), ("n_sink", C.c_int32), ("max_tok", C.c_int32),
                ("max_seq", C.c_int32), ("max_table", C.c_int32)]


class SampleRowsArgs(C.Structure):
    _fields_ = [("type", C.c_int32), ("n_rows", C.c_int32), ("n_vocab", C.c_int32),
                ("logits", C.c_void_p), ("ld", C.c_int64), ("top_k", C.c_void_p),
                ("top_p", C.c_void_p), ("min_p", C.c_void_p), ("temperature", C.c_void_p),
                ("u", C.c_void_p), ("repeat_penalty", C.c_void_p), ("penalty_start", C.c_void_p),
                ("penalty_token", C.c_void_p), ("n_penalty_token", C.c_int32),
                ("token", C.c_void_p)]


class PerfData(C.Structure):
    _fields_ = [("n_decode_calls", C.c_int64), ("n_tokens", C.c_int64), ("n_ubatches", C.c_int64),
                ("n_graph_replays", C.c_int64), ("t_decode_ms", C.c_double),
                ("n_fused_steps", C.c_int64), ("n_defrags", C.c_int64),
                ("weight_device_bytes", C.c_int64)]


ABORT_CB = C.CFUNCTYPE(C.c_int, C.c_void_p)

# every symbol include/llm.h declares, with (restype, argtypes)
SIGNATURES = {
    "llm_cparams_default": (CParams, []),
    "llm_ctx_init": (C.c_void_p, [C.POINTER(HParams), C.POINTER(CParams)]),
    "llm_ctx_free": (None, [C.c_void_p]),
    "llm_load_weights": (C.c_int, [C.c_void_p, C.c_char_p, C.c_int32, C.POINTER(C.c_int64),
                                   C.c_void_p, C.c_size_t]),
    "llm_weights_ready": (C.c_int, [C.c_void_p]),
    "llm_decode": (C.c_int32, [C.c_void_p, Batch]),
    "llm_get_logits_ith": (C.POINTER(C.c_float), [C.c_void_p, C.c_int32]),
    "llm_get_argmax_ith": (C.c_int32, [C.c_void_p, C.c_int32]),
    "llm_n_outputs": (C.c_int32, [C.c_void_p]),
    "llm_seq_rm": (C.c_int, [C.c_void_p, C.c_int32, C.c_int32, C.c_int32]),
    "llm_seq_pos_max": (C.c_int32, [C.c_void_p, C.c_int32]),
    "llm_seq_pos_min": (C.c_int32, [C.c_void_p, C.c_int32]),
    "llm_set_abort_callback": (None, [C.c_void_p, ABORT_CB, C.c_void_p]),
    "llm_n_ctx": (C.c_uint32, [C.c_void_p]),
    "llm_n_ctx_seq": (C.c_uint32, [C.c_void_p]),
    "llm_n_batch": (C.c_uint32, [C.c_void_p]),
    "llm_n_ubatch": (C.c_uint32, [C.c_void_p]),
    "llm_kv_used_cells": (C.c_int32, [C.c_void_p]),
    "llm_last_error": (C.c_char_p, [C.c_void_p]),
    "llm_perf": (None, [C.c_void_p, C.POINTER(PerfData)]),
    "llm_debug_last_slots": (C.c_int32, [C.c_void_p, C.POINTER(C.c_int32), C.c_int32]),
    "llm_debug_ubatch_mask": (C.c_int64, [C.c_void_p, C.c_int32, C.POINTER(C.c_uint8), C.c_int64,
                                          C.POINTER(C.c_int32)]),
    "llm_debug_capture": (C.c_int, [C.c_void_p, C.c_int]),
    "llm_debug_get_tensor": (C.c_int64, [C.c_void_p, C.c_char_p, C.c_int32,
                                         C.POINTER(C.c_float), C.c_int64]),
    "llm_debug_inject_fault": (C.c_int, [C.c_void_p, C.c_int32, C.c_int32]),
    "llm_debug_kv_raw": (C.c_int64, [C.c_void_p, C.c_int32, C.c_int32, C.c_void_p, C.c_int64]),
    "llm_memory_update": (C.c_int, [C.c_void_p, C.c_int]),
    "llm_sample_ith": (C.c_int32, [C.c_void_p, C.c_int32, C.POINTER(SamplerParams), C.c_float]),
    "llm_debug_set_logits": (C.c_int, [C.c_void_p, C.c_int32, C.POINTER(C.c_float)]),
    "llm_debug_step_trace_enable": (C.c_int, [C.c_void_p, C.c_int]),
    "llm_debug_step_trace": (C.c_int64, [C.c_void_p, C.POINTER(C.c_uint64), C.c_int64,
                                         C.POINTER(C.c_int32), C.POINTER(C.c_int32)]),
    "llm_debug_kernel_timing": (C.c_int, [C.c_void_p, C.c_int]),
    "llm_gemm_bf16_noalloc": (C.c_int, [C.c_int32, C.c_void_p, C.c_int64, C.c_int64, C.c_void_p,
                                        C.c_int32, C.c_void_p, C.c_int32, C.c_int32]),
    "llm_debug_noalloc_scratch_poke": (C.c_int, [C.c_uint32]),
    "llm_debug_gemm_tn_f16_trace": (C.c_int64, [C.c_int32, C.c_void_p, C.c_int64, C.c_int64, C.c_void_p, C.c_int32,
                                              C.c_void_p, C.c_int32, C.c_int32, C.c_int32,
                                              C.POINTER(C.c_uint64), C.c_int64]),
    "llm_debug_gemm_tn_q8": (C.c_int, [C.c_int32, C.c_void_p, C.c_void_p, C.c_int64, C.c_int64, C.c_void_p,
                                       C.c_int32, C.c_void_p, C.c_int32, C.c_int32, C.c_int32]),
    "llm_debug_gemm_tn_q8_trace": (C.c_int64, [C.c_int32, C.c_void_p, C.c_void_p, C.c_int64, C.c_int64,
                                             C.c_void_p, C.c_int32, C.c_void_p, C.c_int32, C.c_int32, C.c_int32,
                                             C.POINTER(C.c_uint64), C.c_int64]),
    "llm_debug_gemm_tn_f16": (C.c_int, [C.c_int32, C.c_void_p, C.c_void_p, C.c_int64, C.c_int64, C.c_void_p,
                                        C.c_int32, C.c_void_p, C.c_int32, C.c_int32, C.c_int32, C.c_int32]),
    "llm_debug_gemm_bf16": (C.c_int, [C.c_int32, C.c_void_p, C.c_int64, C.c_int64, C.c_void_p,
                                      C.c_int32, C.c_void_p, C.c_int32, C.c_int32]),
    "llm_set_attn_window": (C.c_int, [C.c_void_p, C.c_int32, C.c_int32]),
    "llm_sample_batch": (C.c_int32, [C.c_void_p, C.c_int32, C.POINTER(C.c_int32),
                                     C.POINTER(SamplerParams), C.POINTER(C.c_float),
                                     C.POINTER(C.c_int32)]),
    "llm_op_last_error": (C.c_char_p, []),
    "llm_kv_store": (C.c_int, [C.POINTER(KvPagesDesc), C.c_int32, C.c_void_p, C.c_void_p, C.c_int64,
                               C.c_int64, C.c_void_p, C.c_int32, C.c_void_p, C.c_void_p]),
    "llm_kv_load": (C.c_int, [C.POINTER(KvPagesDesc), C.c_int32, C.c_void_p, C.c_void_p, C.c_int64,
                              C.c_int64, C.c_void_p, C.c_int32, C.c_void_p, C.c_void_p]),
    "llm_pages_extend": (C.c_int, [C.POINTER(SeqPagesDesc), C.c_void_p, C.c_void_p, C.c_void_p, C.c_int32,
                                   C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p]),
    "llm_pages_trim": (C.c_int, [C.POINTER(SeqPagesDesc), C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p,
                                 C.c_void_p]),
    "llm_attn_plan_init": (C.c_void_p, [C.POINTER(AttnShape), C.POINTER(KvPagesDesc)]),
    "llm_attn_plan_free": (None, [C.c_void_p]),
    "llm_attn_plan_set": (C.c_int, [C.c_void_p, C.c_int32, C.POINTER(C.c_int32),
                                    C.POINTER(C.c_int32), C.POINTER(C.c_int32), C.c_int32,
                                    C.c_void_p]),
    "llm_attn_plan_set_device": (C.c_int, [C.c_void_p, C.c_int32, C.c_void_p, C.c_void_p, C.c_void_p,
                                           C.c_int32, C.c_int32, C.c_void_p]),
    "llm_attn_run": (C.c_int, [C.c_void_p, C.c_void_p, C.c_int64, C.c_int64,
                               C.POINTER(KvPagesDesc), C.c_void_p, C.c_int64, C.c_int64,
                               C.c_void_p]),
    "llm_attn_plan_form": (C.c_int, [C.c_void_p]),
    "llm_attn_plan_error": (C.c_uint32, [C.c_void_p]),
    "llm_sample_rows": (C.c_int, [C.POINTER(SampleRowsArgs), C.c_void_p]),
    "llm_debug_attn_units": (C.c_int64, [C.POINTER(AttnShape), C.POINTER(KvPagesDesc), C.c_int32,
                                         C.c_int32, C.c_int32, C.POINTER(C.c_int32),
                                         C.POINTER(C.c_int32), C.POINTER(C.c_int32), C.c_int64,
                                         C.POINTER(C.c_int64), C.POINTER(C.c_int32), C.POINTER(C.c_int64)]),
    "llm_debug_kernel_stats": (C.c_int32, [C.c_void_p, C.c_int32, C.c_char_p, C.c_int32,
                                           C.POINTER(C.c_int64), C.POINTER(C.c_double),
                                           C.POINTER(C.c_double), C.POINTER(C.c_double)]),
}

_lib = None


def lib():
    """Load libllm.so (built by transformer_decode_kv_gb300.build); raise if it is missing."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m transformer_decode_kv_gb300.build`")
        L = C.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _lib = L
    return _lib


def _i32(a) -> np.ndarray:
    return np.ascontiguousarray(np.asarray(a, dtype=np.int32))


def _ptr(a: np.ndarray, ct):
    return a.ctypes.data_as(C.POINTER(ct))


class LlmError(RuntimeError):
    pass


def debug_gemm_bf16(epi: int, W, X, Y, F: int = 0) -> int:
    """One tensor-core GEMM launch on torch CUDA tensors (W [rows][K] bf16, X [T][K] bf16)."""
    return lib().llm_debug_gemm_bf16(epi, C.c_void_p(W.data_ptr()), W.shape[0], W.shape[1],
                                     C.c_void_p(X.data_ptr()), X.shape[0], C.c_void_p(Y.data_ptr()),
                                     Y.stride(0), F)


def gemm_bf16_noalloc(epi: int, W, X, Y, F: int = 0) -> int:
    """The same GEMM through the entry point that allocates no device memory."""
    return lib().llm_gemm_bf16_noalloc(epi, C.c_void_p(W.data_ptr()), W.shape[0], W.shape[1],
                                       C.c_void_p(X.data_ptr()), X.shape[0],
                                       C.c_void_p(Y.data_ptr()), Y.stride(0), F)


def debug_gemm_tn_f16(epi: int, W, X, Y, F: int = 0, W_lo=None, splits: int = 1, one_cta: bool = False) -> int:
    """One token-major tensor-core GEMM launch on torch CUDA tensors (W [rows][K] f16, X [T][K] f16)."""
    M = W.shape[0] if epi != 2 else 0
    return lib().llm_debug_gemm_tn_f16(epi, C.c_void_p(W.data_ptr()),
                                       C.c_void_p(W_lo.data_ptr()) if W_lo is not None else None,
                                       M, W.shape[1], C.c_void_p(X.data_ptr()), X.shape[0],
                                       C.c_void_p(Y.data_ptr()), Y.stride(0), F, splits, int(one_cta))


def debug_gemm_tn_q8(epi: int, Wq, Ws, X, Y, F: int = 0, splits: int = 1) -> int:
    """The token-major GEMM over a Q8_0 weight (Wq int8 [rows][K], Ws f16 scales [rows][K / 32], X f16
    [T][K]) dequantised inside the kernel."""
    M = Wq.shape[0] if epi != 2 else 0
    return lib().llm_debug_gemm_tn_q8(epi, C.c_void_p(Wq.data_ptr()), C.c_void_p(Ws.data_ptr()), M, Wq.shape[1],
                                      C.c_void_p(X.data_ptr()), X.shape[0], C.c_void_p(Y.data_ptr()), Y.stride(0),
                                      F, splits)


def debug_gemm_tn_q8_trace(epi: int, Wq, Ws, X, Y, F: int = 0, splits: int = 1):
    """The Q8_0 token-major GEMM with its per-CTA counters: returns (status, [n_cta, 8] uint64)."""
    M = Wq.shape[0] if epi != 2 else 0
    cap = 8 * 8192
    out = np.zeros(cap, dtype=np.uint64)
    n = lib().llm_debug_gemm_tn_q8_trace(epi, C.c_void_p(Wq.data_ptr()), C.c_void_p(Ws.data_ptr()), M, Wq.shape[1],
                                         C.c_void_p(X.data_ptr()), X.shape[0], C.c_void_p(Y.data_ptr()), Y.stride(0),
                                         F, splits, out.ctypes.data_as(C.POINTER(C.c_uint64)), cap)
    return (0, out[:n].reshape(-1, 8)) if n > 0 else (int(n), None)


def debug_gemm_tn_f16_trace(epi: int, W, X, Y, F: int = 0, splits: int = 1):
    """The two-CTA token-major GEMM with its per-CTA timeline: returns (status, [n_cta, 8] uint64)."""
    M = W.shape[0] if epi != 2 else 0
    cap = 8 * 4096
    out = np.zeros(cap, dtype=np.uint64)
    n = lib().llm_debug_gemm_tn_f16_trace(epi, C.c_void_p(W.data_ptr()), M, W.shape[1], C.c_void_p(X.data_ptr()),
                                          X.shape[0], C.c_void_p(Y.data_ptr()), Y.stride(0), F, splits,
                                          out.ctypes.data_as(C.POINTER(C.c_uint64)), cap)
    return (0, out[:n].reshape(-1, 8)) if n > 0 else (int(n), None)


def debug_noalloc_scratch_poke(value: int) -> int:
    """Plant a value in the allocation-free GEMM's error word on the current device."""
    return lib().llm_debug_noalloc_scratch_poke(value)


# ---- operators on the caller's own torch CUDA tensors --------------------------------------------
# These calls are made many times a step, so their checks read each tensor property once.
_types = {}


def _type(t):
    """The llm_type of a torch tensor's elements (uint8 holds E4M3 codes), "int32", or None."""
    if not _types:
        import torch
        _types.update({torch.float32: F32, torch.float16: F16, torch.bfloat16: BF16,
                       torch.float8_e4m3fn: F8_E4M3, torch.uint8: F8_E4M3, torch.int32: "int32"})
    return _types.get(t.dtype)


def _type_of(t) -> int:
    """The llm_type of a tensor of values."""
    r = _type(t)
    if not isinstance(r, int):
        raise TypeError(f"unsupported element type {t.dtype}")
    return r


def _host_ints(a, name: str) -> np.ndarray:
    """Host integers as int32; one that int32 does not hold is refused, not wrapped."""
    x = np.asarray(a)
    if x.dtype != np.int32 and x.size:
        if x.dtype.kind not in "iu":
            raise TypeError(f"{name} must be integers, not {x.dtype}")
        if x.min() < -2 ** 31 or x.max() >= 2 ** 31:
            raise ValueError(f"{name} must fit int32")
    return _i32(x)


_raw_stream = None


def _stream_of(t, stream: Optional[int]) -> Optional[int]:
    """The given cudaStream_t, or torch's current stream of t's device."""
    global _raw_stream
    if stream is not None or not t.is_cuda:
        return stream
    if _raw_stream is None:
        import torch
        _raw_stream = torch._C._cuda_getCurrentRawStream
    return _raw_stream(t.get_device())


def _need(t, name: str, dtype, shape) -> int:
    """The address of t, which must be a dense tensor of this type and shape: the library reads it
    as such."""
    if not _types:
        _type(t)
    if _types.get(t.dtype) != dtype or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous tensor of shape {tuple(shape)} (int32 or "
                         f"float32 as documented), not {t.dtype} {tuple(t.shape)}")
    return t.data_ptr()


def _op(status: int) -> None:
    if status != 0:
        raise LlmError(lib().llm_op_last_error().decode() + f" ({status})")


def _rows(t, name: str, heads: int, dim: int):
    """The strides of a [tokens, heads, dim] tensor with dense rows."""
    sh, st = t.shape, t.stride()
    if len(sh) != 3 or sh[1] != heads or sh[2] != dim or st[2] != 1:
        raise ValueError(f"{name} must be [tokens, {heads}, {dim}] with dense rows, "
                         f"not {tuple(sh)} with strides {st}")
    if sh[0] == 1:                          # one row: torch's stride from it to the next says nothing
        return (heads * st[1] if heads > 1 else dim), st[1], 1
    return st


class KvPages:
    """A paged K/V cache held in torch CUDA tensors: k and v [n_pages, page_size, n_head_kv, head_dim]
    (float16, bfloat16, or E4M3 codes as float8_e4m3fn or uint8), in any memory order that keeps the
    rows of head_dim values dense (a [page, head, cell, dim] cache is passed as its transpose).
    k_scale and v_scale [n_pages, page_size, n_head_kv] float32 belong to an E4M3 cache. With k_block and
    v_block [n_pages, page_size, n_head_kv, head_dim / 16] too (E4M3 numbers as float8_e4m3fn or uint8, dense
    rows) it is a 4-bit cache: k and v are uint8 (or float4_e2m1fn_x2) [n_pages, page_size, n_head_kv,
    head_dim / 2], two E2M1 codes a byte, the first value in the low half."""

    def __init__(self, k, v, k_scale=None, v_scale=None, k_block=None, v_block=None):
        import torch
        if k.dim() != 4 or k.shape != v.shape or k.dtype != v.dtype or k.stride() != v.stride():
            raise ValueError("k and v must be alike, [n_pages, page_size, n_head_kv, head_dim]")
        if k.stride(3) != 1:
            raise ValueError("cache rows must be dense")
        d = KvPagesDesc()
        if (k_block is None) != (v_block is None):
            raise ValueError("k_block and v_block come together")
        f4 = k_block is not None
        if f4 and not (k.dtype is torch.uint8 or k.dtype is getattr(torch, "float4_e2m1fn_x2", torch.uint8)):
            raise TypeError(f"a 4-bit cache holds bytes of two codes (uint8), not {k.dtype}")
        d.type = F4_E2M1 if f4 else _type_of(k)
        d.n_pages, d.page_size, d.n_head_kv, d.head_dim = k.shape
        d.k, d.v = k.data_ptr(), v.data_ptr()
        d.stride_page, d.stride_cell, d.stride_head = k.stride()[:3]
        if (d.type in (F8_E4M3, F4_E2M1)) != (k_scale is not None) or (k_scale is None) != (v_scale is None):
            raise ValueError("E4M3 and 4-bit caches have scales, other caches have none")
        if f4:
            d.head_dim *= 2
            for b in (k_block, v_block):
                if _type(b) != F8_E4M3 or b.shape != k.shape[:3] + (d.head_dim // 16,) or \
                        (b.shape[3] > 1 and b.stride(3) != 1):
                    raise ValueError("block scales must be E4M3 bytes [n_pages, page_size, n_head_kv, head_dim / 16] "
                                     "with dense rows")
            if k_block.stride() != v_block.stride():
                raise ValueError("k_block and v_block must be laid out alike")
            d.k_block, d.v_block = k_block.data_ptr(), v_block.data_ptr()
            d.bstride_page, d.bstride_cell, d.bstride_head = k_block.stride()[:3]
        if k_scale is not None:
            for s in (k_scale, v_scale):
                if _type(s) != F32 or s.shape != k.shape[:3]:
                    raise ValueError("scales must be float32 [n_pages, page_size, n_head_kv]")
            if k_scale.stride() != v_scale.stride():
                raise ValueError("k_scale and v_scale must be laid out alike")
            d.k_scale, d.v_scale = k_scale.data_ptr(), v_scale.data_ptr()
            d.sstride_page, d.sstride_cell, d.sstride_head = k_scale.stride()
        self.desc = d
        self.ref = C.byref(d)
        self.heads, self.dim = d.n_head_kv, d.head_dim
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.k_block, self.v_block = k_block, v_block

    def _kv_rows(self, fn, k, v, cell, err, stream):
        st = _rows(k, "k", self.heads, self.dim)
        n = k.shape[0]
        if v.shape != k.shape or v.dtype is not k.dtype or _rows(v, "v", self.heads, self.dim) != st:
            raise ValueError("k and v must be alike")
        cells = _need(cell, "cell", "int32", (n,))
        r = fn(self.ref, _type_of(k), k.data_ptr(), v.data_ptr(), st[0], st[1], cells, n,
               None if err is None else _need(err, "err", "int32", (1,)), _stream_of(k, stream))
        if r != 0:
            _op(r)


def kv_store(pages: KvPages, k, v, cell, err=None, stream: Optional[int] = None) -> None:
    """Write rows k, v [n, n_head_kv, head_dim] into cells cell [n] (int32; negative: skipped) of the
    cache, cast or quantised to its type. err: an optional device word (int32 [1]) for bad cells."""
    pages._kv_rows(lib().llm_kv_store, k, v, cell, err, stream)


def kv_load(pages: KvPages, cell, k, v, err=None, stream: Optional[int] = None) -> None:
    """Read the rows of cells cell [n] back into k, v [n, n_head_kv, head_dim] (rows of negative cells
    are left as they were)."""
    pages._kv_rows(lib().llm_kv_load, k, v, cell, err, stream)


class SeqPages:
    """The pages of a step's sequences, in torch CUDA tensors (int32): table [n_seq, ld], each sequence's pages in
    order; n_kv [n_seq], the rows it holds; free [max_free], the stack of free pages, of which the first n_free [1] count
    (the last of them is handed out first). Pages of page_size cells, numbers below n_pages."""

    def __init__(self, table, n_kv, free, n_free, page_size: int, n_pages: int):
        if table.dim() != 2 or free.dim() != 1:
            raise ValueError("table must be [n_seq, pages] and free [max_free]")
        if not (-2 ** 31 <= page_size < 2 ** 31 and -2 ** 31 <= n_pages < 2 ** 31):
            raise ValueError("page_size and n_pages must fit int32")      # (ctypes would wrap them)
        d = SeqPagesDesc()
        d.n_seq, d.ld_table = table.shape
        d.page_size, d.n_pages, d.max_free = page_size, n_pages, free.shape[0]
        self.n_seq = d.n_seq
        d.table = _need(table, "table", "int32", table.shape)
        d.n_kv = _need(n_kv, "n_kv", "int32", (d.n_seq,))
        d.free_pages = _need(free, "free", "int32", free.shape)
        d.n_free = _need(n_free, "n_free", "int32", (1,))
        self.desc, self.ref = d, C.byref(d)
        self.table, self.n_kv, self.free, self.n_free = table, n_kv, free, n_free

    def _outs(self, n_kv_out, n_free_out, err):
        d = self.desc
        return (d.n_kv if n_kv_out is None else _need(n_kv_out, "n_kv_out", "int32", (self.n_seq,)),
                d.n_free if n_free_out is None else _need(n_free_out, "n_free_out", "int32", (1,)),
                None if err is None else _need(err, "err", "int32", (1,)))


def pages_extend(lists: SeqPages, n_new, cell, pos, start, n_kv_out=None, n_free_out=None, err=None,
                 stream: Optional[int] = None) -> None:
    """Room for n_new [n_seq] tokens behind the sequences' rows, with pages from the stack: cell and pos [max_tok]
    receive the cell and position of every new token (-1 behind the last), start [n_seq + 1] the first token of each sequence,
    n_kv_out and n_free_out (None: in place) the new lengths and the stack's size. A step that does not fit sets
    bit 32 of err, an optional device word (int32 [1]), and has no tokens."""
    kv_out, free_out, e = lists._outs(n_kv_out, n_free_out, err)
    n_seq, n = lists.n_seq, cell.numel()
    row = (n,)
    r = (_lib or lib()).llm_pages_extend(
        lists.ref, _need(n_new, "n_new", "int32", (n_seq,)), kv_out, free_out, n, _need(cell, "cell", "int32", row),
        _need(pos, "pos", "int32", row), _need(start, "start", "int32", (n_seq + 1,)), e,
        _stream_of(lists.n_free, stream))
    if r != 0:
        _op(r)


def pages_trim(lists: SeqPages, keep, n_kv_out=None, n_free_out=None, err=None, stream: Optional[int] = None) -> None:
    """Shorten sequences to keep [n_seq] rows (negative: as it is) and put the pages that this leaves without rows
    on the stack. A call that does not fit sets bit 32 of err and changes nothing."""
    kv_out, free_out, e = lists._outs(n_kv_out, n_free_out, err)
    r = lib().llm_pages_trim(lists.ref, _need(keep, "keep", "int32", (lists.n_seq,)), kv_out, free_out, e,
                             _stream_of(lists.n_free, stream))
    if r != 0:
        _op(r)


class AttnPlan:
    """Attention of new tokens over a paged cache like `pages` (its type and shape, not its memory):
    made once, set once per step, run once per layer. dtype is the type of q and out."""

    _replayed_tok = 0                       # tokens that a step may have which a graph's replay sets: none, or max_tok

    def __init__(self, pages: KvPages, n_head: int, dtype, max_tok: int, max_seq: int, max_table: int,
                 window: int = 0, n_sink: int = 0, scale: float = 0.0):
        import torch
        self.ptr = None
        types = {torch.float32: F32, torch.float16: F16, torch.bfloat16: BF16}
        if dtype not in types:
            raise TypeError(f"unsupported activation type {dtype}")
        self.dtype, self.n_head, self.head_dim = dtype, n_head, pages.dim
        self.device = pages.k.device
        self.n_tok, self.max_tok = 0, max_tok
        self._captured_rows = None          # fewest rows of q and out of the runs that were captured
        self._capturing = torch._C._cuda_isCurrentStreamCapturing if pages.k.is_cuda else (lambda: False)
        self._run = lib().llm_attn_run
        s = AttnShape(types[dtype], n_head, scale, window, n_sink, max_tok, max_seq, max_table)
        with torch.cuda.device(self.device if pages.k.is_cuda else -1):
            self.ptr = lib().llm_attn_plan_init(C.byref(s), pages.ref)
        if not self.ptr:
            raise LlmError("llm_attn_plan_init failed: " + lib().llm_op_last_error().decode())

    def free(self) -> None:
        if self.ptr:
            lib().llm_attn_plan_free(self.ptr)
            self.ptr = None

    def __del__(self):
        try:
            self.free()
        except Exception:
            pass

    def set(self, n_new, n_kv, pages, stream: Optional[int] = None) -> None:
        """The step's sequences: n_new tokens each, n_kv cached rows each (the new ones included), page
        table [n_seq, at least ceil(n_kv / page_size)]; host integers."""
        n_new, n_kv = _host_ints(n_new, "n_new"), _host_ints(n_kv, "n_kv")
        t = _host_ints(pages, "pages")
        if n_new.ndim != 1 or n_new.shape != n_kv.shape or t.ndim != 2 or len(t) != len(n_new):
            raise ValueError("n_new [n_seq], n_kv [n_seq] and pages [n_seq, n] are needed")
        if self._captured_rows is not None and n_new.sum() > self._captured_rows:
            raise ValueError(f"a captured run's q or out has only {self._captured_rows} rows")
        if stream is None:
            import torch
            stream = torch.cuda.current_stream(self.device).cuda_stream
        _op(lib().llm_attn_plan_set(self.ptr, len(n_new), _ptr(n_new, C.c_int32),
                                    _ptr(n_kv, C.c_int32), _ptr(t, C.c_int32), t.shape[1], stream))
        self.n_tok = max(int(n_new.sum()), self._replayed_tok)

    def set_device(self, start, n_kv, pages, max_new: int, stream: Optional[int] = None) -> None:
        """The same from device tensors (int32), as pages_extend leaves them, without a wait: start [n_seq + 1], the
        first new token of each sequence and their number; n_kv [n_seq], cached rows with the new ones; page table
        [n_seq, ld]. max_new bounds a sequence's new tokens. Runs then need q and out of max_tok rows. Captured, the call
        is made again by every replay, whatever the plan was set to before: from then on every run needs max_tok rows."""
        n = n_kv.shape[0]
        if pages.dim() != 2 or pages.shape[0] != n:
            raise ValueError("pages must be [n_seq, n]")
        if not -2 ** 31 <= max_new < 2 ** 31:
            raise ValueError("max_new must fit int32")
        if self._captured_rows is not None and self.max_tok > self._captured_rows:
            raise ValueError(f"a captured run's q or out has only {self._captured_rows} rows, and a step that is set on the "
                             f"device may have {self.max_tok} tokens")
        ld = pages.shape[1]
        _op(lib().llm_attn_plan_set_device(self.ptr, n, _need(start, "start", "int32", (n + 1,)),
                                           _need(n_kv, "n_kv", "int32", (n,)), _need(pages, "pages", "int32", (n, ld)), ld,
                                           max_new, _stream_of(start, stream)))
        self.n_tok = self.max_tok
        if self._captures(stream):
            self._replayed_tok = self.max_tok

    def _captures(self, stream: Optional[int]) -> bool:
        """Whether a run on this stream (None: torch's current one) is recorded into a graph."""
        if stream is None or stream == 0:                   # (the legacy stream, 0, cannot be captured)
            return stream is None and self._capturing()
        import torch
        with torch.cuda.stream(torch.cuda.ExternalStream(stream, device=self.device)):
            return self._capturing()

    def run(self, q, pages: KvPages, out, stream: Optional[int] = None) -> None:
        """out[i] = attention of token i of the step; q and out [at least the step's tokens, n_head,
        head_dim], rows past the tokens are not touched. After a captured run the plan takes no step of
        more tokens than that run's q and out have rows; after a captured set_device every run needs max_tok rows."""
        sq = _rows(q, "q", self.n_head, self.head_dim)
        so = _rows(out, "out", self.n_head, self.head_dim)
        if q.dtype is not self.dtype or out.dtype is not self.dtype:
            raise TypeError(f"q and out must be {self.dtype}")
        if q.shape[0] < self.n_tok or out.shape[0] < self.n_tok:
            raise ValueError(f"q or out has fewer rows than the step has tokens ({self.n_tok})" + (
                ": a graph holds a set_device, whose replay may set as many" if self._replayed_tok else ""))
        if self._captures(stream):
            rows = min(q.shape[0], out.shape[0])
            self._captured_rows = rows if self._captured_rows is None else min(rows, self._captured_rows)
        r = self._run(self.ptr, q.data_ptr(), sq[0], sq[1], pages.ref, out.data_ptr(), so[0], so[1],
                      _stream_of(q, stream))
        if r != 0:
            _op(r)

    @property
    def form(self) -> int:
        return lib().llm_attn_plan_form(self.ptr)

    def error(self) -> int:
        """The plan's error word after the device has finished (0 = none)."""
        return lib().llm_attn_plan_error(self.ptr)


def sample_rows(logits, token, u=None, top_k=None, top_p=None, min_p=None, temperature=None,
                repeat_penalty=None, penalty_start=None, penalty_token=None,
                stream: Optional[int] = None) -> None:
    """The sampler chain for every row of logits [n, n_vocab]; token [n] int32 receives the picks. The
    parameters are device arrays of n values (top_k int32, the others float32; None = off; temperature
    None = greedy); row r's penalty tokens are penalty_token[penalty_start[r]:penalty_start[r + 1]]."""
    sh = logits.shape
    if len(sh) != 2 or (sh[1] > 1 and logits.stride(1) != 1):
        raise ValueError("logits must be [rows, n_vocab] with dense rows")
    R = sh[0]
    row = (R,)
    a = SampleRowsArgs()
    a.type = _type_of(logits)
    a.n_rows, a.n_vocab, a.ld, a.logits = R, sh[1], logits.stride(0), logits.data_ptr()
    a.token = _need(token, "token", "int32", row)
    if u is not None:
        a.u = _need(u, "u", F32, row)
    if top_k is not None:
        a.top_k = _need(top_k, "top_k", "int32", row)
    if top_p is not None:
        a.top_p = _need(top_p, "top_p", F32, row)
    if min_p is not None:
        a.min_p = _need(min_p, "min_p", F32, row)
    if temperature is not None:
        a.temperature = _need(temperature, "temperature", F32, row)
    if repeat_penalty is not None:
        a.repeat_penalty = _need(repeat_penalty, "repeat_penalty", F32, row)
        if penalty_start is not None and penalty_token is not None:
            n = penalty_token.numel()
            a.penalty_start = _need(penalty_start, "penalty_start", "int32", (R + 1,))
            a.penalty_token = _need(penalty_token, "penalty_token", "int32", (n,))
            a.n_penalty_token = n
    r = lib().llm_sample_rows(C.byref(a), _stream_of(logits, stream))
    if r != 0:
        _op(r)


class Context:
    """One llm_ctx: a model's weights, a unified KV cache and the decode state."""

    def __init__(self, hp, n_ctx: int, n_seq_max: int = 1, type_k: int = F16, type_v: int = F16,
                 n_batch: int = 2048, n_ubatch: int = 512, stream: Optional[int] = None,
                 host_only: bool = False, fused_step: bool = False, kv_unified: bool = True):
        L = lib()
        self._hp = HParams(hp.n_layer, hp.n_embd, hp.n_head, hp.n_head_kv, hp.head_dim, hp.n_ff,
                           hp.n_vocab, hp.rope_freq_base, hp.rms_eps, getattr(hp, "rope_type", 0))
        cp = L.llm_cparams_default()
        cp.n_ctx, cp.n_seq_max, cp.n_batch, cp.n_ubatch = n_ctx, n_seq_max, n_batch, n_ubatch
        cp.type_k, cp.type_v = type_k, type_v
        cp.stream = stream
        cp.flags = ((CTX_HOST_ONLY if host_only else 0) | (CTX_FUSED_STEP if fused_step else 0) |
                    (0 if kv_unified else CTX_KV_SPLIT))
        self.n_vocab = hp.n_vocab
        self.type_k = type_k
        self.ptr = L.llm_ctx_init(C.byref(self._hp), C.byref(cp))
        if not self.ptr:
            raise LlmError("llm_ctx_init failed: " + L.llm_last_error(None).decode())
        self._abort = None

    # ---- lifetime
    def free(self):
        if self.ptr:
            lib().llm_ctx_free(self.ptr)
            self.ptr = None

    def __del__(self):
        try:
            self.free()
        except Exception:
            pass

    def last_error(self) -> str:
        return lib().llm_last_error(self.ptr).decode()

    # ---- weights
    def load_weight(self, name: str, wtype: int, shape: Sequence[int], data) -> int:
        """data: a torch tensor (host or CUDA) or numpy array holding the storage bytes."""
        ne = (C.c_int64 * 2)(int(shape[0]), int(shape[1]) if len(shape) > 1 else 1)
        if hasattr(data, "data_ptr"):
            t = data.contiguous()
            ptr, nbytes = t.data_ptr(), t.numel() * t.element_size()
            keep = t
        else:
            keep = np.ascontiguousarray(data)
            ptr, nbytes = keep.ctypes.data, keep.nbytes
        r = lib().llm_load_weights(self.ptr, name.encode(), wtype, ne, C.c_void_p(ptr), nbytes)
        del keep
        return r

    def load_all(self, tensors: Iterable) -> None:
        """Load (name, wtype, shape, storage) tuples; raise on the first failure."""
        for name, wt, shape, t in tensors:
            if self.load_weight(name, wt, shape, t) != 0:
                raise LlmError(f"load {name}: {self.last_error()}")
        if lib().llm_weights_ready(self.ptr) != 0:
            raise LlmError(self.last_error())

    def weights_ready(self) -> int:
        return lib().llm_weights_ready(self.ptr)

    # ---- decode
    def decode(self, tokens, pos=None, seq_ids=None, logits=None) -> int:
        """tokens: ints; pos: ints or None; seq_ids: list of lists (or ints) or None;
        logits: flags or None. Returns llm_decode's status."""
        tok = _i32(tokens)
        n = len(tok)
        keep = [tok]
        b = Batch()
        b.n_tokens = n
        b.token = _ptr(tok, C.c_int32)
        if pos is not None:
            p = _i32(pos); keep.append(p); b.pos = _ptr(p, C.c_int32)
        if seq_ids is not None:
            # one flat id array; row i's pointer is its start inside it
            if len(seq_ids) != n:
                raise ValueError("seq_ids needs one row per token")
            rows = [r if hasattr(r, "__len__") else (r,) for r in seq_ids]
            nsid = np.fromiter((len(r) for r in rows), dtype=np.int32, count=n)
            flat = np.fromiter((x for r in rows for x in r), dtype=np.int32, count=int(nsid.sum()))
            start = np.zeros(n, dtype=np.uint64)
            np.cumsum(nsid[:-1], out=start[1:])
            ptrs = np.ascontiguousarray(np.uint64(flat.ctypes.data) + np.uint64(4) * start)
            keep += [nsid, flat, ptrs]
            b.n_seq_id = _ptr(nsid, C.c_int32)
            b.seq_id = ptrs.ctypes.data_as(C.POINTER(C.POINTER(C.c_int32)))
        if logits is not None:
            lg = np.ascontiguousarray(np.asarray(logits, dtype=np.int8)); keep.append(lg)
            b.logits = _ptr(lg, C.c_int8)
        return lib().llm_decode(self.ptr, b)

    def get_logits_ith(self, i: int) -> Optional[np.ndarray]:
        p = lib().llm_get_logits_ith(self.ptr, i)
        if not p:
            return None
        return np.ctypeslib.as_array(p, shape=(self.n_vocab,)).copy()

    def sample_ith(self, i: int, top_k: int = 40, top_p: float = 1.0, min_p: float = 0.0,
                   temperature: float = 1.0, repeat_penalty: float = 1.0, penalty_tokens=(),
                   u: float = 0.0) -> int:
        """The device sampler chain over logits row i; u in [0, 1) is the uniform draw."""
        pen = np.asarray(list(penalty_tokens), dtype=np.int32)
        p = SamplerParams(top_k, top_p, min_p, temperature, repeat_penalty,
                          pen.ctypes.data_as(C.POINTER(C.c_int32)) if len(pen) else None, len(pen))
        return lib().llm_sample_ith(self.ptr, i, C.byref(p), u)

    def sample_batch(self, rows, u, top_k=40, top_p=1.0, min_p=0.0, temperature=1.0,
                     repeat_penalty=1.0, penalty_tokens=None) -> np.ndarray:
        """The sampler chain for several rows in one launch: row rows[j] with the draw u[j]. The
        parameters are numbers, or one per row; penalty_tokens one list per row. Returns the tokens."""
        rows, u = _i32(rows), np.ascontiguousarray(u, dtype=np.float32)
        n = len(rows)
        if u.shape != (n,):
            raise ValueError("u needs one draw per row")
        col = lambda v: np.broadcast_to(np.asarray(v), (n,))
        cols = [col(x) for x in (top_k, top_p, min_p, temperature, repeat_penalty)]
        pens = [_i32(list(p)) for p in penalty_tokens] if penalty_tokens is not None else [_i32([])] * n
        if len(pens) != n:
            raise ValueError("penalty_tokens needs one list per row")
        ps = (SamplerParams * max(n, 1))()
        for j in range(n):
            ps[j] = SamplerParams(int(cols[0][j]), float(cols[1][j]), float(cols[2][j]), float(cols[3][j]),
                                  float(cols[4][j]), _ptr(pens[j], C.c_int32) if len(pens[j]) else None,
                                  len(pens[j]))
        out = np.zeros(n, dtype=np.int32)
        if lib().llm_sample_batch(self.ptr, n, _ptr(rows, C.c_int32), ps, _ptr(u, C.c_float),
                                  _ptr(out, C.c_int32)) != 0:
            raise LlmError(self.last_error())
        return out

    def set_attn_window(self, window: int, n_sink: int = 0) -> int:
        return lib().llm_set_attn_window(self.ptr, window, n_sink)

    def debug_set_logits(self, i: int, row) -> int:
        r = np.ascontiguousarray(row, dtype=np.float32)
        assert r.shape == (self.n_vocab,)
        return lib().llm_debug_set_logits(self.ptr, i, _ptr(r, C.c_float))

    def get_argmax_ith(self, i: int) -> int:
        return lib().llm_get_argmax_ith(self.ptr, i)

    @property
    def n_outputs(self) -> int:
        return lib().llm_n_outputs(self.ptr)

    # ---- memory
    def seq_rm(self, seq: int, p0: int, p1: int) -> int:
        return lib().llm_seq_rm(self.ptr, seq, p0, p1)

    def memory_update(self, optimize: bool = True) -> int:
        return lib().llm_memory_update(self.ptr, int(optimize))

    def seq_pos_max(self, s: int) -> int:
        return lib().llm_seq_pos_max(self.ptr, s)

    def seq_pos_min(self, s: int) -> int:
        return lib().llm_seq_pos_min(self.ptr, s)

    def set_abort_callback(self, fn):
        """fn() -> bool, or None to remove."""
        if fn is None:
            self._abort = None
            lib().llm_set_abort_callback(self.ptr, ABORT_CB(), None)
            return
        self._abort = ABORT_CB(lambda _ud: 1 if fn() else 0)
        lib().llm_set_abort_callback(self.ptr, self._abort, None)

    @property
    def n_ctx(self) -> int:
        return lib().llm_n_ctx(self.ptr)

    @property
    def n_ctx_seq(self) -> int:
        return lib().llm_n_ctx_seq(self.ptr)

    @property
    def n_batch(self) -> int:
        return lib().llm_n_batch(self.ptr)

    @property
    def n_ubatch(self) -> int:
        return lib().llm_n_ubatch(self.ptr)

    def kv_used_cells(self) -> int:
        return lib().llm_kv_used_cells(self.ptr)

    def perf(self) -> dict:
        d = PerfData()
        lib().llm_perf(self.ptr, C.byref(d))
        return {k: getattr(d, k) for k, _ in PerfData._fields_}

    # ---- debug hooks
    def last_slots(self) -> np.ndarray:
        n = lib().llm_debug_last_slots(self.ptr, None, 0)
        out = np.zeros(n, dtype=np.int32)
        lib().llm_debug_last_slots(self.ptr, _ptr(out, C.c_int32), n)
        return out

    def ubatch_mask(self, ub: int):
        nkv = C.c_int32(0)
        n = lib().llm_debug_ubatch_mask(self.ptr, ub, None, 0, C.byref(nkv))
        if n == 0 and nkv.value == 0:
            return None
        out = np.zeros(n, dtype=np.uint8)
        lib().llm_debug_ubatch_mask(self.ptr, ub, _ptr(out, C.c_uint8), n, C.byref(nkv))
        return out.reshape(-1, nkv.value).astype(bool) if nkv.value else out.reshape(0, 0)

    def debug_capture(self, enable: bool = True) -> int:
        return lib().llm_debug_capture(self.ptr, int(enable))

    def debug_tensor(self, name: str, layer: int = 0) -> Optional[np.ndarray]:
        n = lib().llm_debug_get_tensor(self.ptr, name.encode(), layer, None, 0)
        if n <= 0:
            return None
        out = np.zeros(n, dtype=np.float32)
        lib().llm_debug_get_tensor(self.ptr, name.encode(), layer, _ptr(out, C.c_float), n)
        return out

    def kv_cache(self, layer: int, which: int) -> Optional[np.ndarray]:
        """Layer `layer`'s K (which 0) or V (which 1) cache as stored, [n_head_kv][n_ctx][head_dim]
        (float32 or float16 elements). A Q8_0 cache comes back as its 34-byte blocks (fp16 scale,
        then 32 int8 quants), uint8 [n_head_kv][n_ctx][head_dim / 32 * 34]; an E4M3 cache as rows of a
        float32 scale, then the codes, uint8 [n_head_kv][n_ctx][4 + head_dim]."""
        n = lib().llm_debug_kv_raw(self.ptr, layer, which, None, 0)
        if n <= 0:
            return None
        out = np.zeros(n, dtype=np.uint8)
        lib().llm_debug_kv_raw(self.ptr, layer, which, out.ctypes.data_as(C.c_void_p), n)
        Hkv, hd = self._hp.n_head_kv, self._hp.head_dim
        if self.type_k == Q8_0:
            nq = n // 34 * 32
            q = out[:nq].reshape(Hkv, -1, hd // 32, 32)
            s = out[nq:].reshape(Hkv, -1, hd // 32, 2)
            return np.concatenate([s, q], axis=3).reshape(Hkv, -1, hd // 32 * 34)
        if self.type_k == F8_E4M3:
            nq = Hkv * self.n_ctx * hd
            return np.concatenate([out[nq:].reshape(Hkv, -1, 4), out[:nq].reshape(Hkv, -1, hd)], axis=2)
        es = 4 if n // (self._hp.n_head_kv * self._hp.head_dim) == 4 * self.n_ctx else 2
        v = out.view(np.float32 if es == 4 else np.float16)
        return v.reshape(self._hp.n_head_kv, -1, self._hp.head_dim)

    def kv_f16_copy(self, which: int) -> Optional[np.ndarray]:
        """Q8_0 caches: the f16 copy of the K (which 0) or V (which 1) quants that the last
        attention over query tiles of several tokens read, float16 [n_head_kv][n_ctx][head_dim]
        (cells below that ubatch's n_kv are valid)."""
        n = lib().llm_debug_kv_raw(self.ptr, 0, which + 2, None, 0)
        if n <= 0:
            return None
        out = np.zeros(n, dtype=np.uint8)
        lib().llm_debug_kv_raw(self.ptr, 0, which + 2, out.ctypes.data_as(C.c_void_p), n)
        return out.view(np.float16).reshape(self._hp.n_head_kv, -1, self._hp.head_dim)

    def step_trace_enable(self, enable: bool = True) -> int:
        return lib().llm_debug_step_trace_enable(self.ptr, int(enable))

    def step_trace(self) -> Optional[np.ndarray]:
        """The last traced one-token step as uint64 [blocks][slots][2] (start, end) ns stamps."""
        nb, ns = C.c_int32(0), C.c_int32(0)
        n = lib().llm_debug_step_trace(self.ptr, None, 0, C.byref(nb), C.byref(ns))
        if n <= 0:
            return None
        out = np.zeros(n, dtype=np.uint64)
        lib().llm_debug_step_trace(self.ptr, out.ctypes.data_as(C.POINTER(C.c_uint64)), n, None, None)
        return out.reshape(nb.value, ns.value, 2)

    def kernel_timing(self, enable: bool = True) -> int:
        return lib().llm_debug_kernel_timing(self.ptr, int(enable))

    def kernel_stats(self) -> dict:
        """{class name: {launches, ms, bytes, flops}} of the timed launches."""
        L = lib()
        n = L.llm_debug_kernel_stats(self.ptr, 0, None, 0, None, None, None, None)
        out = {}
        for i in range(n):
            name = C.create_string_buffer(64)
            la, ms, by, fl = C.c_int64(), C.c_double(), C.c_double(), C.c_double()
            L.llm_debug_kernel_stats(self.ptr, i, name, 64, C.byref(la), C.byref(ms), C.byref(by),
                                     C.byref(fl))
            out[name.value.decode()] = {"launches": la.value, "ms": ms.value, "bytes": by.value,
                                        "flops": fl.value}
        return out

    def inject_fault(self, kind: int, ub: int = 0) -> int:
        return lib().llm_debug_inject_fault(self.ptr, kind, ub)
