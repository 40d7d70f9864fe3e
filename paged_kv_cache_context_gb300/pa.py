"""Python binding of the C ABI in include/pa.h (argument marshalling only).

Every function takes torch CUDA tensors, passes their device pointers and
sizes to the same-named C entry point of ``libpagedattn.so`` on the current
torch stream, and raises ``PagedAttentionError`` on a non-zero status. All
computation runs in the library's CUDA kernels; there is no fallback: if the
library is missing, loading fails loudly.

The sizes the C calls receive are read from the tensors' shapes, so before a
call the binding checks what the C side cannot see: that every tensor is a
CUDA tensor on one device (the library takes raw device pointers) and that
the shapes and element types of the arguments agree with each other. A
mismatch raises ``ValueError`` and nothing is enqueued.
"""
from __future__ import annotations

import ctypes
import math
import os
from typing import Optional, Tuple

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_lib", "libpagedattn.so")

# enums of include/pa.h
PA_F32, PA_BF16, PA_F16 = 0, 1, 2
PA_KV_AUTO, PA_KV_FP8_E4M3, PA_KV_INT8, PA_KV_FP8_BLOCK = 0, 1, 2, 4
PA_ERR_DEVICE = -9
DEVERR_BITS = {1: "slot", 2: "block_id", 4: "context_len", 8: "timeout", 16: "seq"}

_DTYPE = {torch.float32: PA_F32, torch.bfloat16: PA_BF16, torch.float16: PA_F16}
_KV = {"auto": PA_KV_AUTO, "fp8_e4m3": PA_KV_FP8_E4M3, "int8": PA_KV_INT8,
       "fp8_block": PA_KV_FP8_BLOCK}

_lib = None


class PagedAttentionError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: status {status} ({status_string(status)})")


def lib() -> ctypes.CDLL:
    """The loaded library (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: build it with "
                              "paged_kv_cache_context_gb300.build.build()")
        L = ctypes.CDLL(LIB_PATH)
        P, I, F, Z = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
        N = ctypes.c_int64
        sig = {
            "pa_slot_mapping": [P, P, P, P, I, I, I, I, I, P],
            "pa_reshape_and_cache": [P, P, P, P, P, I, I, I, I, I, I, I, F, F, P],
            "pa_decode": [P, P, P, P, P, P, I, I, I, I, I, I, I, F, I, I, I, F, F, P, Z, P],
            "pa_decode_plan": [I, I, I, I, I, I, I, P, P],
            "pa_decode_workspace_size": [I, I, I, I, I, I, I],
            "pa_decode_partials": [P, P, P, P, P, P, P, P, I, I, I, I, I, I, I, F, I, I, I, F,
                                   F, I, I, P],
            "pa_reduce": [P, P, P, P, I, I, I, I, I, P],
            "pa_decode_balanced": [P, P, P, P, P, P, I, I, I, I, I, I, I, F, I, I, I, F, F, P,
                                   Z, P, P],
            "pa_decode_workspace_clear": [P, Z, P],
            "pa_decode_cascade_workspace_size": [I, I, I, I, I, I],
            "pa_decode_cascade": [P, P, P, P, P, P, I, I, I, I, I, I, I, F, I, I, P, Z, P],
            "pa_decode_cascade_fp8": [P, P, P, P, P, P, I, I, I, I, I, I, I, F, F, F, I, I, P, Z,
                                      P],
            "pa_decode_cascade_int8": [P, P, P, P, P, P, P, P, I, I, I, I, I, I, I, F, I, I, P, Z,
                                       P],
            "pa_copy_blocks": [P, P, P, I, I, I, I, I, I, P],
            "pa_block_budget": [I, ctypes.c_double, Z, I, I, I, I, I, I],
            "pa_reshape_and_cache_int8": [P, P, P, P, P, P, P, I, I, I, I, I, I, P],
            "pa_decode_int8": [P, P, P, P, P, P, P, P, I, I, I, I, I, I, I, F, I, I, P, Z, P],
            "pa_prefill": [P, P, P, P, P, P, P, I, I, I, I, I, I, I, I, I, F, I, P],
            "pa_prefill_int8": [P, P, P, P, P, P, P, P, P, I, I, I, I, I, I, I, I, I, F, I, P],
            "pa_prefill_fp8": [P, P, P, P, P, P, P, I, I, I, I, I, I, I, I, I, F, F, F, I, P],
            "pa_tree_workspace_size": [I, I, I],
            "pa_tree": [P, P, P, P, P, P, P, P, I, I, I, I, I, I, I, I, I, I, F, I, P, Z, P],
            "pa_tree_int8": [P, P, P, P, P, P, P, P, P, P, I, I, I, I, I, I, I, I, I, I, F, I, P,
                             Z, P],
            "pa_tree_fp8": [P, P, P, P, P, P, P, P, I, I, I, I, I, I, I, I, I, I, F, F, F, I, P,
                            Z, P],
            "pa_decode_scored_workspace_size": [I, I, I, I, I, I],
            "pa_decode_scored": [P, P, P, P, P, P, P, I, I, I, I, I, I, I, F, I, I, F, F, P, Z,
                                 P],
            "pa_decode_scored_int8": [P, P, P, P, P, P, P, P, P, I, I, I, I, I, I, I, F, I, P, Z,
                                      P],
            "pa_evict_select": [P, P, P, P, I, I, I, I, I, I, P],
            "pa_compact": [P, P, P, P, P, P, P, P, P, P, I, I, I, I, I, I, I, I, I, P],
            "pa_norm_rope": [P, P, P, P, P, P, P, P, I, I, I, I, I, I, N, N, N, N, F, I, I, P],
            "pa_norm_rope_and_cache": [P, P, P, P, P, P, P, P, P, P, P, I, I, I, I, I, I, I, I, N,
                                       N, N, N, F, I, I, I, F, F, P],
            "pa_append_fp8_block": [P, P, P, P, P, P, P, P, P, I, I, I, I, I, I, I, N, N, I, P],
            "pa_decode_fp8_block": [P, P, P, P, P, P, P, P, I, I, I, I, I, I, I, F, I, P, Z, P],
            "pa_prefill_fp8_block_workspace_size": [I, I, I],
            "pa_prefill_fp8_block": [P, P, P, P, P, P, P, P, P, I, I, I, I, I, I, I, I, I, F, I, P,
                                     Z, P],
            "pa_decode_static_scratch": [P, P, P, P, P, P, I, I, I, I, I, I, I, F, I, I, I, F,
                                         F, P],
            "pa_get_device_error": [P, P],
            "pa_status_string": [I],
            "pa_version": [],
        }
        for name, args in sig.items():
            fn = getattr(L, name)
            fn.argtypes = args
            fn.restype = I
        L.pa_decode_workspace_size.restype = Z
        L.pa_decode_cascade_workspace_size.restype = Z
        L.pa_tree_workspace_size.restype = Z
        L.pa_prefill_fp8_block_workspace_size.restype = Z
        L.pa_decode_scored_workspace_size.restype = Z
        L.pa_block_budget.restype = ctypes.c_int64
        L.pa_status_string.restype = ctypes.c_char_p
        L.pa_test_set_unarmed_page.argtypes = [I]
        L.pa_test_set_unarmed_page.restype = None
        _lib = L
    return _lib


def status_string(status: int) -> str:
    return lib().pa_status_string(status).decode()


def version() -> int:
    return lib().pa_version()


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return t.data_ptr()


def _is_device_tensor(t: torch.Tensor) -> bool:
    return t.is_cuda


def _need(cond: bool, msg: str):
    if not cond:
        raise ValueError(msg)


def _on_device(**named):
    """Every tensor argument is a CUDA tensor, all on one device."""
    dev = None
    for name, t in named.items():
        if t is None:
            continue
        if not isinstance(t, torch.Tensor):
            raise ValueError(f"{name}: expected a torch tensor")
        if not _is_device_tensor(t):
            raise ValueError(f"{name}: must be a CUDA tensor (the library takes device pointers)")
        if dev is None:
            dev = t.device
        elif t.device != dev:
            raise ValueError(f"{name}: every tensor must be on {dev}")


def _shape(name: str, t: torch.Tensor, shape):
    if t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")


def _dtype(name: str, t: torch.Tensor, dt: torch.dtype):
    if t.dtype != dt:
        raise ValueError(f"{name}: dtype {t.dtype}, expected {dt}")


_CACHE_DTYPE = {"fp8_e4m3": torch.uint8, "int8": torch.int8}


def _check_caches(k_cache, v_cache, num_kv_heads: int, head_dim: int, dtype: torch.dtype):
    _need(k_cache.dim() == 4, "k_cache: expected [num_blocks, num_kv_heads, block_size, D]")
    _shape("v_cache", v_cache, k_cache.shape)
    if k_cache.shape[1] != num_kv_heads or k_cache.shape[3] != head_dim:
        raise ValueError(f"k_cache: shape {tuple(k_cache.shape)} does not hold {num_kv_heads} "
                         f"kv heads of dimension {head_dim}")
    _dtype("k_cache", k_cache, dtype)
    _dtype("v_cache", v_cache, dtype)


def _check_scales(k_scales, v_scales, k_cache):
    for name, t in (("k_scales", k_scales), ("v_scales", v_scales)):
        _shape(name, t, k_cache.shape[:3])
        _dtype(name, t, torch.float32)


def _check_decode_args(out, query, k_cache, v_cache, block_tables, context_lens,
                       num_kv_heads: int, cache_dtype: torch.dtype):
    _need(query.dim() == 3, "query: expected [num_seqs, num_heads, head_dim]")
    S, Hq, D = query.shape
    _shape("out", out, query.shape)
    _dtype("out", out, query.dtype)
    _check_caches(k_cache, v_cache, num_kv_heads, D, cache_dtype)
    if block_tables.dim() != 2 or block_tables.shape[0] != S:
        raise ValueError(f"block_tables: expected [{S}, max_blocks_per_seq]")
    _dtype("block_tables", block_tables, torch.int32)
    _shape("context_lens", context_lens, (S,))
    _dtype("context_lens", context_lens, torch.int32)


# the current device, and the current stream's handle without a Stream object around
# it (3 us less per call)
_raw_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream: Optional[torch.cuda.Stream]) -> int:
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is not None and torch.cuda.is_initialized():
        return _raw_stream(_raw_device())
    return torch.cuda.current_stream().cuda_stream


def _check(rc: int, what: str):
    if rc != 0:
        raise PagedAttentionError(rc, what)


def slot_mapping(out: torch.Tensor, block_tables: torch.Tensor, seq_idx: Optional[torch.Tensor],
                 positions: torch.Tensor, block_size: int, window: int = 0, stream=None):
    """pa_slot_mapping: out[t] = cache slot of token t (ring-aware)."""
    _on_device(out=out, block_tables=block_tables, seq_idx=seq_idx, positions=positions)
    _need(block_tables.dim() == 2, "block_tables: expected [num_seqs, max_blocks_per_seq]")
    _dtype("block_tables", block_tables, torch.int32)
    _dtype("positions", positions, torch.int32)
    _shape("out", out, (positions.numel(),))
    _dtype("out", out, torch.int64)
    if seq_idx is not None:
        _shape("seq_idx", seq_idx, (positions.numel(),))
        _dtype("seq_idx", seq_idx, torch.int32)
    S, MB = block_tables.shape
    _check(lib().pa_slot_mapping(_ptr(out), _ptr(block_tables), _ptr(seq_idx), _ptr(positions),
                                 positions.numel(), S, MB, block_size, window, _stream(stream)),
           "pa_slot_mapping")


def reshape_and_cache(key: torch.Tensor, value: torch.Tensor, k_cache: torch.Tensor,
                      v_cache: torch.Tensor, slot_mapping_: torch.Tensor, kv_dtype: str = "auto",
                      k_scale: float = 1.0, v_scale: float = 1.0, stream=None):
    """pa_reshape_and_cache: key/value [T, Hkv, D] into caches [NB, Hkv, bs, D]."""
    _on_device(key=key, value=value, k_cache=k_cache, v_cache=v_cache,
               slot_mapping=slot_mapping_)
    _need(key.dim() == 3, "key: expected [num_tokens, num_kv_heads, head_dim]")
    _shape("value", value, key.shape)
    _dtype("value", value, key.dtype)
    _check_caches(k_cache, v_cache, key.shape[1], key.shape[2],
                  _CACHE_DTYPE.get(kv_dtype, key.dtype))
    _shape("slot_mapping", slot_mapping_, (key.shape[0],))
    _dtype("slot_mapping", slot_mapping_, torch.int64)
    T, H, D = key.shape
    NB, _, bs, _ = k_cache.shape
    _check(lib().pa_reshape_and_cache(_ptr(key), _ptr(value), _ptr(k_cache), _ptr(v_cache),
                                      _ptr(slot_mapping_), T, H, D, bs, NB, _DTYPE[key.dtype],
                                      _KV[kv_dtype], k_scale, v_scale, _stream(stream)),
           "pa_reshape_and_cache")


def reshape_and_cache_int8(key: torch.Tensor, value: torch.Tensor, k_cache: torch.Tensor,
                           v_cache: torch.Tensor, k_scales: torch.Tensor, v_scales: torch.Tensor,
                           slot_mapping_: torch.Tensor, stream=None):
    """pa_reshape_and_cache_int8: key/value [T, Hkv, D] into int8 caches
    [NB, Hkv, bs, D] and fp32 row scales [NB, Hkv, bs]."""
    _on_device(key=key, value=value, k_cache=k_cache, v_cache=v_cache, k_scales=k_scales,
               v_scales=v_scales, slot_mapping=slot_mapping_)
    _need(key.dim() == 3, "key: expected [num_tokens, num_kv_heads, head_dim]")
    _shape("value", value, key.shape)
    _dtype("value", value, key.dtype)
    _check_caches(k_cache, v_cache, key.shape[1], key.shape[2], torch.int8)
    _check_scales(k_scales, v_scales, k_cache)
    _shape("slot_mapping", slot_mapping_, (key.shape[0],))
    _dtype("slot_mapping", slot_mapping_, torch.int64)
    T, H, D = key.shape
    NB, _, bs, _ = k_cache.shape
    _check(lib().pa_reshape_and_cache_int8(_ptr(key), _ptr(value), _ptr(k_cache), _ptr(v_cache),
                                           _ptr(k_scales), _ptr(v_scales), _ptr(slot_mapping_),
                                           T, H, D, bs, NB, _DTYPE[key.dtype], _stream(stream)),
           "pa_reshape_and_cache_int8")


def decode_int8(out: torch.Tensor, query: torch.Tensor, k_cache: torch.Tensor,
                v_cache: torch.Tensor, k_scales: torch.Tensor, v_scales: torch.Tensor,
                block_tables: torch.Tensor, context_lens: torch.Tensor, num_kv_heads: int,
                scale: float, window: int = 0, workspace: Optional[torch.Tensor] = None,
                stream=None):
    """pa_decode_int8: pa_decode over an INT8 cache with per-row scales."""
    _on_device(out=out, query=query, k_cache=k_cache, v_cache=v_cache, k_scales=k_scales,
               v_scales=v_scales, block_tables=block_tables, context_lens=context_lens,
               workspace=workspace)
    _check_decode_args(out, query, k_cache, v_cache, block_tables, context_lens, num_kv_heads,
                       torch.int8)
    _check_scales(k_scales, v_scales, k_cache)
    S, Hq, D = query.shape
    NB, _, bs, _ = k_cache.shape
    MB = block_tables.shape[1]
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().pa_decode_int8(_ptr(out), _ptr(query), _ptr(k_cache), _ptr(v_cache),
                                _ptr(k_scales), _ptr(v_scales), _ptr(block_tables),
                                _ptr(context_lens), S, Hq, num_kv_heads, D, bs, NB, MB, scale,
                                window, _DTYPE[query.dtype], _ptr(workspace), ws_bytes,
                                _stream(stream)), "pa_decode_int8")


def prefill(out: torch.Tensor, query: torch.Tensor, k_cache: torch.Tensor,
            v_cache: torch.Tensor, block_tables: torch.Tensor, cu_q: torch.Tensor,
            context_lens: torch.Tensor, num_kv_heads: int, max_q_len: int, scale: float,
            stream=None):
    """pa_prefill: causal attention of query [T, Hq, D] (the last tokens of each
    sequence's context, offsets cu_q [S + 1]) over the paged cache."""
    _on_device(out=out, query=query, k_cache=k_cache, v_cache=v_cache,
               block_tables=block_tables, cu_q=cu_q, context_lens=context_lens)
    _need(query.dim() == 3, "query: expected [num_tokens, num_heads, head_dim]")
    _shape("out", out, query.shape)
    _dtype("out", out, query.dtype)
    _check_caches(k_cache, v_cache, num_kv_heads, query.shape[2], query.dtype)
    _need(block_tables.dim() == 2, "block_tables: expected [num_seqs, max_blocks_per_seq]")
    _dtype("block_tables", block_tables, torch.int32)
    S = block_tables.shape[0]
    _shape("cu_q", cu_q, (S + 1,))
    _dtype("cu_q", cu_q, torch.int32)
    _shape("context_lens", context_lens, (S,))
    _dtype("context_lens", context_lens, torch.int32)
    T, Hq, D = query.shape
    NB, _, bs, _ = k_cache.shape
    S, MB = block_tables.shape
    _check(lib().pa_prefill(_ptr(out), _ptr(query), _ptr(k_cache), _ptr(v_cache),
                            _ptr(block_tables), _ptr(cu_q), _ptr(context_lens), T, S, Hq,
                            num_kv_heads, D, bs, NB, MB, max_q_len, scale, _DTYPE[query.dtype],
                            _stream(stream)), "pa_prefill")


def prefill_int8(out: torch.Tensor, query: torch.Tensor, k_cache: torch.Tensor,
                 v_cache: torch.Tensor, k_scales: torch.Tensor, v_scales: torch.Tensor,
                 block_tables: torch.Tensor, cu_q: torch.Tensor, context_lens: torch.Tensor,
                 num_kv_heads: int, max_q_len: int, scale: float, stream=None):
    """pa_prefill_int8: pa_prefill over an INT8 cache with per-row scales."""
    _on_device(out=out, query=query, k_cache=k_cache, v_cache=v_cache, k_scales=k_scales,
               v_scales=v_scales, block_tables=block_tables, cu_q=cu_q,
               context_lens=context_lens)
    _need(query.dim() == 3, "query: expected [num_tokens, num_heads, head_dim]")
    _shape("out", out, query.shape)
    _dtype("out", out, query.dtype)
    _check_caches(k_cache, v_cache, num_kv_heads, query.shape[2], torch.int8)
    _check_scales(k_scales, v_scales, k_cache)
    _need(block_tables.dim() == 2, "block_tables: expected [num_seqs, max_blocks_per_seq]")
    _dtype("block_tables", block_tables, torch.int32)
    S = block_tables.shape[0]
    _shape("cu_q", cu_q, (S + 1,))
    _dtype("cu_q", cu_q, torch.int32)
    _shape("context_lens", context_lens, (S,))
    _dtype("context_lens", context_lens, torch.int32)
    T, Hq, D = query.shape
    NB, _, bs, _ = k_cache.shape
    S, MB = block_tables.shape
    _check(lib().pa_prefill_int8(_ptr(out), _ptr(query), _ptr(k_cache), _ptr(v_cache),
                                 _ptr(k_scales), _ptr(v_scales), _ptr(block_tables), _ptr(cu_q),
                                 _ptr(context_lens), T, S, Hq, num_kv_heads, D, bs, NB, MB,
                                 max_q_len, scale, _DTYPE[query.dtype], _stream(stream)),
           "pa_prefill_int8")


def prefill_fp8(out: torch.Tensor, query: torch.Tensor, k_cache: torch.Tensor,
                v_cache: torch.Tensor, block_tables: torch.Tensor, cu_q: torch.Tensor,
                context_lens: torch.Tensor, num_kv_heads: int, max_q_len: int, scale: float,
                k_scale: float, v_scale: float, stream=None):
    """pa_prefill_fp8: pa_prefill over an FP8 E4M3 cache (uint8 codes) with
    per-tensor scales."""
    _on_device(out=out, query=query, k_cache=k_cache, v_cache=v_cache,
               block_tables=block_tables, cu_q=cu_q, context_lens=context_lens)
    _need(query.dim() == 3, "query: expected [num_tokens, num_heads, head_dim]")
    _shape("out", out, query.shape)
    _dtype("out", out, query.dtype)
    _check_caches(k_cache, v_cache, num_kv_heads, query.shape[2], torch.uint8)
    _need(block_tables.dim() == 2, "block_tables: expected [num_seqs, max_blocks_per_seq]")
    _dtype("block_tables", block_tables, torch.int32)
    S = block_tables.shape[0]
    _shape("cu_q", cu_q, (S + 1,))
    _dtype("cu_q", cu_q, torch.int32)
    _shape("context_lens", context_lens, (S,))
    _dtype("context_lens", context_lens, torch.int32)
    T, Hq, D = query.shape
    NB, _, bs, _ = k_cache.shape
    S, MB = block_tables.shape
    _check(lib().pa_prefill_fp8(_ptr(out), _ptr(query), _ptr(k_cache), _ptr(v_cache),
                                _ptr(block_tables), _ptr(cu_q), _ptr(context_lens), T, S, Hq,
                                num_kv_heads, D, bs, NB, MB, max_q_len, scale, k_scale, v_scale,
                                _DTYPE[query.dtype], _stream(stream)), "pa_prefill_fp8")


def decode_plan(num_seqs: int, num_heads: int, num_kv_heads: int, head_dim: int,
                block_size: int, max_blocks_per_seq: int, window: int = 0) -> Tuple[int, int]:
    """pa_decode_plan: (num_splits, pages_per_split)."""
    ns, pps = ctypes.c_int(), ctypes.c_int()
    _check(lib().pa_decode_plan(num_seqs, num_heads, num_kv_heads, head_dim, block_size,
                                max_blocks_per_seq, window, ctypes.addressof(ns),
                                ctypes.addressof(pps)), "pa_decode_plan")
    return ns.value, pps.value


def decode_workspace_size(num_seqs: int, num_heads: int, num_kv_heads: int, head_dim: int,
                          block_size: int, max_blocks_per_seq: int, window: int = 0) -> int:
    return int(lib().pa_decode_workspace_size(num_seqs, num_heads, num_kv_heads, head_dim,
                                              block_size, max_blocks_per_seq, window))


def decode(out: torch.Tensor, query: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
           block_tables: torch.Tensor, context_lens: torch.Tensor, num_kv_heads: int,
           scale: float, window: int = 0, kv_dtype: str = "auto", k_scale: float = 1.0,
           v_scale: float = 1.0, workspace: Optional[torch.Tensor] = None, stream=None):
    """pa_decode: out [S, Hq, D] = paged attention of query [S, Hq, D]."""
    _on_device(out=out, query=query, k_cache=k_cache, v_cache=v_cache,
               block_tables=block_tables, context_lens=context_lens, workspace=workspace)
    _check_decode_args(out, query, k_cache, v_cache, block_tables, context_lens, num_kv_heads,
                       _CACHE_DTYPE.get(kv_dtype, query.dtype))
    S, Hq, D = query.shape
    NB, _, bs, _ = k_cache.shape
    MB = block_tables.shape[1]
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().pa_decode(_ptr(out), _ptr(query), _ptr(k_cache), _ptr(v_cache),
                           _ptr(block_tables), _ptr(context_lens), S, Hq, num_kv_heads, D, bs, NB,
                           MB, scale, window, _DTYPE[query.dtype], _KV[kv_dtype], k_scale,
                           v_scale, _ptr(workspace), ws_bytes, _stream(stream)), "pa_decode")


def decode_balanced(out: torch.Tensor, query: torch.Tensor, k_cache: torch.Tensor,
                    v_cache: torch.Tensor, block_tables: torch.Tensor, context_lens: torch.Tensor,
                    num_kv_heads: int, scale: float, workspace: torch.Tensor, window: int = 0,
                    kv_dtype: str = "auto", k_scale: float = 1.0, v_scale: float = 1.0,
                    stream=None) -> int:
    """pa_decode_balanced: the balanced path's decode launch (arrival counters
    must be zero: see decode_workspace_clear); returns num_ctas."""
    _on_device(out=out, query=query, k_cache=k_cache, v_cache=v_cache,
               block_tables=block_tables, context_lens=context_lens, workspace=workspace)
    _check_decode_args(out, query, k_cache, v_cache, block_tables, context_lens, num_kv_heads,
                       _CACHE_DTYPE.get(kv_dtype, query.dtype))
    S, Hq, D = query.shape
    NB, _, bs, _ = k_cache.shape
    MB = block_tables.shape[1]
    n = ctypes.c_int()
    _check(lib().pa_decode_balanced(_ptr(out), _ptr(query), _ptr(k_cache), _ptr(v_cache),
                                    _ptr(block_tables), _ptr(context_lens), S, Hq, num_kv_heads,
                                    D, bs, NB, MB, scale, window, _DTYPE[query.dtype],
                                    _KV[kv_dtype], k_scale, v_scale, _ptr(workspace),
                                    workspace.numel() * workspace.element_size(),
                                    ctypes.addressof(n), _stream(stream)), "pa_decode_balanced")
    return n.value


def decode_workspace_clear(workspace: torch.Tensor, stream=None):
    """pa_decode_workspace_clear: zero the balanced path's arrival counters."""
    _on_device(workspace=workspace)
    _check(lib().pa_decode_workspace_clear(_ptr(workspace),
                                           workspace.numel() * workspace.element_size(),
                                           _stream(stream)), "pa_decode_workspace_clear")


def decode_cascade_workspace_size(num_seqs: int, num_heads: int, num_kv_heads: int,
                                  head_dim: int, block_size: int, prefix_pages: int) -> int:
    return int(lib().pa_decode_cascade_workspace_size(num_seqs, num_heads, num_kv_heads,
                                                      head_dim, block_size, prefix_pages))


def decode_cascade(out: torch.Tensor, query: torch.Tensor, k_cache: torch.Tensor,
                   v_cache: torch.Tensor, block_tables: torch.Tensor, context_lens: torch.Tensor,
                   num_kv_heads: int, scale: float, prefix_pages: int,
                   workspace: torch.Tensor, stream=None):
    """pa_decode_cascade: decode of a batch sharing its first prefix_pages blocks."""
    _on_device(out=out, query=query, k_cache=k_cache, v_cache=v_cache,
               block_tables=block_tables, context_lens=context_lens, workspace=workspace)
    _check_decode_args(out, query, k_cache, v_cache, block_tables, context_lens, num_kv_heads,
                       query.dtype)
    S, Hq, D = query.shape
    NB, _, bs, _ = k_cache.shape
    MB = block_tables.shape[1]
    _check(lib().pa_decode_cascade(_ptr(out), _ptr(query), _ptr(k_cache), _ptr(v_cache),
                                   _ptr(block_tables), _ptr(context_lens), S, Hq, num_kv_heads, D,
                                   bs, NB, MB, scale, _DTYPE[query.dtype], prefix_pages,
                                   _ptr(workspace), workspace.numel() * workspace.element_size(),
                                   _stream(stream)), "pa_decode_cascade")


def decode_cascade_fp8(out: torch.Tensor, query: torch.Tensor, k_cache: torch.Tensor,
                       v_cache: torch.Tensor, block_tables: torch.Tensor,
                       context_lens: torch.Tensor, num_kv_heads: int, scale: float,
                       k_scale: float, v_scale: float, prefix_pages: int,
                       workspace: torch.Tensor, stream=None):
    """pa_decode_cascade_fp8: pa_decode_cascade over an FP8 E4M3 cache (uint8
    codes) with per-tensor scales."""
    _on_device(out=out, query=query, k_cache=k_cache, v_cache=v_cache,
               block_tables=block_tables, context_lens=context_lens, workspace=workspace)
    _check_decode_args(out, query, k_cache, v_cache, block_tables, context_lens, num_kv_heads,
                       torch.uint8)
    S, Hq, D = query.shape
    NB, _, bs, _ = k_cache.shape
    MB = block_tables.shape[1]
    _check(lib().pa_decode_cascade_fp8(_ptr(out), _ptr(query), _ptr(k_cache), _ptr(v_cache),
                                       _ptr(block_tables), _ptr(context_lens), S, Hq,
                                       num_kv_heads, D, bs, NB, MB, scale, k_scale, v_scale,
                                       _DTYPE[query.dtype], prefix_pages, _ptr(workspace),
                                       workspace.numel() * workspace.element_size(),
                                       _stream(stream)), "pa_decode_cascade_fp8")


def decode_cascade_int8(out: torch.Tensor, query: torch.Tensor, k_cache: torch.Tensor,
                        v_cache: torch.Tensor, k_scales: torch.Tensor, v_scales: torch.Tensor,
                        block_tables: torch.Tensor, context_lens: torch.Tensor,
                        num_kv_heads: int, scale: float, prefix_pages: int,
                        workspace: torch.Tensor, stream=None):
    """pa_decode_cascade_int8: pa_decode_cascade over an INT8 cache with per-row
    scales."""
    _on_device(out=out, query=query, k_cache=k_cache, v_cache=v_cache, k_scales=k_scales,
               v_scales=v_scales, block_tables=block_tables, context_lens=context_lens,
               workspace=workspace)
    _check_decode_args(out, query, k_cache, v_cache, block_tables, context_lens, num_kv_heads,
                       torch.int8)
    _check_scales(k_scales, v_scales, k_cache)
    S, Hq, D = query.shape
    NB, _, bs, _ = k_cache.shape
    MB = block_tables.shape[1]
    _check(lib().pa_decode_cascade_int8(_ptr(out), _ptr(query), _ptr(k_cache), _ptr(v_cache),
                                        _ptr(k_scales), _ptr(v_scales), _ptr(block_tables),
                                        _ptr(context_lens), S, Hq, num_kv_heads, D, bs, NB, MB,
                                        scale, _DTYPE[query.dtype], prefix_pages,
                                        _ptr(workspace),
                                        workspace.numel() * workspace.element_size(),
                                        _stream(stream)), "pa_decode_cascade_int8")


def copy_blocks(k_cache: torch.Tensor, v_cache: torch.Tensor, block_pairs: torch.Tensor,
                stream=None):
    """pa_copy_blocks: block_pairs int32 [n, 2] = (source, destination)."""
    _on_device(k_cache=k_cache, v_cache=v_cache, block_pairs=block_pairs)
    _need(k_cache.dim() == 4, "k_cache: expected [num_blocks, num_kv_heads, block_size, D]")
    _shape("v_cache", v_cache, k_cache.shape)
    _dtype("v_cache", v_cache, k_cache.dtype)
    _need(block_pairs.dim() == 2 and block_pairs.shape[1] == 2, "block_pairs: expected [n, 2]")
    _dtype("block_pairs", block_pairs, torch.int32)
    NB, H, bs, D = k_cache.shape
    _check(lib().pa_copy_blocks(_ptr(k_cache), _ptr(v_cache), _ptr(block_pairs),
                                block_pairs.shape[0], H, D, bs, NB, k_cache.element_size(),
                                _stream(stream)), "pa_copy_blocks")


def _nbytes(t: torch.Tensor) -> int:
    return t.numel() * t.element_size()


def _pointers(stream, names: str, *tensors):
    """Device pointers of contiguous tensors on the current device, which is the
    one the library launches on (None where an optional one is missing). The
    names are for what is raised; they are not looked at otherwise."""
    cur = _raw_device() if torch.cuda.is_initialized() else -1
    out = []
    for t in tensors:
        if t is None:
            out.append(None)
        elif isinstance(t, torch.Tensor) and t.get_device() == cur >= 0 and t.is_contiguous():
            out.append(t.data_ptr())
        else:
            break
    if len(out) == len(tensors) and (stream is None or stream.device.index == cur):
        return out
    _on_device(**dict(zip(names.split(), tensors)))
    for t in tensors:
        if t is not None and t.is_cuda and t.device.index != torch.cuda.current_device():
            raise ValueError(f"tensors are on {t.device}, the current device is "
                             f"cuda:{torch.cuda.current_device()}")
    if stream is not None and stream.device.index != torch.cuda.current_device():
        raise ValueError(f"the stream is on {stream.device}, the current device is "
                         f"cuda:{torch.cuda.current_device()}")
    return [_ptr(t) for t in tensors]


def tree_mask_from_parents(parents, cu_q) -> torch.Tensor:
    """The tree mask of drafts given as parent indices, on the CPU.

    parents [T]: the node's parent within its own sequence's draft (an earlier
    node), or -1 for a child of the context's last token; cu_q [S + 1] the
    drafts' offsets. Returns int64 words [T, W], W = ceil(longest draft / 64):
    a node sees itself and its ancestors.
    """
    par = torch.as_tensor(parents).cpu().tolist()
    cu = torch.as_tensor(cu_q).cpu().tolist()
    _need(len(cu) >= 1 and cu[0] == 0 and cu[-1] == len(par) and
          all(a <= b for a, b in zip(cu, cu[1:])), "cu_q: expected offsets from 0 to len(parents)")
    words = max([1] + [-(-(b - a) // 64) for a, b in zip(cu, cu[1:])])
    out = torch.zeros(len(par), words, dtype=torch.int64)
    for a, b in zip(cu, cu[1:]):
        seen = []
        for i in range(b - a):
            p = par[a + i]
            _need(-1 <= p < i, f"parents[{a + i}] = {p}: expected -1 or an earlier node of the draft")
            seen.append((seen[p] if p >= 0 else 0) | 1 << i)
            for k in range(words):
                w = seen[i] >> (64 * k) & (1 << 64) - 1
                out[a + i, k] = w - (1 << 64) if w >> 63 else w
    return out


def tree_workspace_size(num_heads: int, num_kv_heads: int, head_dim: int) -> int:
    return int(lib().pa_tree_workspace_size(num_heads, num_kv_heads, head_dim))


def _check_tree_args(out, query, k_cache, v_cache, block_tables, cu_q, context_lens, tree_mask,
                     num_kv_heads: int, cache_dtype: torch.dtype):
    """Sizes (T, S, Hq, Hkv, D, bs, NB, MB) of consistent arguments; raises on others."""
    q, k, bt = query.shape, k_cache.shape, block_tables.shape
    if (len(q) == 3 and len(k) == 4 and len(bt) == 2 and out.shape == q and v_cache.shape == k and
            k[1] == num_kv_heads and k[3] == q[2] and cu_q.shape == (bt[0] + 1,) and
            context_lens.shape == (bt[0],) and tree_mask.dim() == 2 and
            tree_mask.shape[0] == q[0] and query.dtype in _DTYPE and
            out.dtype == query.dtype and k_cache.dtype == v_cache.dtype == cache_dtype and
            block_tables.dtype == cu_q.dtype == context_lens.dtype == torch.int32 and
            tree_mask.dtype == torch.int64):
        return q[0], bt[0], q[1], num_kv_heads, q[2], k[2], k[0], bt[1]
    _need(query.dim() == 3, "query: expected [num_tokens, num_heads, head_dim]")
    _shape("out", out, query.shape)
    _dtype("out", out, query.dtype)
    _need(query.dtype in _DTYPE, f"query: unsupported dtype {query.dtype}")
    _check_caches(k_cache, v_cache, num_kv_heads, query.shape[2], cache_dtype)
    _need(block_tables.dim() == 2, "block_tables: expected [num_seqs, max_blocks_per_seq]")
    _dtype("block_tables", block_tables, torch.int32)
    S = block_tables.shape[0]
    _shape("cu_q", cu_q, (S + 1,))
    _dtype("cu_q", cu_q, torch.int32)
    _shape("context_lens", context_lens, (S,))
    _dtype("context_lens", context_lens, torch.int32)
    _need(tree_mask.dim() == 2 and tree_mask.shape[0] == query.shape[0],
          "tree_mask: expected [num_tokens, mask_words]")
    _dtype("tree_mask", tree_mask, torch.int64)
    raise ValueError("inconsistent arguments")


_TREE = "out query k_cache v_cache block_tables cu_q context_lens tree_mask workspace"


def tree_attention(out: torch.Tensor, query: torch.Tensor, k_cache: torch.Tensor,
                   v_cache: torch.Tensor, block_tables: torch.Tensor, cu_q: torch.Tensor,
                   context_lens: torch.Tensor, tree_mask: torch.Tensor, num_kv_heads: int,
                   max_q_len: int, scale: float, workspace: torch.Tensor, stream=None):
    """pa_tree: attention of drafted nodes query [T, Hq, D] (offsets cu_q [S + 1],
    the last tokens of each sequence's context) to the context and to the nodes
    that tree_mask [T, W] (int64 words, see tree_mask_from_parents) names. max_q_len:
    the longest draft; a bound above it is allowed, but past 128 / (Hq / Hkv) nodes it
    chooses tiles that short drafts pay for."""
    *ptrs, ws = _pointers(stream, _TREE, out, query, k_cache, v_cache, block_tables, cu_q,
                          context_lens, tree_mask, workspace)
    sizes = _check_tree_args(out, query, k_cache, v_cache, block_tables, cu_q, context_lens,
                             tree_mask, num_kv_heads, query.dtype)
    _check(lib().pa_tree(*ptrs, *sizes, max_q_len, tree_mask.shape[1], scale,
                         _DTYPE[query.dtype], ws, _nbytes(workspace), _stream(stream)), "pa_tree")


def tree_attention_int8(out: torch.Tensor, query: torch.Tensor, k_cache: torch.Tensor,
                        v_cache: torch.Tensor, k_scales: torch.Tensor, v_scales: torch.Tensor,
                        block_tables: torch.Tensor, cu_q: torch.Tensor,
                        context_lens: torch.Tensor, tree_mask: torch.Tensor, num_kv_heads: int,
                        max_q_len: int, scale: float, workspace: torch.Tensor, stream=None):
    """pa_tree_int8: tree_attention over an INT8 cache with per-row scales."""
    *ptrs, ws = _pointers(stream, "out query k_cache v_cache k_scales v_scales block_tables cu_q "
                          "context_lens tree_mask workspace", out, query, k_cache, v_cache,
                          k_scales, v_scales, block_tables, cu_q, context_lens, tree_mask,
                          workspace)
    sizes = _check_tree_args(out, query, k_cache, v_cache, block_tables, cu_q, context_lens,
                             tree_mask, num_kv_heads, torch.int8)
    _check_scales(k_scales, v_scales, k_cache)
    _check(lib().pa_tree_int8(*ptrs, *sizes, max_q_len, tree_mask.shape[1], scale,
                              _DTYPE[query.dtype], ws, _nbytes(workspace), _stream(stream)),
           "pa_tree_int8")


def tree_attention_fp8(out: torch.Tensor, query: torch.Tensor, k_cache: torch.Tensor,
                       v_cache: torch.Tensor, block_tables: torch.Tensor, cu_q: torch.Tensor,
                       context_lens: torch.Tensor, tree_mask: torch.Tensor, num_kv_heads: int,
                       max_q_len: int, scale: float, k_scale: float, v_scale: float,
                       workspace: torch.Tensor, stream=None):
    """pa_tree_fp8: tree_attention over an FP8 E4M3 cache (uint8 codes) with
    per-tensor scales."""
    *ptrs, ws = _pointers(stream, _TREE, out, query, k_cache, v_cache, block_tables, cu_q,
                          context_lens, tree_mask, workspace)
    sizes = _check_tree_args(out, query, k_cache, v_cache, block_tables, cu_q, context_lens,
                             tree_mask, num_kv_heads, torch.uint8)
    _check(lib().pa_tree_fp8(*ptrs, *sizes, max_q_len, tree_mask.shape[1], scale, k_scale, v_scale,
                             _DTYPE[query.dtype], ws, _nbytes(workspace), _stream(stream)),
           "pa_tree_fp8")


def decode_scored_workspace_size(num_seqs: int, num_heads: int, num_kv_heads: int, head_dim: int,
                                 block_size: int, max_blocks_per_seq: int) -> int:
    return int(lib().pa_decode_scored_workspace_size(num_seqs, num_heads, num_kv_heads, head_dim,
                                                     block_size, max_blocks_per_seq))


def _check_scores(scores, num_seqs: int, num_kv_heads: int, length: int):
    _shape("scores", scores, (num_seqs, num_kv_heads, length))
    _dtype("scores", scores, torch.float32)


def _check_scored_args(out, scores, query, k_cache, v_cache, block_tables, context_lens,
                       num_kv_heads: int, cache_dtype: torch.dtype):
    """Sizes (S, Hq, Hkv, D, bs, NB, MB) of consistent arguments; raises on others."""
    q, k, bt = query.shape, k_cache.shape, block_tables.shape
    if (len(q) == 3 and len(k) == 4 and len(bt) == 2 and out.shape == q and v_cache.shape == k and
            k[1] == num_kv_heads and k[3] == q[2] and bt[0] == q[0] and
            context_lens.shape == (q[0],) and scores.shape == (q[0], k[1], bt[1] * k[2]) and
            scores.dtype == torch.float32 and query.dtype in _DTYPE and
            out.dtype == query.dtype and
            k_cache.dtype == v_cache.dtype == cache_dtype and
            block_tables.dtype == context_lens.dtype == torch.int32):
        return q[0], q[1], num_kv_heads, q[2], k[2], k[0], bt[1]
    _check_decode_args(out, query, k_cache, v_cache, block_tables, context_lens, num_kv_heads,
                       cache_dtype)
    _check_scores(scores, q[0], num_kv_heads, bt[1] * k[2])
    _need(query.dtype in _DTYPE, f"query: unsupported dtype {query.dtype}")
    raise ValueError("inconsistent arguments")


def decode_scored(out: torch.Tensor, scores: torch.Tensor, query: torch.Tensor,
                  k_cache: torch.Tensor, v_cache: torch.Tensor, block_tables: torch.Tensor,
                  context_lens: torch.Tensor, num_kv_heads: int, scale: float,
                  workspace: torch.Tensor, kv_dtype: str = "auto", k_scale: float = 1.0,
                  v_scale: float = 1.0, stream=None):
    """pa_decode_scored: decode (up to rounding: the sum takes unrounded weights), and
    scores [S, Hkv, MB * bs] += every token's softmax weight summed over its kv head's
    query heads."""
    *ptrs, ws = _pointers(stream, "out scores query k_cache v_cache block_tables context_lens "
                          "workspace", out, scores, query, k_cache, v_cache, block_tables,
                          context_lens, workspace)
    sizes = _check_scored_args(out, scores, query, k_cache, v_cache, block_tables, context_lens,
                               num_kv_heads, _CACHE_DTYPE.get(kv_dtype, query.dtype))
    _check(lib().pa_decode_scored(*ptrs, *sizes, scale, _DTYPE[query.dtype], _KV[kv_dtype],
                                  k_scale, v_scale, ws, _nbytes(workspace), _stream(stream)),
           "pa_decode_scored")


def decode_scored_int8(out: torch.Tensor, scores: torch.Tensor, query: torch.Tensor,
                       k_cache: torch.Tensor, v_cache: torch.Tensor, k_scales: torch.Tensor,
                       v_scales: torch.Tensor, block_tables: torch.Tensor,
                       context_lens: torch.Tensor, num_kv_heads: int, scale: float,
                       workspace: torch.Tensor, stream=None):
    """pa_decode_scored_int8: decode_scored over an INT8 cache with per-row scales."""
    *ptrs, ws = _pointers(stream, "out scores query k_cache v_cache k_scales v_scales "
                          "block_tables context_lens workspace", out, scores, query, k_cache,
                          v_cache, k_scales, v_scales, block_tables, context_lens, workspace)
    sizes = _check_scored_args(out, scores, query, k_cache, v_cache, block_tables, context_lens,
                               num_kv_heads, torch.int8)
    _check_scales(k_scales, v_scales, k_cache)
    _check(lib().pa_decode_scored_int8(*ptrs, *sizes, scale, _DTYPE[query.dtype], ws,
                                       _nbytes(workspace), _stream(stream)),
           "pa_decode_scored_int8")


def evict_select(keep: torch.Tensor, new_lens: torch.Tensor, scores: torch.Tensor,
                 context_lens: torch.Tensor, num_sink: int = 0, num_recent: int = 0, stream=None):
    """pa_evict_select: keep [S, Hkv, budget] = the ascending positions an
    eviction to `budget` tokens keeps (-1 past new_lens [S])."""
    ptrs = _pointers(stream, "keep new_lens scores context_lens", keep, new_lens, scores,
                     context_lens)
    sc, kp = scores.shape, keep.shape
    if not (len(sc) == len(kp) == 3 and kp[0] == sc[0] and kp[1] == sc[1] and
            new_lens.shape == context_lens.shape == sc[:1] and scores.dtype == torch.float32 and
            keep.dtype == new_lens.dtype == context_lens.dtype == torch.int32):
        _need(len(sc) == 3, "scores: expected [num_seqs, num_kv_heads, length]")
        _dtype("scores", scores, torch.float32)
        _need(len(kp) == 3 and kp[:2] == sc[:2], "keep: expected [num_seqs, num_kv_heads, budget]")
        _dtype("keep", keep, torch.int32)
        for name, t in (("new_lens", new_lens), ("context_lens", context_lens)):
            _shape(name, t, sc[:1])
            _dtype(name, t, torch.int32)
        raise ValueError("inconsistent arguments")
    _check(lib().pa_evict_select(*ptrs, *sc, kp[2], num_sink, num_recent, _stream(stream)),
           "pa_evict_select")


def compact(k_cache: torch.Tensor, v_cache: torch.Tensor, block_tables: torch.Tensor,
            context_lens: torch.Tensor, keep: torch.Tensor, keep_lens: torch.Tensor,
            starts: Optional[torch.Tensor] = None, k_scales: Optional[torch.Tensor] = None,
            v_scales: Optional[torch.Tensor] = None, scores: Optional[torch.Tensor] = None,
            stream=None):
    """pa_compact: row starts[s] + j of sequence s <- row keep[s, g, j] for
    j < keep_lens[s], in place (keep [S, Hkv or 1, budget])."""
    ptrs = _pointers(stream, "k_cache v_cache k_scales v_scales scores block_tables context_lens "
                     "keep keep_lens starts", k_cache, v_cache, k_scales, v_scales, scores,
                     block_tables, context_lens, keep, keep_lens, starts)
    k, bt, kp = k_cache.shape, block_tables.shape, keep.shape
    if not (len(k) == 4 and len(bt) == 2 and len(kp) == 3 and v_cache.shape == k and
            v_cache.dtype == k_cache.dtype and kp[0] == bt[0] and kp[1] in (1, k[1]) and
            context_lens.shape == keep_lens.shape == bt[:1] and
            (starts is None or starts.shape == bt[:1] and starts.dtype == torch.int32) and
            block_tables.dtype == keep.dtype == context_lens.dtype == keep_lens.dtype ==
            torch.int32):
        _need(len(k) == 4, "k_cache: expected [num_blocks, num_kv_heads, block_size, D]")
        _shape("v_cache", v_cache, k)
        _dtype("v_cache", v_cache, k_cache.dtype)
        _need(len(bt) == 2, "block_tables: expected [num_seqs, max_blocks_per_seq]")
        _dtype("block_tables", block_tables, torch.int32)
        _need(len(kp) == 3 and kp[0] == bt[0] and kp[1] in (1, k[1]),
              f"keep: expected [{bt[0]}, {k[1]} or 1, budget]")
        _dtype("keep", keep, torch.int32)
        for name, t in (("context_lens", context_lens), ("keep_lens", keep_lens),
                        ("starts", starts)):
            if t is not None:
                _shape(name, t, bt[:1])
                _dtype(name, t, torch.int32)
        raise ValueError("inconsistent arguments")
    _need((k_scales is None) == (v_scales is None), "give both row scales or neither")
    if k_scales is not None:
        _check_scales(k_scales, v_scales, k_cache)
    if scores is not None:
        _check_scores(scores, bt[0], k[1], bt[1] * k[2])
    _check(lib().pa_compact(*ptrs, bt[0], k[1], kp[1], kp[2], k[3], k[2], k[0], bt[1],
                            k_cache.element_size(), _stream(stream)), "pa_compact")


def rope_turns(inv_freq, device=None) -> torch.Tensor:
    """The `turns` of norm_rope from frequencies in radians per position.

    inv_freq [R / 2], or [A, R / 2] for positions of A axes (0 where an axis does not turn a
    pair), taken in 64 bits (an angle is off by about 2^-54 of a turn a position). Returns int64
    [A, R / 2] on `device` (inv_freq's by default): the fraction of a turn per position in units
    of 2^-64. Made once, as weights are.
    """
    try:
        f = torch.as_tensor(inv_freq)
    except (TypeError, RuntimeError) as e:
        raise ValueError("inv_freq: expected numbers") from e
    _need(not f.is_complex(), "inv_freq: expected real numbers")
    _need(f.dim() in (1, 2), "inv_freq: expected [rot_dim / 2] or [num_axes, rot_dim / 2]")
    f = f[None] if f.dim() == 1 else f
    dev = f.device if device is None else device
    f = f.detach().to("cpu", torch.float64)
    _need(bool(torch.isfinite(f).all()), "inv_freq: expected finite numbers")
    # the fraction of a turn in [-1/2, 1/2], as two whole numbers of 32 bits (a double holds
    # each exactly)
    part = f / (2.0 * math.pi)
    part = (part - part.round()) * 2.0 ** 32
    high = part.floor()
    low = ((part - high) * 2.0 ** 32).floor()
    turns = (high.to(torch.int64) << 32) + low.to(torch.int64)
    return turns.to(dev).contiguous()


def _heads(name: str, t) -> torch.Tensor:
    """t [num_tokens, heads, head_dim] with its heads dense (tokens may be strided)."""
    _need(isinstance(t, torch.Tensor) and t.dim() == 3,
          f"{name}: expected a tensor [num_tokens, heads, head_dim]")
    D = t.shape[2]
    _need((t.stride(2) == 1 or D == 1) and (t.stride(1) == D or t.shape[1] == 1),
          f"{name}: the heads of a token must be contiguous")
    return t


def _token_stride(t: torch.Tensor) -> int:
    """Elements between tokens (one token: its own size)."""
    return t.stride(0) if t.shape[0] > 1 else t.shape[1] * t.shape[2]


def _rope_args(query, key, q_weight, k_weight, turns, positions):
    """(T, Hq, Hkv, D, R, A) of consistent arguments; raises on others."""
    T, Hq, D = query.shape
    _need(key.shape[0] == T and key.shape[2] == D,
          f"key: shape {tuple(key.shape)}, expected {T} tokens of head_dim {D}")
    _need(query.dtype in _DTYPE, f"query: unsupported dtype {query.dtype}")
    _dtype("key", key, query.dtype)
    for name, w in (("q_weight", q_weight), ("k_weight", k_weight)):
        if w is not None:
            _shape(name, w, (D,))
            _dtype(name, w, torch.float32)
    _need(turns.dim() == 2, "turns: expected [num_axes, rot_dim / 2]")
    _dtype("turns", turns, torch.int64)
    A = turns.shape[0]
    _need(positions.shape == (A, T) or (A == 1 and positions.shape == (T,)),
          f"positions: shape {tuple(positions.shape)}, expected [{A}, {T}]")
    _dtype("positions", positions, torch.int32)
    return T, Hq, key.shape[1], D, 2 * turns.shape[1], A


# what the checks run into where an argument is no tensor or has too few dimensions
_MISFITS = (AttributeError, IndexError, TypeError)


def _misfit(names: str, *tensors) -> ValueError:
    """What is raised then (a norm's weight may be missing)."""
    for name, t in zip(names.split(), tensors):
        if not isinstance(t, torch.Tensor) and not (t is None and name.endswith("_weight")):
            return ValueError(f"{name}: expected a torch tensor")
    return ValueError(f"too few dimensions among {names}")


def _strided(stream, names: str, *tensors):
    """Device pointers of tensors on the current device, whatever their strides (None where an
    optional one is missing)."""
    cur = _raw_device() if torch.cuda.is_initialized() else -1
    if cur >= 0 and (stream is None or stream.device.index == cur):
        out = [None if t is None else t.data_ptr() if t.get_device() == cur else -1
               for t in tensors]
        if -1 not in out:
            return out
    _pointers(stream, names, *(t.new_empty(0) if isinstance(t, torch.Tensor) else t
                               for t in tensors))
    raise ValueError("tensors are not on the current device")


def _dense_heads(t, shape, dtype) -> int:
    """Elements between the tokens of t [T, heads, D] (one token: its own size) where it has that
    shape and type and its heads are dense, else 0."""
    if t.shape != shape or t.dtype is not dtype:
        return 0
    st, D = t.stride(), shape[2]
    if st[2] != 1 or st[1] != D and shape[1] != 1:
        return 0
    return st[0] if shape[0] > 1 else shape[1] * D


def _rope_sizes(query, key, out, other, name, q_weight, k_weight, turns, positions):
    """(T, Hq, Hkv, D, R, A) of consistent arguments, and the token strides of query, key, out
    (q_out) and other (`name`: k_out or value); raises on others."""
    q, k, tu, dtype, f32 = query.shape, key.shape, turns.shape, query.dtype, torch.float32
    if len(q) == len(k) == 3 and len(tu) == 2 and k[0] == q[0] and k[2] == q[2] and dtype in _DTYPE:
        strides = (_dense_heads(query, q, dtype), _dense_heads(key, k, dtype),
                   _dense_heads(out, q, dtype), _dense_heads(other, k, dtype))
        if (0 not in strides and
                (q_weight is None or q_weight.shape == q[2:] and q_weight.dtype is f32 and
                 q_weight.is_contiguous()) and
                (k_weight is None or k_weight.shape == q[2:] and k_weight.dtype is f32 and
                 k_weight.is_contiguous()) and
                turns.dtype is torch.int64 and turns.is_contiguous() and
                positions.dtype is torch.int32 and positions.is_contiguous() and
                (positions.shape == (tu[0], q[0]) or tu[0] == 1 and positions.shape == q[:1])):
            return (q[0], q[1], k[1], q[2], 2 * tu[1], tu[0]), strides
    _heads("query", query)
    _heads("key", key)
    sizes = _rope_args(query, key, q_weight, k_weight, turns, positions)
    for n, t, like in (("q_out", out, query), (name, other, key)):
        _heads(n, t)
        _shape(n, t, like.shape)
        _dtype(n, t, dtype)
    for n, t in (("q_weight", q_weight), ("k_weight", k_weight), ("turns", turns),
                 ("positions", positions)):
        _need(t is None or t.is_contiguous(), f"{n}: must be contiguous")
    return sizes, tuple(_token_stride(t) for t in (query, key, out, other))


_ROPE = "q_out k_out query key q_weight k_weight turns positions"
_ROPE_STORE = ("q_out query key value k_cache v_cache slot_mapping q_weight k_weight turns "
               "positions")


def norm_rope(q_out: torch.Tensor, k_out: torch.Tensor, query: torch.Tensor, key: torch.Tensor,
              turns: torch.Tensor, positions: torch.Tensor,
              q_weight: Optional[torch.Tensor] = None, k_weight: Optional[torch.Tensor] = None,
              eps: float = 1e-6, interleaved: bool = False, stream=None):
    """pa_norm_rope: the norm of every head of query [T, Hq, D] and key [T, Hkv, D] (weights
    fp32 [D], None: no norm) and the rotation of its first R dims by positions int32 [A, T]
    ([T] for one axis) with turns [A, R / 2] (see rope_turns); pairs (i, i + R / 2), or with
    interleaved (2i, 2i + 1). Tokens may be strided (views of one projection's output); the
    outputs may be the inputs."""
    args = q_out, k_out, query, key, q_weight, k_weight, turns, positions
    try:
        sizes, (sq, sk, sqo, sko) = _rope_sizes(query, key, q_out, k_out, "k_out", q_weight,
                                                k_weight, turns, positions)
        ptrs = _strided(stream, _ROPE, *args)
    except _MISFITS as e:
        raise _misfit(_ROPE, *args) from e
    _check(lib().pa_norm_rope(*ptrs, *sizes, sqo, sko, sq, sk, eps, interleaved,
                              _DTYPE[query.dtype], _stream(stream)), "pa_norm_rope")


def norm_rope_and_cache(q_out: torch.Tensor, query: torch.Tensor, key: torch.Tensor,
                        value: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                        slot_mapping_: torch.Tensor, turns: torch.Tensor,
                        positions: torch.Tensor, q_weight: Optional[torch.Tensor] = None,
                        k_weight: Optional[torch.Tensor] = None, eps: float = 1e-6,
                        interleaved: bool = False, kv_dtype: str = "auto", k_scale: float = 1.0,
                        v_scale: float = 1.0, stream=None):
    """pa_norm_rope_and_cache: norm_rope whose keys go, with value [T, Hkv, D], to their cache
    slots (as reshape_and_cache after it, bit for bit)."""
    args = (q_out, query, key, value, k_cache, v_cache, slot_mapping_, q_weight, k_weight, turns,
            positions)
    try:
        sizes, (sq, sk, sqo, sv) = _rope_sizes(query, key, q_out, value, "value", q_weight,
                                               k_weight, turns, positions)
        kc, stored = k_cache.shape, torch.uint8 if kv_dtype == "fp8_e4m3" else key.dtype
        if not (kv_dtype in ("auto", "fp8_e4m3") and len(kc) == 4 and v_cache.shape == kc and
                kc[1] == sizes[2] and kc[3] == sizes[3] and
                k_cache.dtype is v_cache.dtype is stored and
                slot_mapping_.shape == query.shape[:1] and slot_mapping_.dtype is torch.int64 and
                k_cache.is_contiguous() and v_cache.is_contiguous() and
                slot_mapping_.is_contiguous()):
            _need(kv_dtype in ("auto", "fp8_e4m3"),
                  f"kv_dtype: {kv_dtype!r} is not 'auto' or 'fp8_e4m3'")
            _check_caches(k_cache, v_cache, sizes[2], sizes[3], stored)
            _shape("slot_mapping", slot_mapping_, query.shape[:1])
            _dtype("slot_mapping", slot_mapping_, torch.int64)
            raise ValueError("k_cache, v_cache, slot_mapping: must be contiguous")
        ptrs = _strided(stream, _ROPE_STORE, *args)
    except _MISFITS as e:
        raise _misfit(_ROPE_STORE, *args) from e
    _check(lib().pa_norm_rope_and_cache(*ptrs, *sizes, kc[2], kc[0], sqo, sq, sk, sv, eps,
                                        interleaved, _DTYPE[query.dtype], _KV[kv_dtype], k_scale,
                                        v_scale, _stream(stream)), "pa_norm_rope_and_cache")


def _check_page_scales(k_scales, v_scales, k_cache):
    for name, t in (("k_scales", k_scales), ("v_scales", v_scales)):
        _shape(name, t, k_cache.shape[:2])
        _dtype(name, t, torch.float32)


def _block_args(k_cache, v_cache, k_scales, v_scales, block_tables, context_lens, num_kv_heads: int,
                head_dim: int, cu_q=...):
    """(NB, bs, S, MB) of a consistent block-scaled cache and its tables (with offsets, where
    the call has them); raises on others."""
    k, bt, i32 = k_cache.shape, block_tables.shape, torch.int32
    if (len(k) == 4 and len(bt) == 2 and k[1] == num_kv_heads and k[3] == head_dim and
            v_cache.shape == k and k_cache.dtype is v_cache.dtype is torch.uint8 and
            k_scales.shape == v_scales.shape == k[:2] and
            k_scales.dtype is v_scales.dtype is torch.float32 and
            context_lens.shape == bt[:1] and block_tables.dtype is context_lens.dtype is i32 and
            (cu_q is ... or cu_q.dtype is i32 and cu_q.shape == (bt[0] + 1,) and
             cu_q.is_contiguous()) and
            k_cache.is_contiguous() and v_cache.is_contiguous() and k_scales.is_contiguous() and
            v_scales.is_contiguous() and block_tables.is_contiguous() and
            context_lens.is_contiguous()):
        return k[0], k[2], bt[0], bt[1]
    _check_caches(k_cache, v_cache, num_kv_heads, head_dim, torch.uint8)
    _check_page_scales(k_scales, v_scales, k_cache)
    _need(len(bt) == 2, "block_tables: expected [num_seqs, max_blocks_per_seq]")
    _dtype("block_tables", block_tables, torch.int32)
    if cu_q is not ...:
        _shape("cu_q", cu_q, (bt[0] + 1,))
        _dtype("cu_q", cu_q, torch.int32)
    _shape("context_lens", context_lens, bt[:1])
    _dtype("context_lens", context_lens, torch.int32)
    raise ValueError("caches, scales, tables, offsets and lengths must be contiguous")


_BLOCK_CACHE = "k_cache v_cache k_scales v_scales block_tables"
_BLOCK_APPEND = "key value " + _BLOCK_CACHE + " cu_q context_lens"
_BLOCK_DECODE = "out query " + _BLOCK_CACHE + " context_lens workspace"
_BLOCK_PREFILL = "out query " + _BLOCK_CACHE + " cu_q context_lens workspace"


def append_fp8_block(key: torch.Tensor, value: torch.Tensor, k_cache: torch.Tensor,
                     v_cache: torch.Tensor, k_scales: torch.Tensor, v_scales: torch.Tensor,
                     block_tables: torch.Tensor, cu_q: torch.Tensor, context_lens: torch.Tensor,
                     stream=None):
    """pa_append_fp8_block: key / value [T, Hkv, D] (offsets cu_q [S + 1], the last tokens of
    each sequence's context; tokens may be strided) into FP8 E4M3 caches (uint8 codes) with a
    scale per block and kv head (fp32 [NB, Hkv])."""
    args = (key, value, k_cache, v_cache, k_scales, v_scales, block_tables, cu_q, context_lens)
    try:
        kv, dtype = key.shape, key.dtype
        ok = len(kv) == 3 and dtype in _DTYPE
        sk, sv = (_dense_heads(key, kv, dtype), _dense_heads(value, kv, dtype)) if ok else (0, 0)
        if not (sk and sv):
            _heads("key", key)
            _heads("value", value)
            _need(dtype in _DTYPE, f"key: unsupported dtype {dtype}")
            _shape("value", value, kv)
            _dtype("value", value, dtype)
        NB, bs, S, MB = _block_args(k_cache, v_cache, k_scales, v_scales, block_tables,
                                    context_lens, kv[1], kv[2], cu_q)
        ptrs = _strided(stream, _BLOCK_APPEND, *args)
    except _MISFITS as e:
        raise _misfit(_BLOCK_APPEND, *args) from e
    _check(lib().pa_append_fp8_block(*ptrs, kv[0], S, kv[1], kv[2], bs, NB, MB, sk, sv,
                                     _DTYPE[dtype], _stream(stream)), "pa_append_fp8_block")


def decode_fp8_block(out: torch.Tensor, query: torch.Tensor, k_cache: torch.Tensor,
                     v_cache: torch.Tensor, k_scales: torch.Tensor, v_scales: torch.Tensor,
                     block_tables: torch.Tensor, context_lens: torch.Tensor, num_kv_heads: int,
                     scale: float, workspace: torch.Tensor, stream=None):
    """pa_decode_fp8_block: decode over the cache of append_fp8_block (workspace:
    decode_workspace_size bytes)."""
    args = (out, query, k_cache, v_cache, k_scales, v_scales, block_tables, context_lens, workspace)
    try:
        *ptrs, ws = _strided(stream, _BLOCK_DECODE, *args)
        q = query.shape
        NB, bs, S, MB = _block_args(k_cache, v_cache, k_scales, v_scales, block_tables,
                                    context_lens, num_kv_heads, q[-1])
        if not (len(q) == 3 and q[0] == S and out.shape == q and query.dtype in _DTYPE and
                out.dtype is query.dtype and out.is_contiguous() and query.is_contiguous() and
                workspace.is_contiguous()):
            _check_decode_args(out, query, k_cache, v_cache, block_tables, context_lens,
                               num_kv_heads, torch.uint8)
            _need(query.dtype in _DTYPE, f"query: unsupported dtype {query.dtype}")
            raise ValueError("out, query, workspace: must be contiguous")
    except _MISFITS as e:
        raise _misfit(_BLOCK_DECODE, *args) from e
    _check(lib().pa_decode_fp8_block(*ptrs, S, q[1], num_kv_heads, q[2], bs, NB, MB, scale,
                                     _DTYPE[query.dtype], ws, _nbytes(workspace),
                                     _stream(stream)), "pa_decode_fp8_block")


def prefill_fp8_block_workspace_size(num_heads: int, num_kv_heads: int, head_dim: int) -> int:
    return int(lib().pa_prefill_fp8_block_workspace_size(num_heads, num_kv_heads, head_dim))


def prefill_fp8_block(out: torch.Tensor, query: torch.Tensor, k_cache: torch.Tensor,
                      v_cache: torch.Tensor, k_scales: torch.Tensor, v_scales: torch.Tensor,
                      block_tables: torch.Tensor, cu_q: torch.Tensor, context_lens: torch.Tensor,
                      num_kv_heads: int, max_q_len: int, scale: float, workspace: torch.Tensor,
                      stream=None):
    """pa_prefill_fp8_block: causal attention of query [T, Hq, D] (the last tokens of each
    sequence's context, offsets cu_q [S + 1]) over the cache of append_fp8_block."""
    args = (out, query, k_cache, v_cache, k_scales, v_scales, block_tables, cu_q, context_lens,
            workspace)
    try:
        *ptrs, ws = _strided(stream, _BLOCK_PREFILL, *args)
        q = query.shape
        if not (len(q) == 3 and out.shape == q and query.dtype in _DTYPE and
                out.dtype is query.dtype and out.is_contiguous() and query.is_contiguous() and
                workspace.is_contiguous()):
            _need(len(q) == 3, "query: expected [num_tokens, num_heads, head_dim]")
            _shape("out", out, q)
            _dtype("out", out, query.dtype)
            _need(query.dtype in _DTYPE, f"query: unsupported dtype {query.dtype}")
            raise ValueError("out, query, workspace: must be contiguous")
        NB, bs, S, MB = _block_args(k_cache, v_cache, k_scales, v_scales, block_tables,
                                    context_lens, num_kv_heads, q[2], cu_q)
    except _MISFITS as e:
        raise _misfit(_BLOCK_PREFILL, *args) from e
    _check(lib().pa_prefill_fp8_block(*ptrs, q[0], S, q[1], num_kv_heads, q[2], bs, NB, MB,
                                      max_q_len, scale, _DTYPE[query.dtype], ws,
                                      _nbytes(workspace), _stream(stream)),
           "pa_prefill_fp8_block")


PA_BUDGET_MB, PA_BUDGET_FRACTION, PA_BUDGET_CONTEXT = 0, 1, 2


def block_budget(num_layers: int, num_kv_heads: int, head_dim: int, block_size: int,
                 dtype: torch.dtype, kv_dtype: str = "auto", *, mb: Optional[float] = None,
                 fraction: Optional[float] = None, context_tokens: Optional[int] = None,
                 available_bytes: Optional[int] = None) -> int:
    """pa_block_budget: cache blocks for a budget given as exactly one of mb,
    fraction (of available_bytes, by default the device's free memory) or
    context_tokens."""
    given = [x is not None for x in (mb, fraction, context_tokens)]
    if sum(given) != 1:
        raise ValueError("give exactly one of mb, fraction, context_tokens")
    if fraction is not None and available_bytes is None:
        available_bytes = torch.cuda.mem_get_info()[0]
    kind, amount = ((PA_BUDGET_MB, mb) if mb is not None else
                    (PA_BUDGET_FRACTION, fraction) if fraction is not None else
                    (PA_BUDGET_CONTEXT, context_tokens))
    n = lib().pa_block_budget(kind, float(amount), int(available_bytes or 0), num_layers,
                              num_kv_heads, head_dim, block_size, _DTYPE[dtype], _KV[kv_dtype])
    if n < 0:
        raise PagedAttentionError(int(n), "pa_block_budget")
    return int(n)


def decode_partials(tmp_out: torch.Tensor, max_logits: torch.Tensor, exp_sums: torch.Tensor,
                    query: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                    block_tables: torch.Tensor, context_lens: torch.Tensor, num_kv_heads: int,
                    scale: float, num_splits: int, pages_per_split: int, window: int = 0,
                    kv_dtype: str = "auto", k_scale: float = 1.0, v_scale: float = 1.0,
                    stream=None):
    """pa_decode_partials: split partials tmp_out [S, Hq, NS, D], max_logits and
    exp_sums [S, Hq, NS]."""
    _on_device(tmp_out=tmp_out, max_logits=max_logits, exp_sums=exp_sums, query=query,
               k_cache=k_cache, v_cache=v_cache, block_tables=block_tables,
               context_lens=context_lens)
    _check_decode_args(query, query, k_cache, v_cache, block_tables, context_lens, num_kv_heads,
                       _CACHE_DTYPE.get(kv_dtype, query.dtype))
    S, Hq, D = query.shape
    _shape("tmp_out", tmp_out, (S, Hq, num_splits, D))
    for name, t in (("max_logits", max_logits), ("exp_sums", exp_sums)):
        _shape(name, t, (S, Hq, num_splits))
        _dtype(name, t, torch.float32)
    _dtype("tmp_out", tmp_out, torch.float32)
    NB, _, bs, _ = k_cache.shape
    MB = block_tables.shape[1]
    _check(lib().pa_decode_partials(_ptr(tmp_out), _ptr(max_logits), _ptr(exp_sums),
                                    _ptr(query), _ptr(k_cache), _ptr(v_cache),
                                    _ptr(block_tables), _ptr(context_lens), S, Hq, num_kv_heads,
                                    D, bs, NB, MB, scale, window, _DTYPE[query.dtype],
                                    _KV[kv_dtype], k_scale, v_scale, num_splits,
                                    pages_per_split, _stream(stream)), "pa_decode_partials")


def reduce(out: torch.Tensor, tmp_out: torch.Tensor, max_logits: torch.Tensor,
           exp_sums: torch.Tensor, stream=None):
    """pa_reduce: LSE combination of [S, Hq, NS, D] partials into out [S, Hq, D]."""
    _on_device(out=out, tmp_out=tmp_out, max_logits=max_logits, exp_sums=exp_sums)
    _need(tmp_out.dim() == 4, "tmp_out: expected [num_seqs, num_heads, num_splits, D]")
    S, Hq, NS, D = tmp_out.shape
    _shape("out", out, (S, Hq, D))
    _dtype("tmp_out", tmp_out, torch.float32)
    for name, t in (("max_logits", max_logits), ("exp_sums", exp_sums)):
        _shape(name, t, (S, Hq, NS))
        _dtype(name, t, torch.float32)
    _check(lib().pa_reduce(_ptr(out), _ptr(tmp_out), _ptr(max_logits), _ptr(exp_sums), S, Hq,
                           D, NS, _DTYPE[out.dtype], _stream(stream)), "pa_reduce")


def test_set_unarmed_page(page: int) -> None:
    """pa_test_set_unarmed_page: test hook; the producer of every CTA of later
    decodes stops before arming its page number ``page`` (negative: off)."""
    lib().pa_test_set_unarmed_page(int(page))


def get_device_error(stream=None) -> int:
    """pa_get_device_error: synchronise, return and clear the device error bits."""
    bits = ctypes.c_uint32()
    rc = lib().pa_get_device_error(_stream(stream), ctypes.addressof(bits))
    if rc not in (0, PA_ERR_DEVICE):
        raise PagedAttentionError(rc, "pa_get_device_error")
    return bits.value
