"""Thin Python binding of ``libckv.so`` (argument marshalling only).

Every function here has the name of the C entry point it calls (include/ckv.h)
and takes torch tensors; it checks dtypes/devices, passes raw pointers, sizes
and the current CUDA stream, and raises ``CkvError`` on a nonzero status.  All
arithmetic happens in the CUDA kernels; there is no fallback: if the library
is missing or the tensors are not on a CUDA device, the call fails.
"""
from __future__ import annotations

import contextlib
import ctypes
import importlib.machinery
import importlib.util
import os
import threading

import torch

from . import build as _build

_lock = threading.Lock()
_lib = None
_binding = None

CKV_F32 = 0
CKV_BF16 = 1
PLAN_ENTRY_BYTES = 16
SENTINEL = 0xFFFFFFFF

_STATUS_FUNCS = {
    "ckv_kpool_decode_update": 25,
    "ckv_kpool_compress": 20,
    "ckv_kpool_seed_tail": 10,
    "ckv_c128_online_decode": 13,
    "ckv_c128_online_prefill": 18,
    "ckv_c128_online_decode_fp8": 18,
    "ckv_c128_online_prefill_fp8": 23,
    "ckv_plan_online_prefill": 9,
    "ckv_plan_online_prefill_device": 11,
    "ckv_c128_online_prefill_counted": 17,
    "ckv_c128_online_prefill_counted_fp8": 22,
    "ckv_expand_pools_and_append_tail": 9,
    "ckv_wait_timeout_selftest": 3,
    "ckv_check_distinct": 8,
    "ckv_check_distinct_noalloc": 6,
    "ckv_latency_probe": 9,
    "ckv_build_step_maps": 25,
    "ckv_qk_norm_rope": 12,
    "ckv_fp4_store": 13,
    "ckv_fp4_load": 13,
    "ckv_fp4_attention": 26,
    "ckv_kv_append": 18,
    "ckv_build_tree_masks": 11,
    "ckv_kv_attention": 26,
    "ckv_merge_attention": 12,
}
EXPORTED = tuple(_STATUS_FUNCS) + ("ckv_status_string", "ckv_last_cuda_error", "ckv_abi_version",
                                    "ckv_c128_prefill_set_variant", "ckv_kpool_compress_set_variant",
                                    "ckv_fp4_attention_workspace", "ckv_kv_attention_workspace")


class NormRows(ctypes.Structure):
    """ckv_norm_rows of include/ckv.h."""

    _fields_ = [("x", ctypes.c_void_p), ("out", ctypes.c_void_p), ("weight", ctypes.c_void_p),
                ("positions", ctypes.c_void_p), ("stride_t", ctypes.c_int64), ("stride_h", ctypes.c_int64),
                ("out_stride_t", ctypes.c_int64), ("out_stride_h", ctypes.c_int64), ("tokens", ctypes.c_int64),
                ("heads", ctypes.c_int32), ("dtype", ctypes.c_int32), ("out_dtype", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


class KvCache(ctypes.Structure):
    """ckv_kv_cache of include/ckv.h."""

    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_stride_page", ctypes.c_int64),
                ("k_stride_row", ctypes.c_int64), ("k_stride_head", ctypes.c_int64), ("v_stride_page", ctypes.c_int64),
                ("v_stride_row", ctypes.c_int64), ("v_stride_head", ctypes.c_int64), ("num_pages", ctypes.c_int64),
                ("page_size", ctypes.c_int32), ("heads", ctypes.c_int32), ("D", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


class KvRows(ctypes.Structure):
    """ckv_kv_rows of include/ckv.h."""

    _fields_ = [("x", ctypes.c_void_p), ("stride_t", ctypes.c_int64), ("stride_h", ctypes.c_int64),
                ("heads", ctypes.c_int32), ("dtype", ctypes.c_int32)]


class AttentionPart(ctypes.Structure):
    """ckv_attention_part of include/ckv.h."""

    _fields_ = [("out", ctypes.c_void_p), ("lse", ctypes.c_void_p)]


class CkvError(RuntimeError):
    def __init__(self, func, status, lib):
        msg = lib.ckv_status_string(status).decode()
        if status == 6:
            msg += f" (cudaError {lib.ckv_last_cuda_error()})"
        super().__init__(f"{func}: status {status}: {msg}")
        self.status = status


def lib_path() -> str:
    return _build.LIB


def load():
    """Load libckv.so; raise if it has not been built (no fallback path exists)."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(_build.LIB):
                raise RuntimeError(
                    f"{_build.LIB} is missing: build it first "
                    "(python -c 'import __graft_entry__ as g; g.build()')")
            L = ctypes.CDLL(_build.LIB)
            for name, nargs in _STATUS_FUNCS.items():
                fn = getattr(L, name)
                fn.restype = ctypes.c_int32
            L.ckv_kpool_decode_update.argtypes = [
                ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_void_p, ctypes.c_int64,
                ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64,
                ctypes.c_int64, ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64, ctypes.c_void_p,
                ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32,
                ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int32, ctypes.c_void_p,
                ctypes.c_void_p]
            L.ckv_kpool_compress.argtypes = [
                ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_void_p, ctypes.c_void_p,
                ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int32, ctypes.c_void_p,
                ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32,
                ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int32, ctypes.c_void_p,
                ctypes.c_void_p]
            L.ckv_kpool_seed_tail.argtypes = [
                ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                ctypes.c_int64, ctypes.c_int32, ctypes.c_int32, ctypes.c_void_p, ctypes.c_void_p]
            L.ckv_c128_online_decode.argtypes = [
                ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p, ctypes.c_int32, ctypes.c_void_p,
                ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int32, ctypes.c_int32,
                ctypes.c_int32, ctypes.c_void_p, ctypes.c_void_p]
            L.ckv_c128_online_prefill.argtypes = [
                ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64,
                ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int32,
                ctypes.c_void_p, ctypes.c_uint32, ctypes.c_void_p, ctypes.c_uint32, ctypes.c_int32,
                ctypes.c_int32, ctypes.c_void_p, ctypes.c_void_p]
            L.ckv_c128_online_decode_fp8.argtypes = [
                ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p, ctypes.c_int32, ctypes.c_void_p,
                ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int32, ctypes.c_int32,
                ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_void_p, ctypes.c_int32,
                ctypes.c_int32, ctypes.c_void_p, ctypes.c_void_p]
            L.ckv_c128_online_prefill_fp8.argtypes = [
                ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64,
                ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int32,
                ctypes.c_void_p, ctypes.c_uint32, ctypes.c_void_p, ctypes.c_uint32, ctypes.c_int32,
                ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_void_p, ctypes.c_int32,
                ctypes.c_int32, ctypes.c_void_p, ctypes.c_void_p]
            L.ckv_plan_online_prefill.argtypes = [
                ctypes.c_void_p, ctypes.c_void_p, ctypes.c_uint32, ctypes.c_uint32, ctypes.c_void_p,
                ctypes.c_void_p, ctypes.c_int32, ctypes.POINTER(ctypes.c_uint32),
                ctypes.POINTER(ctypes.c_uint32)]
            L.ckv_plan_online_prefill_device.argtypes = [
                ctypes.c_void_p, ctypes.c_void_p, ctypes.c_uint32, ctypes.c_uint32, ctypes.c_void_p,
                ctypes.c_void_p, ctypes.c_int32, ctypes.c_void_p, ctypes.c_int32, ctypes.c_void_p,
                ctypes.c_void_p]
            L.ckv_c128_online_prefill_counted.argtypes = [
                ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64,
                ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int32,
                ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int32, ctypes.c_int32,
                ctypes.c_void_p, ctypes.c_void_p]
            L.ckv_c128_online_prefill_counted_fp8.argtypes = [
                ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64,
                ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int32,
                ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int32, ctypes.c_void_p,
                ctypes.c_int64, ctypes.c_int32, ctypes.c_void_p, ctypes.c_int32, ctypes.c_int32,
                ctypes.c_void_p, ctypes.c_void_p]
            L.ckv_expand_pools_and_append_tail.argtypes = [
                ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p, ctypes.c_int32, ctypes.c_int32,
                ctypes.c_int32, ctypes.c_void_p, ctypes.c_int32, ctypes.c_void_p]
            L.ckv_wait_timeout_selftest.argtypes = [ctypes.c_void_p, ctypes.c_uint32, ctypes.c_void_p]
            L.ckv_check_distinct.argtypes = [
                ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_int64, ctypes.c_void_p,
                ctypes.c_int64, ctypes.c_void_p, ctypes.c_void_p]
            L.ckv_check_distinct_noalloc.argtypes = [
                ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_int64, ctypes.c_void_p, ctypes.c_void_p]
            L.ckv_latency_probe.argtypes = [
                ctypes.c_int32, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p, ctypes.c_int32,
                ctypes.c_int32, ctypes.c_int32, ctypes.c_void_p]
            vp, i32, i64, f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float
            L.ckv_build_step_maps.argtypes = [vp, vp, i32, i32, i32, vp, i64, i32, vp, i64, vp, vp, vp, i32,
                                              vp, vp, vp, vp, vp, vp, vp, vp, i32, vp, vp]
            L.ckv_qk_norm_rope.argtypes = [ctypes.POINTER(NormRows), ctypes.POINTER(NormRows), vp, i64, i32, i32, i32,
                                           i32, f32, i32, vp, vp]
            L.ckv_fp4_store.argtypes = [vp, i32, i64, i64, i32, vp, i64, i32, vp, f32, i32, vp, vp]
            L.ckv_fp4_load.argtypes = [vp, i64, i32, vp, i64, i32, vp, i32, i64, f32, i32, vp, vp]
            L.ckv_fp4_attention_workspace.restype = ctypes.c_int64
            L.ckv_fp4_attention_workspace.argtypes = [i64, i32, i32, i32, i64]
            L.ckv_fp4_attention.argtypes = [vp, i64, i64, i64, i32, i32, vp, i64, i32, f32, vp, i64, i32, vp, i32, vp,
                                            i64, f32, vp, vp, vp, vp, i64, i32, vp, vp]
            cache, rows = ctypes.POINTER(KvCache), ctypes.POINTER(KvRows)
            L.ckv_kv_append.argtypes = [rows, rows, rows, vp, i64, i64, i64, cache, vp, vp, vp, i64, i32, i32, i32, i32,
                                        vp, vp]
            L.ckv_build_tree_masks.argtypes = [vp, vp, i32, vp, i64, i32, vp, vp, i32, vp, vp]
            L.ckv_kv_attention_workspace.restype = ctypes.c_int64
            L.ckv_kv_attention_workspace.argtypes = [i64, i32, i32, i32, i32, i64, i32, i32, i32]
            L.ckv_kv_attention.argtypes = [vp, i64, i64, i64, i32, cache, vp, i64, i32, vp, i32, vp, i64, i32, i32, vp,
                                           i32, f32, vp, vp, vp, vp, i64, i32, vp, vp]
            L.ckv_merge_attention.argtypes = [ctypes.POINTER(AttentionPart), i32, i32, i64, i32, i32, vp, vp, i32, vp,
                                              i32, vp]
            L.ckv_status_string.restype = ctypes.c_char_p
            L.ckv_status_string.argtypes = [ctypes.c_int32]
            L.ckv_last_cuda_error.restype = ctypes.c_int32
            L.ckv_last_cuda_error.argtypes = []
            L.ckv_abi_version.restype = ctypes.c_int32
            L.ckv_abi_version.argtypes = []
            for fn in (L.ckv_c128_prefill_set_variant, L.ckv_kpool_compress_set_variant):
                fn.restype = ctypes.c_int32
                fn.argtypes = [ctypes.c_int32]
            _lib = L
    return _lib


# ------------------------------------------------------------------ helpers
def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream, ref):
    if stream is not None:
        return ctypes.c_void_p(stream if isinstance(stream, int) else stream.cuda_stream)
    return ctypes.c_void_p(torch.cuda.current_stream(ref.device).cuda_stream)


def _on(stream):
    """Allocate for `stream`: the caching allocator hands out memory that is free
    on torch's current stream, so tensors made here for another one are made with it current."""
    if stream is None:
        return contextlib.nullcontext()
    if isinstance(stream, int):  # 0 is the default stream, which ExternalStream(0) is not
        stream = torch.cuda.ExternalStream(stream) if stream else torch.cuda.default_stream()
    return torch.cuda.stream(stream)


def _cuda(name, *ts):
    """Every tensor on one CUDA device, the current one: the kernels run on the
    current device, and a pointer into another device's memory would fault."""
    devs = set()
    for t in ts:
        if t is None:
            continue
        if not t.is_cuda:
            raise ValueError(f"{name}: every tensor must be on a CUDA device")
        devs.add(t.device.index)
    if len(devs) > 1:
        raise ValueError(f"{name}: tensors on several CUDA devices {sorted(devs)}")
    if devs and devs.pop() != torch.cuda.current_device():
        raise ValueError(f"{name}: the tensors are not on the current CUDA device "
                         f"(torch.cuda.set_device or torch.cuda.device(...) first)")


def _check(func, status):
    if status != 0:
        raise CkvError(func, status, load())


def _dtype(t):
    if t.dtype == torch.float32:
        return CKV_F32
    if t.dtype == torch.bfloat16:
        return CKV_BF16
    raise ValueError("input must be float32 or bfloat16")


def _need(cond, msg):
    if not cond:
        raise ValueError(msg)


def ckv_wait_timeout_selftest(err_word, limit_us=20000, stream=None):
    """Run the bounded-wait self-test (see include/ckv.h); err_word: CUDA int32 [1]."""
    L = load()
    _cuda("ckv_wait_timeout_selftest", err_word)
    _check("ckv_wait_timeout_selftest", L.ckv_wait_timeout_selftest(_ptr(err_word), int(limit_us),
                                                                    _stream(stream, err_word)))


# ------------------------------------------------------------ pooled path
def ckv_kpool_decode_update(kv_cache, tail_ring, tail_slot_mapping, slot_mapping, positions, key,
                            score, ape, round_scale=True, tap_x=None, tap_xb=None, tap_yb=None,
                            use_pdl=False, err_word=None, stream=None):
    """Pooled decode/verify update; see ckv_kpool_decode_update in include/ckv.h.

    kv_cache uint8 [pages, page_size, D+4]; tail_ring bf16 [blocks, 2, P, D];
    index tensors int32 [B, N] (contiguous); key/score bf16 [B, N, D] (last dim
    contiguous); ape float32 [P, D].
    """
    L = load()
    _cuda("ckv_kpool_decode_update", kv_cache, tail_ring, tail_slot_mapping, slot_mapping, positions,
          key, score, ape, tap_x, tap_xb, tap_yb, err_word)
    B, N, D = key.shape
    P = tail_ring.shape[2]
    _need(kv_cache.dtype == torch.uint8 and kv_cache.dim() == 3 and kv_cache.is_contiguous(),
          "kv_cache must be contiguous uint8 [pages, page_size, D+4]")
    _need(tail_ring.dtype == torch.bfloat16 and tail_ring.is_contiguous() and tail_ring.dim() == 4
          and tail_ring.shape[1] == 2 and tail_ring.shape[3] == D, "tail_ring must be bf16 [blocks, 2, P, D]")
    _need(key.dtype == torch.bfloat16 and score.dtype == torch.bfloat16 and score.shape == key.shape
          and key.stride(2) == 1 and score.stride(2) == 1, "key/score must be bf16 [B, N, D], last dim contiguous")
    for t in (tail_slot_mapping, slot_mapping, positions):
        _need(t.dtype == torch.int32 and t.is_contiguous() and tuple(t.shape) == (B, N),
              "index tensors must be contiguous int32 [B, N]")
    _need(ape.dtype == torch.float32 and ape.is_contiguous() and tuple(ape.shape) == (P, D),
          "ape must be contiguous float32 [P, D]")
    _check("ckv_kpool_decode_update", L.ckv_kpool_decode_update(
        _ptr(kv_cache), kv_cache.shape[0], kv_cache.shape[1], _ptr(tail_ring), tail_ring.shape[0],
        _ptr(tail_slot_mapping), _ptr(slot_mapping), _ptr(positions), _ptr(key), key.stride(0),
        key.stride(1), _ptr(score), score.stride(0), score.stride(1), _ptr(ape), B, N, P, D,
        int(bool(round_scale)), _ptr(tap_x), _ptr(tap_xb), _ptr(tap_yb), int(bool(use_pdl)), _ptr(err_word),
        _stream(stream, key)))


def ckv_kpool_compress(slot_k, slot_score, ape, kv_cache=None, loc=None, write_mask=None,
                       write_cache=True, out_fp8=None, out_scale=None, round_scale=True, tap_x=None,
                       tap_xb=None, tap_yb=None, use_pdl=False, err_word=None, stream=None):
    """One-shot pooled compression; see ckv_kpool_compress in include/ckv.h.

    slot_k/slot_score bf16 [n, P, D] contiguous; ape float32 [P, D]; loc int64 [n];
    write_mask bool/uint8 [n]; out_fp8 uint8 (or float8_e4m3fn) [n, D]; out_scale float32 [n].
    """
    L = load()
    _cuda("ckv_kpool_compress", slot_k, slot_score, ape, kv_cache, loc, write_mask, out_fp8, out_scale,
          tap_x, tap_xb, tap_yb, err_word)
    n, P, D = slot_k.shape
    _need(slot_k.dtype == torch.bfloat16 and slot_score.dtype == torch.bfloat16
          and slot_k.is_contiguous() and slot_score.is_contiguous() and slot_score.shape == slot_k.shape,
          "slot_k/slot_score must be contiguous bf16 [n, P, D]")
    _need(ape.dtype == torch.float32 and ape.is_contiguous() and tuple(ape.shape) == (P, D),
          "ape must be contiguous float32 [P, D]")
    pages = ps = 0
    if write_cache:
        _need(kv_cache is not None and loc is not None, "write_cache needs kv_cache and loc")
        _need(kv_cache.dtype == torch.uint8 and kv_cache.dim() == 3 and kv_cache.is_contiguous(),
              "kv_cache must be contiguous uint8 [pages, page_size, D+4]")
        _need(loc.dtype == torch.int64 and loc.is_contiguous() and loc.numel() == n, "loc must be int64 [n]")
        pages, ps = kv_cache.shape[0], kv_cache.shape[1]
    if write_mask is not None:
        _need(write_mask.dtype in (torch.bool, torch.uint8) and write_mask.is_contiguous()
              and write_mask.numel() == n, "write_mask must be bool [n]")
    if out_fp8 is not None:
        _need(out_fp8.element_size() == 1 and out_fp8.is_contiguous() and out_fp8.numel() == n * D,
              "out_fp8 must be a contiguous 1-byte tensor [n, D]")
        _need(out_scale is not None and out_scale.dtype == torch.float32 and out_scale.numel() == n,
              "out_scale must be float32 [n]")
    _check("ckv_kpool_compress", L.ckv_kpool_compress(
        _ptr(kv_cache) if write_cache else None, pages, ps, _ptr(slot_k), _ptr(slot_score), _ptr(ape),
        _ptr(loc) if write_cache else None, _ptr(write_mask), int(bool(write_cache)), _ptr(out_fp8),
        _ptr(out_scale), n, P, D, int(bool(round_scale)), _ptr(tap_x), _ptr(tap_xb), _ptr(tap_yb),
        int(bool(use_pdl)), _ptr(err_word), _stream(stream, slot_k)))


def ckv_kpool_seed_tail(tail_ring, key, score, tslot, err_word=None, stream=None):
    """Seed the tail ring from a prefill batch; see ckv_kpool_seed_tail in include/ckv.h."""
    L = load()
    _cuda("ckv_kpool_seed_tail", tail_ring, key, score, tslot, err_word)
    n, D = key.shape
    P = tail_ring.shape[2]
    _need(tail_ring.dtype == torch.bfloat16 and tail_ring.is_contiguous(), "tail_ring must be bf16")
    _need(key.dtype == torch.bfloat16 and score.dtype == torch.bfloat16 and key.is_contiguous()
          and score.is_contiguous() and score.shape == key.shape, "key/score must be contiguous bf16 [n, D]")
    _need(tslot.dtype == torch.int32 and tslot.is_contiguous() and tslot.numel() == n, "tslot must be int32 [n]")
    _check("ckv_kpool_seed_tail", L.ckv_kpool_seed_tail(
        _ptr(tail_ring), tail_ring.shape[0], _ptr(key), _ptr(score), _ptr(tslot), n, P, D,
        _ptr(err_word), _stream(stream, key)))


def ckv_expand_pools_and_append_tail(pool_ids, seq_lens, pool_size, out=None, use_pdl=False, stream=None):
    """Pool -> token index expansion with the tail appended; see include/ckv.h.

    pool_ids: CUDA int32 [rows, n_groups] (last dim contiguous); seq_lens: CUDA
    int64 [rows].  Returns int32 [rows, n_groups * pool_size + pool_size - 1].
    """
    L = load()
    _cuda("ckv_expand_pools_and_append_tail", pool_ids, seq_lens, out)
    _need(pool_ids.dtype == torch.int32 and pool_ids.dim() == 2 and pool_ids.stride(1) == 1,
          "pool_ids must be int32 [rows, n_groups], last dim contiguous")
    _need(seq_lens.dtype == torch.int64 and seq_lens.is_contiguous(), "seq_lens must be int64 [rows]")
    rows, groups = pool_ids.shape
    cols = groups * pool_size + pool_size - 1
    if out is None:
        out = torch.empty((rows, cols), dtype=torch.int32, device=pool_ids.device)
    _need(out.dtype == torch.int32 and out.is_contiguous() and tuple(out.shape) == (rows, cols),
          "out must be contiguous int32 [rows, n_groups * P + P - 1]")
    _check("ckv_expand_pools_and_append_tail", L.ckv_expand_pools_and_append_tail(
        _ptr(pool_ids), pool_ids.stride(0), _ptr(seq_lens), rows, groups, int(pool_size), _ptr(out),
        int(bool(use_pdl)), _stream(stream, pool_ids)))
    return out


# ------------------------------------------------------------ online c128
def ckv_c128_online_decode(state, input, out, ape, indices, seq_lens, use_pdl=False, err_word=None,
                           stream=None):
    """Online c128 decode; see ckv_c128_online_decode in include/ckv.h.

    state float32 [slots, 3, D] (or [slots, 1, 3D]); input float32/bf16 [B, 2D];
    out float32 [B, D]; ape float32 [128, D]; indices/seq_lens int32 [B].
    """
    L = load()
    _cuda("ckv_c128_online_decode", state, input, out, ape, indices, seq_lens, err_word)
    B = input.shape[0]
    D = input.shape[1] // 2
    _need(state.dtype == torch.float32 and state.is_contiguous() and state.numel() % (3 * D) == 0,
          "state must be contiguous float32 [slots, 3, D]")
    _need(input.is_contiguous() and input.dim() == 2, "input must be contiguous [B, 2D]")
    _need(out.dtype == torch.float32 and out.is_contiguous() and tuple(out.shape) == (B, D), "out must be float32 [B, D]")
    _need(ape.dtype == torch.float32 and ape.is_contiguous() and tuple(ape.shape) == (128, D), "ape must be float32 [128, D]")
    for t in (indices, seq_lens):
        _need(t.dtype == torch.int32 and t.is_contiguous() and t.numel() == B, "indices/seq_lens must be int32 [B]")
    _check("ckv_c128_online_decode", L.ckv_c128_online_decode(
        _ptr(state), state.numel() // (3 * D), _ptr(input), _dtype(input), _ptr(out), _ptr(ape),
        _ptr(indices), _ptr(seq_lens), B, D, int(bool(use_pdl)), _ptr(err_word), _stream(stream, input)))


def ckv_c128_online_prefill(state, input, out, ape, indices, compress_plan, num_compress, write_plan,
                            num_write, load_indices=None, use_pdl=False, err_word=None, stream=None):
    """Online c128 prefill (compress pass, then write pass); see include/ckv.h.

    state float32 [slots, 3, D]; input float32/bf16 [T, 2D]; out float32 [T, D];
    ape float32 [128, D]; indices (and load_indices) int32 [B]; plans are device
    tensors of 16-byte entries (uint8 [M, 16] or int32 [M, 4]).
    """
    L = load()
    _cuda("ckv_c128_online_prefill", state, input, out, ape, indices, load_indices, compress_plan,
          write_plan, err_word)
    T = input.shape[0]
    D = input.shape[1] // 2
    B = indices.numel()
    _need(state.dtype == torch.float32 and state.is_contiguous() and state.numel() % (3 * D) == 0,
          "state must be contiguous float32 [slots, 3, D]")
    _need(input.is_contiguous() and input.dim() == 2, "input must be contiguous [T, 2D]")
    _need(out.dtype == torch.float32 and out.is_contiguous() and tuple(out.shape) == (T, D), "out must be float32 [T, D]")
    _need(ape.dtype == torch.float32 and ape.is_contiguous() and tuple(ape.shape) == (128, D), "ape must be float32 [128, D]")
    _need(indices.dtype == torch.int32 and indices.is_contiguous(), "indices must be int32 [B]")
    if load_indices is not None:
        _need(load_indices.dtype == torch.int32 and load_indices.is_contiguous() and load_indices.numel() == B,
              "load_indices must be int32 [B]")
    for pl, cnt in ((compress_plan, num_compress), (write_plan, num_write)):
        _need(pl.is_contiguous() and pl.numel() * pl.element_size() >= cnt * PLAN_ENTRY_BYTES,
              "plan tensors must hold num_* 16-byte entries")
    _check("ckv_c128_online_prefill", L.ckv_c128_online_prefill(
        _ptr(state), state.numel() // (3 * D), _ptr(input), _dtype(input), T, _ptr(out), _ptr(ape),
        _ptr(indices), _ptr(load_indices), B, _ptr(compress_plan), int(num_compress), _ptr(write_plan),
        int(num_write), D, int(bool(use_pdl)), _ptr(err_word), _stream(stream, input)))


def _fp8_cache(kv_cache, cache_loc, D, n_loc):
    blocks = D // 128
    _need(kv_cache.dtype == torch.uint8 and kv_cache.is_contiguous() and kv_cache.dim() == 3
          and kv_cache.shape[2] == D + 4 * blocks, "kv_cache must be contiguous uint8 [pages, page_size, D + 4*D/128]")
    _need(cache_loc.dtype == torch.int64 and cache_loc.is_contiguous() and cache_loc.numel() == n_loc,
          "cache_loc must be contiguous int64")
    return kv_cache.shape[0], kv_cache.shape[1]


def ckv_c128_online_decode_fp8(state, input, out, ape, indices, seq_lens, kv_cache, cache_loc, round_scale=True,
                               use_pdl=False, err_word=None, stream=None):
    """Online c128 decode with the FP8 output stage; see ckv_c128_online_decode_fp8
    in include/ckv.h.  kv_cache uint8 [pages, page_size, D + 4*D/128];
    cache_loc int64 [B]; out float32 [B, D] or None."""
    L = load()
    _cuda("ckv_c128_online_decode_fp8", state, input, out, ape, indices, seq_lens, kv_cache, cache_loc, err_word)
    B = input.shape[0]
    D = input.shape[1] // 2
    _need(state.dtype == torch.float32 and state.is_contiguous() and state.numel() % (3 * D) == 0,
          "state must be contiguous float32 [slots, 3, D]")
    _need(input.is_contiguous() and input.dim() == 2, "input must be contiguous [B, 2D]")
    _need(out is None or (out.dtype == torch.float32 and out.is_contiguous() and tuple(out.shape) == (B, D)),
          "out must be float32 [B, D] or None")
    _need(ape.dtype == torch.float32 and ape.is_contiguous() and tuple(ape.shape) == (128, D), "ape must be float32 [128, D]")
    for t in (indices, seq_lens):
        _need(t.dtype == torch.int32 and t.is_contiguous() and t.numel() == B, "indices/seq_lens must be int32 [B]")
    pages, ps = _fp8_cache(kv_cache, cache_loc, D, B)
    _check("ckv_c128_online_decode_fp8", L.ckv_c128_online_decode_fp8(
        _ptr(state), state.numel() // (3 * D), _ptr(input), _dtype(input), _ptr(out), _ptr(ape),
        _ptr(indices), _ptr(seq_lens), B, D, _ptr(kv_cache), pages, ps, _ptr(cache_loc), int(bool(round_scale)),
        int(bool(use_pdl)), _ptr(err_word), _stream(stream, input)))


def ckv_c128_online_prefill_fp8(state, input, out, ape, indices, compress_plan, num_compress, write_plan,
                                num_write, kv_cache, cache_loc, round_scale=True, load_indices=None, use_pdl=False,
                                err_word=None, stream=None):
    """Online c128 prefill with the FP8 output stage; see ckv_c128_online_prefill_fp8
    in include/ckv.h.  kv_cache uint8 [pages, page_size, D + 4*D/128];
    cache_loc int64 [T] (read at compress rows); out float32 [T, D] or None."""
    L = load()
    _cuda("ckv_c128_online_prefill_fp8", state, input, out, ape, indices, load_indices, compress_plan,
          write_plan, kv_cache, cache_loc, err_word)
    T = input.shape[0]
    D = input.shape[1] // 2
    B = indices.numel()
    _need(state.dtype == torch.float32 and state.is_contiguous() and state.numel() % (3 * D) == 0,
          "state must be contiguous float32 [slots, 3, D]")
    _need(input.is_contiguous() and input.dim() == 2, "input must be contiguous [T, 2D]")
    _need(out is None or (out.dtype == torch.float32 and out.is_contiguous() and tuple(out.shape) == (T, D)),
          "out must be float32 [T, D] or None")
    _need(ape.dtype == torch.float32 and ape.is_contiguous() and tuple(ape.shape) == (128, D), "ape must be float32 [128, D]")
    _need(indices.dtype == torch.int32 and indices.is_contiguous(), "indices must be int32 [B]")
    if load_indices is not None:
        _need(load_indices.dtype == torch.int32 and load_indices.is_contiguous() and load_indices.numel() == B,
              "load_indices must be int32 [B]")
    for pl, cnt in ((compress_plan, num_compress), (write_plan, num_write)):
        _need(pl.is_contiguous() and pl.numel() * pl.element_size() >= cnt * PLAN_ENTRY_BYTES,
              "plan tensors must hold num_* 16-byte entries")
    pages, ps = _fp8_cache(kv_cache, cache_loc, D, T)
    _check("ckv_c128_online_prefill_fp8", L.ckv_c128_online_prefill_fp8(
        _ptr(state), state.numel() // (3 * D), _ptr(input), _dtype(input), T, _ptr(out), _ptr(ape),
        _ptr(indices), _ptr(load_indices), B, _ptr(compress_plan), int(num_compress), _ptr(write_plan),
        int(num_write), D, _ptr(kv_cache), pages, ps, _ptr(cache_loc), int(bool(round_scale)), int(bool(use_pdl)),
        _ptr(err_word), _stream(stream, input)))


def ckv_c128_prefill_set_variant(variant: int) -> int:
    """Select the compress-pass kernel (0 auto, 1 one CTA per segment, 2 TMA pipeline).

    Returns the previous setting; raises on an unknown value."""
    prev = load().ckv_c128_prefill_set_variant(int(variant))
    if prev < 0:
        raise ValueError(f"unknown prefill variant {variant}")
    return prev


def ckv_kpool_compress_set_variant(variant: int) -> int:
    """Select the pooled one-shot kernel (0 auto, 1 one warp per pool, 2 bulk-copy pipeline).

    Returns the previous setting; raises on an unknown value."""
    prev = load().ckv_kpool_compress_set_variant(int(variant))
    if prev < 0:
        raise ValueError(f"unknown kpool compress variant {variant}")
    return prev


def ckv_plan_online_prefill_device(seq_lens, extend_lens, num_tokens, compress_plan=None, write_plan=None,
                                   counts=None, pad_for_graph=False, use_pdl=False, err_word=None, stream=None):
    """Device-side planner; see ckv_plan_online_prefill_device in include/ckv.h.

    seq_lens/extend_lens: CUDA int64 tensors [B].  Returns (compress_plan,
    write_plan, counts) as CUDA tensors (uint8 [num_tokens, 16] x2, int32 [2]);
    nothing is copied to the host.
    """
    L = load()
    _cuda("ckv_plan_online_prefill_device", seq_lens, extend_lens, compress_plan, write_plan, counts, err_word)
    _need(seq_lens.dtype == torch.int64 and extend_lens.dtype == torch.int64 and seq_lens.is_contiguous()
          and extend_lens.is_contiguous() and seq_lens.numel() == extend_lens.numel(),
          "seq_lens/extend_lens must be contiguous int64 [B]")
    dev = seq_lens.device
    if compress_plan is None:
        compress_plan = torch.empty((num_tokens, PLAN_ENTRY_BYTES), dtype=torch.uint8, device=dev)
    if write_plan is None:
        write_plan = torch.empty((num_tokens, PLAN_ENTRY_BYTES), dtype=torch.uint8, device=dev)
    if counts is None:
        counts = torch.zeros((2,), dtype=torch.int32, device=dev)
    for pl in (compress_plan, write_plan):
        _need(pl.is_contiguous() and pl.numel() * pl.element_size() >= num_tokens * PLAN_ENTRY_BYTES,
              "plan buffers must hold num_tokens 16-byte rows")
    _need(counts.numel() >= 2 and counts.element_size() == 4, "counts must be a 4-byte tensor of 2 elements")
    _check("ckv_plan_online_prefill_device", L.ckv_plan_online_prefill_device(
        _ptr(seq_lens), _ptr(extend_lens), seq_lens.numel(), int(num_tokens), _ptr(compress_plan),
        _ptr(write_plan), int(bool(pad_for_graph)), _ptr(counts), int(bool(use_pdl)), _ptr(err_word),
        _stream(stream, seq_lens)))
    return compress_plan, write_plan, counts


def ckv_c128_online_prefill_counted(state, input, out, ape, indices, compress_plan, write_plan, counts,
                                    load_indices=None, use_pdl=False, err_word=None, stream=None):
    """Online c128 prefill with device-resident segment counts; see include/ckv.h."""
    L = load()
    _cuda("ckv_c128_online_prefill_counted", state, input, out, ape, indices, load_indices, compress_plan,
          write_plan, counts, err_word)
    T = input.shape[0]
    D = input.shape[1] // 2
    B = indices.numel()
    _need(state.dtype == torch.float32 and state.is_contiguous() and state.numel() % (3 * D) == 0,
          "state must be contiguous float32 [slots, 3, D]")
    _need(input.is_contiguous() and input.dim() == 2, "input must be contiguous [T, 2D]")
    _need(out.dtype == torch.float32 and out.is_contiguous() and tuple(out.shape) == (T, D), "out must be float32 [T, D]")
    _need(ape.dtype == torch.float32 and ape.is_contiguous() and tuple(ape.shape) == (128, D), "ape must be float32 [128, D]")
    _need(indices.dtype == torch.int32 and indices.is_contiguous(), "indices must be int32 [B]")
    for pl in (compress_plan, write_plan):
        _need(pl.is_contiguous() and pl.numel() * pl.element_size() >= min(T, T // 128 + B) * PLAN_ENTRY_BYTES,
              "plan tensors too small")
    _check("ckv_c128_online_prefill_counted", L.ckv_c128_online_prefill_counted(
        _ptr(state), state.numel() // (3 * D), _ptr(input), _dtype(input), T, _ptr(out), _ptr(ape), _ptr(indices),
        _ptr(load_indices), B, _ptr(compress_plan), _ptr(write_plan), _ptr(counts), D, int(bool(use_pdl)),
        _ptr(err_word), _stream(stream, input)))


def ckv_c128_online_prefill_counted_fp8(state, input, out, ape, indices, compress_plan, write_plan, counts,
                                        kv_cache, cache_loc, round_scale=True, load_indices=None, use_pdl=False,
                                        err_word=None, stream=None):
    """The device-counted prefill with the FP8 output stage; see include/ckv.h.
    kv_cache uint8 [pages, page_size, D + 4*D/128]; cache_loc int64 [T]; out
    float32 [T, D] or None."""
    L = load()
    _cuda("ckv_c128_online_prefill_counted_fp8", state, input, out, ape, indices, load_indices, compress_plan,
          write_plan, counts, kv_cache, cache_loc, err_word)
    T = input.shape[0]
    D = input.shape[1] // 2
    B = indices.numel()
    _need(state.dtype == torch.float32 and state.is_contiguous() and state.numel() % (3 * D) == 0,
          "state must be contiguous float32 [slots, 3, D]")
    _need(input.is_contiguous() and input.dim() == 2, "input must be contiguous [T, 2D]")
    _need(out is None or (out.dtype == torch.float32 and out.is_contiguous() and tuple(out.shape) == (T, D)),
          "out must be float32 [T, D] or None")
    _need(ape.dtype == torch.float32 and ape.is_contiguous() and tuple(ape.shape) == (128, D), "ape must be float32 [128, D]")
    _need(indices.dtype == torch.int32 and indices.is_contiguous(), "indices must be int32 [B]")
    for pl in (compress_plan, write_plan):
        _need(pl.is_contiguous() and pl.numel() * pl.element_size() >= min(T, T // 128 + B) * PLAN_ENTRY_BYTES,
              "plan tensors too small")
    pages, ps = _fp8_cache(kv_cache, cache_loc, D, T)
    _check("ckv_c128_online_prefill_counted_fp8", L.ckv_c128_online_prefill_counted_fp8(
        _ptr(state), state.numel() // (3 * D), _ptr(input), _dtype(input), T, _ptr(out), _ptr(ape), _ptr(indices),
        _ptr(load_indices), B, _ptr(compress_plan), _ptr(write_plan), _ptr(counts), D, _ptr(kv_cache), pages, ps,
        _ptr(cache_loc), int(bool(round_scale)), int(bool(use_pdl)), _ptr(err_word), _stream(stream, input)))


def ckv_plan_online_prefill(seq_lens, extend_lens, num_tokens=None, pad_for_graph=False,
                            compress_plan=None, write_plan=None):
    """Host planner; see ckv_plan_online_prefill in include/ckv.h.

    seq_lens/extend_lens: CPU int64 tensors [B].  Returns (compress_plan,
    write_plan, num_compress, num_write) with the plans as CPU uint8 tensors
    [num_tokens, 16] (pass pinned tensors to fill them in place).
    """
    L = load()
    _need(not seq_lens.is_cuda and not extend_lens.is_cuda, "planner inputs must be host tensors")
    seq_lens = seq_lens.to(torch.int64).contiguous()
    extend_lens = extend_lens.to(torch.int64).contiguous()
    B = seq_lens.numel()
    if num_tokens is None:
        num_tokens = int(extend_lens.sum())
    if compress_plan is None:
        compress_plan = torch.empty((num_tokens, PLAN_ENTRY_BYTES), dtype=torch.uint8)
    if write_plan is None:
        write_plan = torch.empty((num_tokens, PLAN_ENTRY_BYTES), dtype=torch.uint8)
    for pl in (compress_plan, write_plan):
        _need(not pl.is_cuda and pl.is_contiguous() and pl.numel() * pl.element_size() >= num_tokens * 16,
              "plan buffers must be host tensors of num_tokens 16-byte rows")
    nc = ctypes.c_uint32()
    nw = ctypes.c_uint32()
    _check("ckv_plan_online_prefill", L.ckv_plan_online_prefill(
        _ptr(seq_lens), _ptr(extend_lens), B, num_tokens, _ptr(compress_plan), _ptr(write_plan),
        int(bool(pad_for_graph)), ctypes.byref(nc), ctypes.byref(nw)))
    return compress_plan, write_plan, nc.value, nw.value


# ------------------------------------------- a serving step around the cache
# These launch as programmatic dependents by default: a kernel may be set up while the one
# before it in the stream still runs, and waits for its end before it touches memory.
STEP_MAPS = ("row_start", "positions", "batch_ids", "slot_mapping", "cache_loc", "tail_slots", "row_positions",
             "ctx_rows")


def _native():
    """The compiled checks and calls of the serving-step entry points (csrc/binding.cpp)."""
    global _binding
    if _binding is None:
        load()
        with _lock:
            if _binding is None:
                if not os.path.exists(_build.BINDING):
                    raise RuntimeError(f"{_build.BINDING} is missing: build it first "
                                       "(python -c 'import __graft_entry__ as g; g.build()')")
                loader = importlib.machinery.ExtensionFileLoader("ckv_binding", _build.BINDING)
                _binding = importlib.util.module_from_spec(
                    importlib.util.spec_from_file_location("ckv_binding", _build.BINDING, loader=loader))
    return _binding


def _raw(stream):
    return stream if stream is None or isinstance(stream, int) else stream.cuda_stream


def ckv_build_step_maps(seq_lens, query_lens, block_table, free_pages, cursor, pool_size, page_size, num_tokens,
                        tail_blocks=None, cursor_out=None, out=None, use_pdl=True, err_word=None, stream=None):
    """Block tables and slot maps of one step; see ckv_build_step_maps in include/ckv.h.

    seq_lens/query_lens (and tail_blocks) int32 [B]; block_table int32 [B,
    max_pages] (last dim contiguous, new pages are written to it); free_pages int32
    [F]; cursor int32 [1], or [2] with cursor[1] == 0 when it is moved in
    place (cursor_out None).  num_tokens is the size of the token maps.
    Returns a dict of the maps (STEP_MAPS; tail_slots only with tail_blocks).
    `out`, such a dict, names the maps to fill instead: row_start int32 [B + 1],
    cache_loc int64 [num_tokens], the others int32 [num_tokens]; maps that it
    lacks are not built.
    """
    native = _binding or _native()
    if stream is not None and out is None:
        _cuda("ckv_build_step_maps", seq_lens)
        with _on(stream):
            out = {k: torch.empty(seq_lens.numel() + 1 if k == "row_start" else num_tokens,
                                  dtype=torch.int64 if k == "cache_loc" else torch.int32, device=seq_lens.device)
                   for k in STEP_MAPS if k != "tail_slots" or tail_blocks is not None}
    status, out = native.step_maps(seq_lens, query_lens, block_table, free_pages, cursor, pool_size, page_size,
                                   num_tokens, tail_blocks, cursor_out, out, use_pdl, err_word, _raw(stream))
    if status:
        _check("ckv_build_step_maps", status)
    return out


def ckv_qk_norm_rope(q, q_positions, cos_sin=None, q_weight=None, q_out=None, k=None, k_positions=None, k_weight=None,
                     k_out=None, rope_offset=None, interleaved=False, eps=1e-6, use_pdl=True, err_word=None, stream=None):
    """Norm and rotation of queries and keys (or compressed rows) in one pass;
    see ckv_qk_norm_rope in include/ckv.h.

    q [T, H, D] and k [Tk, Hk, D] float32/bf16 (last dim contiguous); positions
    int32 [T] / [Tk], < 0 skips a token; weights float32 [D] or None; cos_sin
    float32 [positions, rope_dim] or None (norm only); rope_offset defaults to
    the last rope_dim channels.  Returns (q_out, k_out): new bf16 tensors, or
    the float32/bf16 ones given (q_out may be q).
    """
    native = _binding or _native()
    if stream is not None:
        _cuda("ckv_qk_norm_rope", q, k)
        with _on(stream):
            q_out = torch.empty(q.shape, dtype=torch.bfloat16, device=q.device) if q_out is None else q_out
            if k is not None and k_out is None:
                k_out = torch.empty(k.shape, dtype=torch.bfloat16, device=k.device)
    status, q_out, k_out = native.qk_norm_rope(q, q_positions, cos_sin, q_weight, q_out, k, k_positions, k_weight,
                                               k_out, rope_offset, interleaved, eps, use_pdl, err_word, _raw(stream))
    if status:
        _check("ckv_qk_norm_rope", status)
    return q_out, k_out


def ckv_fp4_store(rows, kv_cache, loc, cache_scale=1.0, use_pdl=True, err_word=None, stream=None):
    """Store rows in the 4-bit cache; see ckv_fp4_store in include/ckv.h.

    rows float32/bf16 [n, D] (last dim contiguous); kv_cache uint8 [pages,
    page_size, D/2 + D/16]; loc int64 [n], < 0 skips a row; cache_scale a power
    of two.
    """
    status = (_binding or _native()).fp4_store(rows, kv_cache, loc, cache_scale, use_pdl, err_word, _raw(stream))
    if status:
        _check("ckv_fp4_store", status)


def ckv_fp4_load(kv_cache, loc, out, cache_scale=1.0, use_pdl=True, err_word=None, stream=None):
    """Load rows of the 4-bit cache; see ckv_fp4_load in include/ckv.h.

    kv_cache, loc, cache_scale as for ckv_fp4_store; out float32/bf16 [n, D] (last
    dim contiguous); rows with loc < 0 are left as they are.
    """
    status = (_binding or _native()).fp4_load(out, kv_cache, loc, cache_scale, use_pdl, err_word, _raw(stream))
    if status:
        _check("ckv_fp4_load", status)
    return out


def ckv_fp4_attention_workspace(T, B, H, D, max_rows):
    """Bytes of workspace that ckv_fp4_attention needs for these sizes (0 for those that it refuses)."""
    return load().ckv_fp4_attention_workspace(int(T), int(B), int(H), int(D), int(max_rows))


def ckv_fp4_attention(q, kv_cache, block_table, row_start, ctx_rows, max_rows, softmax_scale, cache_scale=1.0, sink=None,
                      out=None, lse=None, workspace=None, use_pdl=True, err_word=None, stream=None):
    """Attention over the 4-bit cache; see ckv_fp4_attention in include/ckv.h.

    q bf16 [T, H, D] (last dim contiguous); kv_cache uint8 [pages, page_size,
    D/2 + D/16]; block_table int32 [B, max_pages] (last dim contiguous; rows apart,
    or one row expanded over all requests);
    row_start int32 [B + 1]; ctx_rows int32 [T], at most max_rows; sink
    float32 [H] or None.  Returns (out, lse): bf16 [T, H, D] and float32 [T, H].
    workspace: a uint8 tensor of ckv_fp4_attention_workspace() bytes, by default
    taken from the caching allocator of torch for this call.
    """
    native = _binding or _native()
    if stream is not None:
        _cuda("ckv_fp4_attention", q)
        T, H, D = q.shape
        need = ckv_fp4_attention_workspace(T, row_start.numel() - 1, H, D, max_rows)
        with _on(stream):
            out = torch.empty((T, H, D), dtype=torch.bfloat16, device=q.device) if out is None else out
            lse = torch.empty((T, H), dtype=torch.float32, device=q.device) if lse is None else lse
            if workspace is None and need:
                workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    status, out, lse = native.fp4_attention(q, kv_cache, block_table, row_start, ctx_rows, max_rows, softmax_scale,
                                            cache_scale, sink, out, lse, workspace, use_pdl, err_word, _raw(stream))
    if status:
        _check("ckv_fp4_attention", status)
    return out, lse


# ------------------------------------------- the tokens that are not compressed yet
def ckv_kv_append(k, v, k_cache, v_cache, loc, positions=None, cos_sin=None, rope_offset=None, interleaved=False, q=None,
                  q_out=None, use_pdl=True, err_word=None, stream=None):
    """Append keys (rotated) and values to a paged cache and rotate queries in the same pass; see
    ckv_kv_append in include/ckv.h.

    k, v [T, KH, D] and q [T, H, D] float32/bf16 of one type (last dim contiguous); v None: only
    keys are stored; caches bf16 [pages, page_size, KH, D] (last dim contiguous, any other
    strides without overlap, e.g. a transposed [pages, KH, page_size, D]); loc int64 [T], < 0: not
    stored; positions int32 [T], < 0 skips a token; cos_sin float32 [positions, rope_dim] or
    None (no rotation); rope_offset defaults to the last rope_dim channels.  Returns q_out: a new
    bf16 tensor, or the one given (it may be q), or None without q.
    """
    native = _binding or _native()
    if stream is not None and q is not None and q_out is None:
        _cuda("ckv_kv_append", k, q)
        with _on(stream):
            q_out = torch.empty(q.shape, dtype=torch.bfloat16, device=q.device)
    status, q_out = native.kv_append(k, v, k_cache, v_cache, loc, positions, cos_sin, rope_offset, interleaved, q, q_out,
                                     use_pdl, err_word, _raw(stream))
    if status:
        _check("ckv_kv_append", status)
    return q_out


def ckv_build_tree_masks(parents, row_start, ctx_rows=None, words=1, tree_mask=None, positions=None, use_pdl=True,
                         err_word=None, stream=None):
    """Masks and positions of trees of drafted tokens; see ckv_build_tree_masks in include/ckv.h.

    parents int32 [T]: index within its request, or -1; row_start int32 [B + 1]; ctx_rows int32 [T]
    or None; words 1..16, 64 drafts each.  Returns (tree_mask, positions): int64 [T, words] and
    int32 [T], new or the ones given.
    """
    native = _binding or _native()
    if stream is not None:
        _cuda("ckv_build_tree_masks", parents)
        T = parents.numel()
        with _on(stream):
            tree_mask = torch.empty((T, words), dtype=torch.int64, device=parents.device) if tree_mask is None else tree_mask
            positions = torch.empty(T, dtype=torch.int32, device=parents.device) if positions is None else positions
    status, tree_mask, positions = native.tree_masks(parents, row_start, ctx_rows, words, tree_mask, positions, use_pdl,
                                                     err_word, _raw(stream))
    if status:
        _check("ckv_build_tree_masks", status)
    return tree_mask, positions


def ckv_kv_attention_workspace(T, B, H, KH, D, max_rows, window=0, first_rows=0, mask_words=0):
    """Bytes of workspace that ckv_kv_attention needs for these sizes (0 for those that it refuses)."""
    return load().ckv_kv_attention_workspace(int(T), int(B), int(H), int(KH), int(D), int(max_rows), int(window),
                                             int(first_rows), int(mask_words))


def ckv_kv_attention(q, k_cache, v_cache, block_table, row_start, ctx_rows, max_rows, softmax_scale, window=0, first_rows=0,
                     tree_mask=None, sink=None, out=None, lse=None, workspace=None, use_pdl=True, err_word=None, stream=None):
    """Attention over the uncompressed cache; see ckv_kv_attention in include/ckv.h.

    q bf16 [T, H, D] (last dim contiguous); caches as for ckv_kv_append, one tensor for both where
    rows are key and value; block_table int32 [B, max_pages] (last dim contiguous; rows apart, or
    one row expanded over all requests); row_start int32 [B + 1]; ctx_rows int32 [T]: rows of the
    context, with the token itself, or with tree_mask the committed rows alone; max_rows at least
    the rows of every request, drafts included; window 0 or the rows of the window, first_rows that
    stay visible beside it; tree_mask int64 [T, words] or None; sink float32 [H] or None.  Returns
    (out, lse): bf16 [T, H, D] and float32 [T, H].  workspace: a uint8 tensor of
    ckv_kv_attention_workspace() bytes, by default taken from the caching allocator of torch.
    """
    native = _binding or _native()
    if stream is not None:
        _cuda("ckv_kv_attention", q)
        T, H, D = q.shape
        words = 0 if tree_mask is None else tree_mask.shape[1]
        need = ckv_kv_attention_workspace(T, row_start.numel() - 1, H, k_cache.shape[2], D, max_rows, window, first_rows, words)
        with _on(stream):
            out = torch.empty((T, H, D), dtype=torch.bfloat16, device=q.device) if out is None else out
            lse = torch.empty((T, H), dtype=torch.float32, device=q.device) if lse is None else lse
            if workspace is None and need:
                workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    status, out, lse = native.kv_attention(q, k_cache, v_cache, block_table, row_start, ctx_rows, max_rows, softmax_scale,
                                           window, first_rows, tree_mask, sink, out, lse, workspace, use_pdl, err_word,
                                           _raw(stream))
    if status:
        _check("ckv_kv_attention", status)
    return out, lse


def ckv_merge_attention(outs, lses, out=None, lse=None, positions=None, use_pdl=True, stream=None):
    """One attention from those over several sets of rows; see ckv_merge_attention in include/ckv.h.

    outs: 1..8 float32/bf16 [T, H, D] of one type, lses: as many float32 [T, H], contiguous;
    positions int32 [T] or None, < 0: a token's rows are left as they are.  Returns (out, lse):
    a new bf16 tensor and a float32 one, or those given (out float32/bf16, it may be one of outs).
    """
    native = _binding or _native()
    if stream is not None:
        _cuda("ckv_merge_attention", *outs)
        with _on(stream):
            out = torch.empty(outs[0].shape, dtype=torch.bfloat16, device=outs[0].device) if out is None else out
            lse = torch.empty(outs[0].shape[:2], dtype=torch.float32, device=outs[0].device) if lse is None else lse
    status, out, lse = native.merge_attention(outs, lses, positions, out, lse, use_pdl, _raw(stream))
    if status:
        _check("ckv_merge_attention", status)
    return out, lse


# ------------------------------------------------------------ contract check
def ckv_check_distinct(ids, id_range, scratch, err_word, stream=None):
    """Flag repeated or out-of-range ids; see ckv_check_distinct in include/ckv.h.

    ids: CUDA int32 or int64 tensor (flattened; negative entries ignored);
    scratch: CUDA int32 tensor of at least ceil(id_range / 32) elements
    (overwritten); err_word: CUDA int32 [1], CKV_DEVERR_DISTINCT (0x40) is
    OR-ed into it on a violation.
    """
    L = load()
    _cuda("ckv_check_distinct", ids, scratch, err_word)
    _need(ids.dtype in (torch.int32, torch.int64) and ids.is_contiguous(), "ids must be contiguous int32/int64")
    _need(scratch.dtype == torch.int32 and scratch.is_contiguous(), "scratch must be contiguous int32")
    _need(err_word.dtype == torch.int32, "err_word must be int32")
    _check("ckv_check_distinct", L.ckv_check_distinct(
        _ptr(ids), ids.element_size(), ids.numel(), int(id_range), _ptr(scratch), scratch.numel(),
        _ptr(err_word), _stream(stream, ids)))


NOALLOC_MAX_RANGE = 1 << 21


def ckv_check_distinct_noalloc(ids, id_range, err_word, stream=None):
    """ckv_check_distinct with the library's own static bitmap (no scratch
    argument, nothing allocated); for callers that cannot allocate device
    memory.  id_range must be at most NOALLOC_MAX_RANGE (2^21).  The first call
    on a device looks up the bitmap's address: make it before any stream
    capture.  Calls that overlap on the GPU share the bitmap and race."""
    L = load()
    _cuda("ckv_check_distinct_noalloc", ids, err_word)
    _need(ids.dtype in (torch.int32, torch.int64) and ids.is_contiguous(), "ids must be contiguous int32/int64")
    _need(err_word.dtype == torch.int32, "err_word must be int32")
    _check("ckv_check_distinct_noalloc", L.ckv_check_distinct_noalloc(
        _ptr(ids), ids.element_size(), ids.numel(), int(id_range), _ptr(err_word), _stream(stream, ids)))


def ckv_latency_probe(hops, n_warps, idx=None, rows=None, out=None, warps_per_cta=4, use_pdl=False, stream=None):
    """Latency floor of a decode-sized launch (see include/ckv.h): hops 0, 1 or
    2 dependent global round trips per warp, 3 for one round trip with the
    pooled decode's first-hop loads, 4 for the pooled decode's memory pattern
    without its arithmetic.  idx int32 [n_warps]; rows and out uint8 [*, 256]
    (out: n_warps rows, 4 * n_warps for hops 4); stream defaults to the current
    stream."""
    L = load()
    _cuda("ckv_latency_probe", idx, rows, out)
    if idx is not None:
        _need(idx.dtype == torch.int32 and idx.is_contiguous() and idx.numel() >= n_warps, "idx must be int32 [n_warps]")
    for t in (rows, out):
        if t is not None:
            _need(t.dtype == torch.uint8 and t.is_contiguous() and t.dim() == 2 and t.shape[1] == 256,
                  "rows/out must be contiguous uint8 [n, 256]")
    if out is not None:
        _need(out.shape[0] >= (4 if hops == 4 else 1) * n_warps, "out must have n_warps rows (4 n_warps for hops 4)")
    num_rows = rows.shape[0] if rows is not None else 0
    if stream is None:
        stream = torch.cuda.current_stream()
    strm = ctypes.c_void_p(stream if isinstance(stream, int) else stream.cuda_stream)
    _check("ckv_latency_probe", L.ckv_latency_probe(int(hops), _ptr(idx), _ptr(rows), num_rows, _ptr(out),
                                                    int(n_warps), int(warps_per_cta), int(bool(use_pdl)), strm))
