"""Thin ctypes binding of ``libindexer.so`` (argument marshalling only).

Every function here has the name of the C entry point it calls (see
``include/indexer.h``) and does nothing but turn torch tensors into raw
pointers and the current CUDA stream into a ``cudaStream_t``.  All compute
runs in the library's CUDA kernels.  If the library has not been built,
loading it raises: there is no other implementation to fall back to.
"""
from __future__ import annotations

import ctypes
import os
import struct
from dataclasses import dataclass
from typing import Optional

import numpy as np
import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libindexer.so")

IDX_OK = 0
IDX_ERR_INVALID_ARG = -1
IDX_ERR_UNSUPPORTED = -2
IDX_ERR_WORKSPACE = -3
IDX_ERR_CUDA = -4
IDX_ERR_TIMEOUT = -5
IDX_ERR_DEVICE_CHECK = -6
IDX_K_FP8_E4M3 = 0
IDX_K_FP4_E2M1_UE8M0 = 1
IDX_Q_FP8_E4M3 = 0
IDX_Q_FP4_E2M1_UE8M0 = 1
IDX_SELECT_AUTO = 0
IDX_SELECT_STREAM = 1
IDX_BF16 = 0
IDX_FP16 = 1
IDX_FP32 = 2
IDX_CODES = 3
IDX_ROPE_HALF = 0
IDX_ROPE_INTERLEAVED = 1
IDX_KV_DENSE = 0
IDX_KV_FP8_E4M3 = 1
IDX_MAX_PARTS = 8

EXPORTED = ("indexer_plan", "indexer_plan_destroy", "indexer_plan_info", "indexer_logits",
            "indexer_topk", "indexer_fused_topk", "indexer_candidate_blocks",
            "indexer_expand_mask", "indexer_status", "indexer_selftest_timeout",
            "indexer_set_wait_budget", "indexer_launch_count", "indexer_error_string",
            "indexer_version", "indexer_fused_topk_noalloc", "indexer_profile_main_kernel",
            "indexer_chunk_rows", "indexer_page_indices", "indexer_candidate_blocks_tail",
            "indexer_fused_topk_mapped", "indexer_convert_fp4", "indexer_fallback_rows",
            "indexer_noalloc_status", "indexer_rope_create", "indexer_rope_destroy",
            "indexer_rope", "indexer_cache_write", "indexer_cache_read", "indexer_page_slots",
            "indexer_attention_create", "indexer_attention_destroy", "indexer_sparse_attention",
            "indexer_mask_blocks", "indexer_cache_append", "indexer_attention_join",
            "indexer_rms_norm", "indexer_causal_attention_create",
            "indexer_causal_attention_destroy", "indexer_causal_attention",
            "indexer_causal_attention_info")
IDX_NOALLOC_SCRATCH_BYTES = 64 << 20


class IndexerError(RuntimeError):
    def __init__(self, fn: str, code: int):
        self.code = code
        super().__init__(f"{fn} failed: {code} ({error_string(code)})")


class _Problem(ctypes.Structure):
    _fields_ = [
        ("num_requests", ctypes.c_int32), ("total_rows", ctypes.c_int32),
        ("total_keys", ctypes.c_int32), ("H", ctypes.c_int32), ("D", ctypes.c_int32),
        ("topk", ctypes.c_int32),
        ("cu_seqlens_q", ctypes.POINTER(ctypes.c_int32)),
        ("cu_seqlens_k", ctypes.POINTER(ctypes.c_int32)),
        ("compress_len", ctypes.POINTER(ctypes.c_int32)),
        ("kdtype", ctypes.c_int32), ("cand_block", ctypes.c_int32),
        ("cand_topk", ctypes.c_int32), ("key_block", ctypes.c_int32),
        ("transient_budget_bytes", ctypes.c_uint64),
        ("select_mode", ctypes.c_int32), ("qdtype", ctypes.c_int32),
    ]


class _RopeSpec(ctypes.Structure):
    _fields_ = [
        ("D", ctypes.c_int32), ("rot_dim", ctypes.c_int32), ("rot_offset", ctypes.c_int32),
        ("layout", ctypes.c_int32), ("base", ctypes.c_double), ("factor", ctypes.c_double),
        ("original_len", ctypes.c_double), ("beta_fast", ctypes.c_double),
        ("beta_slow", ctypes.c_double), ("amplitude", ctypes.c_double),
    ]


class _AttentionSpec(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "Hq", "Hkv", "D", "block", "num_sel", "dtype", "kv_format", "num_slots", "page_size")]
    _fields_ += [("scale", ctypes.c_float)]


class _CausalSpec(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "Hq", "Hkv", "D", "window", "sinks", "dtype", "kv_format", "num_slots", "page_size")]
    _fields_ += [("scale", ctypes.c_float)]


class _AttentionIo(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in (
        "q", "k", "v", "out", "k_scale", "v_scale", "sel", "sel_count", "compress_len",
        "page_table", "lse")]
    _fields_ += [(n, ctypes.c_int64) for n in (
        "q_row", "q_head", "k_slot", "k_head", "v_slot", "v_head", "out_row", "out_head",
        "ld_sel", "ld_page_table")]


# the same layout, packed in one go: eleven addresses, ten strides
_ATTENTION_IO = struct.Struct("11P10q").pack
# indexer_causal_io, indexer_append_io, indexer_join_io and indexer_norm_io
_CAUSAL_IO = struct.Struct("9P9q").pack
_APPEND_IO = struct.Struct("9P9q7i").pack
_JOIN_IO = struct.Struct("16P16q3P2q6i").pack
_NORM_IO = struct.Struct("7P4q5if").pack

_lib = None
_C = torch._C


def lib():
    """Load the library (raises if it is missing)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is not built; run "
                               "python -m sparse_attention_prefill_tcgen05_gb300.build")
        L = ctypes.CDLL(LIB_PATH)
        P, i32, i64, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
        L.indexer_plan.argtypes = [ctypes.POINTER(_Problem), ctypes.POINTER(P),
                                   ctypes.POINTER(sz)]
        L.indexer_plan_destroy.argtypes = [P]
        L.indexer_plan_destroy.restype = None
        L.indexer_plan_info.argtypes = [P, ctypes.POINTER(ctypes.c_int32),
                                        ctypes.POINTER(ctypes.c_int32),
                                        ctypes.POINTER(ctypes.c_int32),
                                        ctypes.POINTER(ctypes.c_int32)]
        L.indexer_logits.argtypes = [P, P, P, P, P, P, P, P, i64, P, sz, P]
        L.indexer_topk.argtypes = [P, P, i64, P, P, P, P, sz, P]
        L.indexer_fused_topk.argtypes = [P, P, P, P, P, P, P, P, i64, P, P, P, sz, P]
        L.indexer_candidate_blocks.argtypes = [P, P, P, P, P, P, P, P, i64, P, sz, P]
        L.indexer_expand_mask.argtypes = [P, P, i64, P, P, i64, P]
        L.indexer_status.argtypes = [P, P, P]
        L.indexer_selftest_timeout.argtypes = [P, ctypes.c_longlong, P]
        L.indexer_set_wait_budget.argtypes = [P, ctypes.c_longlong]
        L.indexer_launch_count.argtypes = []
        L.indexer_profile_main_kernel.argtypes = [P, P]
        L.indexer_profile_main_kernel.restype = None
        L.indexer_fused_topk_noalloc.argtypes = [P, P, P, P, P, P, P, P, i64, P, P, P]
        L.indexer_noalloc_status.argtypes = [P]
        L.indexer_chunk_rows.argtypes = [i64, ctypes.c_double, i32, i32, i32, i32]
        L.indexer_page_indices.argtypes = [P, P, P, i64, i32, P, P]
        L.indexer_convert_fp4.argtypes = [P, P, i64, i32, P, P, P, sz, P]
        L.indexer_candidate_blocks_tail.argtypes = [P, P, P, P, P, P, P, P, P, i64, P, sz, P]
        L.indexer_fused_topk_mapped.argtypes = [P, P, P, P, P, P, P, P, i64, P, i64, P, P, P,
                                                sz, P]
        L.indexer_rope_create.argtypes = [ctypes.POINTER(_RopeSpec), ctypes.POINTER(P)]
        L.indexer_rope_destroy.argtypes = [P]
        L.indexer_rope_destroy.restype = None
        L.indexer_rope.argtypes = [P, P, i32, i32, i32, i64, i64, P, i32, P, i64, i64, P]
        L.indexer_cache_write.argtypes = [P, P, i32, i32, i32, i32, i64, i64, P, P, i32, i32, P,
                                          P, P]
        L.indexer_cache_read.argtypes = [P, P, i32, i32, i32, i32, P, i32, i32, P, P, P]
        L.indexer_page_slots.argtypes = [P, P, i64, i32, P, P]
        L.indexer_attention_create.argtypes = [P, ctypes.POINTER(_AttentionSpec),
                                               ctypes.POINTER(P), ctypes.POINTER(sz)]
        L.indexer_attention_destroy.argtypes = [P]
        L.indexer_attention_destroy.restype = None
        L.indexer_sparse_attention.argtypes = [P, P, P, sz, P]
        L.indexer_mask_blocks.argtypes = [P, P, i64, P, i32, P, i32, P, P]
        L.indexer_causal_attention_create.argtypes = [P, ctypes.POINTER(_CausalSpec),
                                                      ctypes.POINTER(P), ctypes.POINTER(sz)]
        L.indexer_causal_attention_destroy.argtypes = [P]
        L.indexer_causal_attention_destroy.restype = None
        L.indexer_causal_attention.argtypes = [P, P, P, sz, P]
        L.indexer_causal_attention_info.argtypes = [P] + [ctypes.POINTER(ctypes.c_int32)] * 3
        L.indexer_cache_append.argtypes = [P, P, P, P]
        L.indexer_attention_join.argtypes = [P, P]
        L.indexer_rms_norm.argtypes = [P, P]
        L.indexer_error_string.argtypes = [i32]
        L.indexer_error_string.restype = ctypes.c_char_p
        for name in EXPORTED:
            if name not in ("indexer_plan_destroy", "indexer_error_string",
                            "indexer_rope_destroy", "indexer_attention_destroy",
                            "indexer_causal_attention_destroy"):
                getattr(L, name).restype = ctypes.c_int
        L.indexer_launch_count.restype = ctypes.c_longlong
        L.indexer_fallback_rows.argtypes = [P, P, P]
        L.indexer_fallback_rows.restype = ctypes.c_longlong
        _lib = L
    return _lib


def error_string(code: int) -> str:
    try:
        return lib().indexer_error_string(int(code)).decode()
    except Exception:  # library missing: still format the code
        return str(code)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _stream(stream=None):
    """The cudaStream_t of a torch stream (default: the current one of the current device)."""
    if stream is None:
        # the raw handle: building a torch.cuda.Stream object takes longer than a small kernel
        # (no lazy initialisation either: there are CUDA tensors)
        return _C._cuda_getCurrentRawStream(_C._cuda_getDevice())
    return stream.cuda_stream


def _new(stream, make, *args, **kw):
    """A tensor that a call on ``stream`` writes, from that stream's memory: the current stream's may
    still be in use by work queued there."""
    if stream is None:
        return make(*args, **kw)
    with torch.cuda.stream(stream):
        return make(*args, **kw)


def _check(fn: str, rc: int):
    if rc != IDX_OK:
        raise IndexerError(fn, rc)


class Plan:
    """Owns an ``indexer_plan_t``; destroyed with the object."""

    def __init__(self, handle, workspace_bytes: int, problem: _Problem, keepalive):
        self.handle = handle
        self.workspace_bytes = workspace_bytes
        self.problem = problem
        self._keep = keepalive
        keys = keepalive[1]
        self.max_keys = int((keys[1:] - keys[:-1]).max()) if keys.numel() > 1 else 0

    def info(self):
        kb, rc, ns, st = ctypes.c_int32(), ctypes.c_int32(), ctypes.c_int32(), ctypes.c_int32()
        _check("indexer_plan_info", lib().indexer_plan_info(
            self.handle, ctypes.byref(kb), ctypes.byref(rc), ctypes.byref(ns), ctypes.byref(st)))
        return {"key_block": kb.value, "row_chunk": rc.value, "max_splits": ns.value,
                "sample_stride": st.value}

    def __del__(self):
        h, self.handle = getattr(self, "handle", None), None
        if h is not None and _lib is not None:
            _lib.indexer_plan_destroy(h)


def indexer_plan(cu_seqlens_q, cu_seqlens_k, compress_len, H: int, D: int, topk: int,
                 kdtype: int = IDX_K_FP8_E4M3, cand_block: int = 0, cand_topk: int = 0,
                 key_block: int = 0, transient_budget_bytes: int = 0,
                 select_mode: int = 0, qdtype: int = IDX_Q_FP8_E4M3) -> Plan:
    """Host-only planning: lengths are host (CPU) int32 arrays/tensors.  With
    ``qdtype=IDX_Q_FP4_E2M1_UE8M0`` the calls take q as packed e2m1 [T, H, D/2] and its
    ue8m0 block scales [T, H, D/32] (uint8) in the ``s_q`` argument."""
    def host_i32(x):
        t = torch.as_tensor(x).to(device="cpu", dtype=torch.int32).contiguous()
        return t, t.numpy().ctypes.data_as(ctypes.POINTER(ctypes.c_int32))

    cq, pq = host_i32(cu_seqlens_q)
    ck, pk = host_i32(cu_seqlens_k)
    cl, pl = host_i32(compress_len)
    prob = _Problem(num_requests=cq.numel() - 1, total_rows=int(cq[-1]), total_keys=int(ck[-1]),
                    H=H, D=D, topk=topk, cu_seqlens_q=pq, cu_seqlens_k=pk, compress_len=pl,
                    kdtype=kdtype, cand_block=cand_block, cand_topk=cand_topk,
                    key_block=key_block, transient_budget_bytes=transient_budget_bytes,
                    select_mode=select_mode, qdtype=qdtype)
    handle = ctypes.c_void_p()
    ws = ctypes.c_size_t()
    _check("indexer_plan", lib().indexer_plan(ctypes.byref(prob), ctypes.byref(handle),
                                              ctypes.byref(ws)))
    return Plan(handle, ws.value, prob, (cq, ck, cl))


def indexer_logits(plan: Plan, q, s_q, w, k, k_scale, compress_len, logits, ws, stream=None):
    _check("indexer_logits", lib().indexer_logits(
        plan.handle, _ptr(q), _ptr(s_q), _ptr(w), _ptr(k), _ptr(k_scale), _ptr(compress_len),
        _ptr(logits), logits.stride(0), _ptr(ws), ws.numel() * ws.element_size(),
        _stream(stream)))


def indexer_topk(plan: Plan, logits, compress_len, out_idx, out_val, ws, stream=None):
    _check("indexer_topk", lib().indexer_topk(
        plan.handle, _ptr(logits), logits.stride(0), _ptr(compress_len), _ptr(out_idx),
        _ptr(out_val), _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)))


def indexer_fused_topk(plan: Plan, q, s_q, w, k, k_scale, compress_len, cand_mask, out_idx,
                       out_val, ws, stream=None):
    ldm = cand_mask.stride(0) if cand_mask is not None else 0
    _check("indexer_fused_topk", lib().indexer_fused_topk(
        plan.handle, _ptr(q), _ptr(s_q), _ptr(w), _ptr(k), _ptr(k_scale), _ptr(compress_len),
        _ptr(cand_mask), ldm, _ptr(out_idx), _ptr(out_val), _ptr(ws),
        ws.numel() * ws.element_size(), _stream(stream)))


def indexer_candidate_blocks(plan: Plan, q, s_q, w, k, k_scale, compress_len, cand_mask, ws,
                             stream=None):
    _check("indexer_candidate_blocks", lib().indexer_candidate_blocks(
        plan.handle, _ptr(q), _ptr(s_q), _ptr(w), _ptr(k), _ptr(k_scale), _ptr(compress_len),
        _ptr(cand_mask), cand_mask.stride(0), _ptr(ws), ws.numel() * ws.element_size(),
        _stream(stream)))


def indexer_candidate_blocks_tail(plan: Plan, q, s_q, w, k, k_scale, compress_len,
                                  publish_rows, cand_mask, ws, stream=None):
    """Candidate blocks of each request's last ``publish_rows[r]`` rows only, packed into
    ``cand_mask`` [sum(publish_rows), ld_mask] (``publish_rows``: a host sequence)."""
    pr = np.ascontiguousarray(np.asarray(publish_rows, dtype=np.int32))
    _check("indexer_candidate_blocks_tail", lib().indexer_candidate_blocks_tail(
        plan.handle, _ptr(q), _ptr(s_q), _ptr(w), _ptr(k), _ptr(k_scale), _ptr(compress_len),
        pr.ctypes.data_as(ctypes.c_void_p), _ptr(cand_mask), cand_mask.stride(0), _ptr(ws),
        ws.numel() * ws.element_size(), _stream(stream)))


def indexer_fused_topk_mapped(plan: Plan, q, s_q, w, k, k_scale, compress_len, cand_mask,
                              mask_rows, out_idx, out_val, ws, stream=None):
    """indexer_fused_topk where row t reads candidate-mask row ``mask_rows[t]`` (device int32)."""
    _check("indexer_fused_topk_mapped", lib().indexer_fused_topk_mapped(
        plan.handle, _ptr(q), _ptr(s_q), _ptr(w), _ptr(k), _ptr(k_scale), _ptr(compress_len),
        _ptr(cand_mask), cand_mask.stride(0), _ptr(mask_rows), cand_mask.shape[0],
        _ptr(out_idx), _ptr(out_val), _ptr(ws), ws.numel() * ws.element_size(),
        _stream(stream)))


def indexer_expand_mask(plan: Plan, cand_mask, compress_len, key_mask, stream=None):
    _check("indexer_expand_mask", lib().indexer_expand_mask(
        plan.handle, _ptr(cand_mask), cand_mask.stride(0), _ptr(compress_len), _ptr(key_mask),
        key_mask.stride(0), _stream(stream)))


def indexer_status(plan: Optional[Plan], ws, stream=None) -> int:
    return int(lib().indexer_status(plan.handle if plan is not None else None, _ptr(ws),
                                    _stream(stream)))


def indexer_selftest_timeout(ws, cycles: int, stream=None):
    _check("indexer_selftest_timeout",
           lib().indexer_selftest_timeout(_ptr(ws), int(cycles), _stream(stream)))


def indexer_set_wait_budget(plan: Plan, cycles: int):
    _check("indexer_set_wait_budget", lib().indexer_set_wait_budget(plan.handle, int(cycles)))


def indexer_fused_topk_noalloc(plan: Plan, q, s_q, w, k, k_scale, compress_len, cand_mask,
                               out_idx, out_val, stream=None):
    """indexer_fused_topk with the library's fixed device scratch as the workspace."""
    ldm = cand_mask.stride(0) if cand_mask is not None else 0
    _check("indexer_fused_topk_noalloc", lib().indexer_fused_topk_noalloc(
        plan.handle, _ptr(q), _ptr(s_q), _ptr(w), _ptr(k), _ptr(k_scale), _ptr(compress_len),
        _ptr(cand_mask), ldm, _ptr(out_idx), _ptr(out_val), _stream(stream)))


def indexer_noalloc_status(stream=None) -> int:
    """Status word of the last indexer_fused_topk_noalloc call on this device (syncs)."""
    return int(lib().indexer_noalloc_status(_stream(stream)))


def indexer_launch_count() -> int:
    return int(lib().indexer_launch_count())


def indexer_profile_main_kernel(start_event=None, stop_event=None):
    """Record two torch.cuda.Event (already created, timing enabled) around the main
    logits launch of the following top-k calls; no arguments turns it off."""
    h = lambda e: ctypes.c_void_p(e.cuda_event) if e is not None else None
    lib().indexer_profile_main_kernel(h(start_event), h(stop_event))


def indexer_fallback_rows(plan: Plan, ws, stream=None) -> int:
    """Rows the last top-k / candidate call on ``ws`` sent to the exact path (syncs)."""
    n = int(lib().indexer_fallback_rows(plan.handle, _ptr(ws), _stream(stream)))
    if n < 0:
        raise IndexerError("indexer_fallback_rows", n)
    return n


def indexer_version() -> int:
    return int(lib().indexer_version())


def indexer_convert_fp4(codes, block_scales, out_e4m3, out_scale, ws, stream=None):
    """e2m1 + ue8m0/32 rows -> e4m3 rows + fp32 row scales, exactly (see the header);
    ``codes`` [rows, D/2] and ``block_scales`` [rows, D/32] uint8 on the device."""
    rows, half = codes.shape[0], codes.shape[-1]
    _check("indexer_convert_fp4", lib().indexer_convert_fp4(
        _ptr(codes), _ptr(block_scales), rows, 2 * half, _ptr(out_e4m3), _ptr(out_scale),
        _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)))


def indexer_page_indices(plan: Plan, raw_idx, page_table, page_size: int, page_idx=None,
                         stream=None):
    """KV-slot indices of selected raw key indices: page_table[r, j // page_size] *
    page_size + j % page_size, -1 for -1 / out-of-range keys / unmapped pages.  ``raw_idx``
    int32 [rows, topk] and ``page_table`` int32 [requests, ld] on the device; writes into
    ``page_idx`` (default: a new tensor; may be ``raw_idx``) and returns it."""
    if page_idx is None:
        page_idx = _new(stream, torch.empty_like, raw_idx)
    for name, t in (("raw_idx", raw_idx), ("page_table", page_table), ("page_idx", page_idx)):
        if t.dtype != torch.int32 or not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name}: contiguous int32 CUDA tensor expected")
    _check("indexer_page_indices", lib().indexer_page_indices(
        plan.handle, _ptr(raw_idx), _ptr(page_table), page_table.stride(0), int(page_size),
        _ptr(page_idx), _stream(stream)))
    return page_idx


def indexer_chunk_rows(prefix_len: int, budget_token2: float = 2.0e8, chunk_min: int = 256,
                       chunk_max: int = 2048, page: int = 256, pow2: bool = False) -> int:
    """Prefill chunk size for a prefix of ``prefix_len`` compressed keys under a T x L budget
    (the library's host-only planner helper; raises on invalid arguments)."""
    r = int(lib().indexer_chunk_rows(int(prefix_len), float(budget_token2), int(chunk_min),
                                     int(chunk_max), int(page), 1 if pow2 else 0))
    if r < 0:
        raise IndexerError("indexer_chunk_rows", r)
    return r


# ------------------------------------------------------- operators around the indexer
# The checks are written out and pointers passed as plain integers: a call of a decode step
# runs for a few microseconds on the GPU, and as long here.

_INT32 = torch.int32
_DTYPES = {torch.bfloat16: IDX_BF16, torch.float16: IDX_FP16, torch.float32: IDX_FP32}
# what codes and masks come in: bytes, or the type itself
_E4M3 = frozenset((torch.uint8, torch.int8, torch.float8_e4m3fn))
_E2M1 = frozenset((torch.uint8, torch.int8)
                  + ((torch.float4_e2m1fn_x2,) if hasattr(torch, "float4_e2m1fn_x2") else ()))
_E8M0 = frozenset((torch.uint8, torch.int8)
                  + ((torch.float8_e8m0fnu,) if hasattr(torch, "float8_e8m0fnu") else ()))
_FLOAT = frozenset((torch.float32,))
_MASK = frozenset((torch.uint8, torch.int8, torch.bool))


def _dense(name: str, t):
    """Type code and strides of a 3-d CUDA tensor whose last axis is contiguous."""
    code = _DTYPES.get(t.dtype)
    st = t.stride()
    if code is None or len(st) != 3 or not t.is_cuda:
        raise ValueError(f"{name}: 3-d bf16, fp16 or fp32 CUDA tensor expected")
    if st[2] != 1 and t.shape[2] > 1:
        raise ValueError(f"{name}: a contiguous last axis expected")
    return code, st


def _i32(name: str, t, shape):
    """Address of a contiguous int32 CUDA tensor of that shape, or None."""
    if t is None:
        return None
    if t.dtype is not _INT32 or t.shape != shape or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name}: contiguous int32 CUDA tensor of shape {tuple(shape)} expected")
    return t.data_ptr()


class Rope:
    """Owns an ``indexer_rope_t``; destroyed with the object."""

    def __init__(self, handle, spec: _RopeSpec):
        self.handle = handle
        self.spec = spec
        self.D = spec.D

    def __del__(self):
        h, self.handle = getattr(self, "handle", None), None
        if h is not None and _lib is not None:
            _lib.indexer_rope_destroy(h)


def indexer_rope_create(D: int, rot_dim: int, rot_offset: int = 0, layout: int = IDX_ROPE_HALF,
                        base: float = 10000.0, factor: float = 1.0, original_len: float = 0.0,
                        beta_fast: float = 32.0, beta_slow: float = 1.0,
                        amplitude: float = 1.0) -> Rope:
    """A rotation of ``rot_dim`` of a head vector's ``D`` elements (host only; see the header
    for the scaling of long contexts)."""
    spec = _RopeSpec(D, rot_dim, rot_offset, layout, base, factor, original_len, beta_fast,
                     beta_slow, amplitude)
    handle = ctypes.c_void_p()
    _check("indexer_rope_create", lib().indexer_rope_create(ctypes.byref(spec),
                                                            ctypes.byref(handle)))
    return Rope(handle, spec)


def indexer_rope(rope: Rope, x, positions, out=None, inverse: bool = False, stream=None):
    """Rotate ``x`` [rows, heads, D] at ``positions`` (int32 [rows]) into ``out`` (default: a
    new tensor; may be ``x``) and return it; ``inverse`` turns back."""
    code, sx = _dense("x", x)
    if out is None:
        out = _new(stream, torch.empty_like, x)
    shape = x.shape
    rows, heads, D = shape
    ocode, so = (code, sx) if out is x else _dense("out", out)
    if ocode != code or out.shape != shape or D != rope.D:
        raise ValueError("out: a tensor of x's shape and type, D elements a head, expected")
    rc = (_lib or lib()).indexer_rope(rope.handle, x.data_ptr(), code, rows, heads, sx[0], sx[1],
                            _i32("positions", positions, (rows,)), 1 if inverse else 0,
                            out.data_ptr(), so[0], so[1], _stream(stream))
    if rc != IDX_OK:
        raise IndexerError("indexer_rope", rc)
    return out


def _cache_shape(codes, scales, fmt: int):
    """(slots, heads, D) of a cache's codes and scales."""
    slots, heads, n = codes.shape
    if fmt == IDX_K_FP4_E2M1_UE8M0:
        D, want, kind, name = 2 * n, (slots, heads, n // 16), _E2M1, "e2m1 codes and ue8m0"
        scale_kind = _E8M0
    else:
        D, want, kind, name = n, (slots, heads), _E4M3, "e4m3 codes and fp32"
        scale_kind = _FLOAT
    if (codes.dtype not in kind or scales.dtype not in scale_kind or scales.shape != want
            or not codes.is_cuda or not scales.is_cuda or not codes.is_contiguous()
            or not scales.is_contiguous()):
        raise ValueError(f"cache: contiguous CUDA {name} scales (or their bytes) of shape {want} "
                         "expected")
    return slots, heads, D


def indexer_cache_write(x, codes, scales, fmt: int = IDX_K_FP8_E4M3, rope: Optional[Rope] = None,
                        positions=None, slots=None, stream=None):
    """Rotate (``rope``) and quantise ``x`` [rows, heads, D] into rows ``slots`` (int32 [rows];
    default: row i) of a cache: ``codes`` [num_slots, heads, D] (e2m1: D/2) and ``scales``."""
    n, heads, D = _cache_shape(codes, scales, fmt)
    code, sx = _dense("x", x)
    rows, x_heads, x_D = x.shape
    if x_heads != heads or x_D != D:
        raise ValueError(f"x: [rows, {heads}, {D}] expected")
    shape = (rows,)
    rc = (_lib or lib()).indexer_cache_write(
        None if rope is None else rope.handle, x.data_ptr(), code, rows, heads, D, sx[0], sx[1],
        _i32("positions", positions, shape), _i32("slots", slots, shape), n, fmt,
        codes.data_ptr(), scales.data_ptr(), _stream(stream))
    if rc != IDX_OK:
        raise IndexerError("indexer_cache_write", rc)


def indexer_cache_read(codes, scales, fmt: int, slots, out, out_scales=None, stream=None):
    """Rows ``slots`` (int32 [rows]; None: row i) of a cache into ``out``: as bf16, fp16 or fp32
    values [rows, heads, D], or, with ``out_scales``, as packed codes and scales."""
    n, heads, D = _cache_shape(codes, scales, fmt)
    rows = out.shape[0]
    if out_scales is not None:
        code = IDX_CODES
        if _cache_shape(out, out_scales, fmt) != (rows, heads, D):
            raise ValueError("out: codes of the cache's heads and size expected")
    else:
        code, _ = _dense("out", out)
        if out.shape != (rows, heads, D) or not out.is_contiguous():
            raise ValueError(f"out: contiguous [rows, {heads}, {D}] expected")
    rc = (_lib or lib()).indexer_cache_read(
        codes.data_ptr(), scales.data_ptr(), fmt, n, heads, D, _i32("slots", slots, (rows,)), rows,
        code, out.data_ptr(), _ptr(out_scales), _stream(stream))
    if rc != IDX_OK:
        raise IndexerError("indexer_cache_read", rc)
    return out


def indexer_page_slots(plan: Plan, page_table, page_size: int, slots=None, stream=None):
    """Cache slots of the batch's packed keys (int32 [total_keys]) from a page table."""
    if slots is None:
        slots = _new(stream, torch.empty, plan.problem.total_keys, dtype=torch.int32,
                     device=page_table.device)
    table = _i32("page_table", page_table, (plan.problem.num_requests, page_table.shape[-1]))
    _check("indexer_page_slots", lib().indexer_page_slots(
        plan.handle, table, page_table.shape[1], int(page_size),
        _i32("slots", slots, (plan.problem.total_keys,)), _stream(stream)))
    return slots


class Attention:
    """Owns an ``indexer_attention_t``; destroyed with the object."""

    def __init__(self, handle, workspace_bytes: int, spec: _AttentionSpec, rows: int,
                 requests: int, max_keys: int):
        self.handle = handle
        self.workspace_bytes = workspace_bytes
        self.spec = spec
        self.rows = rows
        self.requests = requests
        self.pages = -(-max_keys // spec.page_size) if spec.page_size > 0 else 0
        # what the tensors of a call are compared with
        self.dtype = torch.bfloat16 if spec.dtype == IDX_BF16 else torch.float16
        self.dense = spec.kv_format == IDX_KV_DENSE
        self.row_shape = (rows,)
        self.q_shape = (rows, spec.Hq, spec.D)
        self.kv_shape = (spec.num_slots, spec.Hkv, spec.D)
        self.sel_shape = (rows, spec.num_sel)
        self.scale_shape = (spec.num_slots, spec.Hkv)
        self.lse_shape = (rows, spec.Hq)

    def __del__(self):
        h, self.handle = getattr(self, "handle", None), None
        if h is not None and _lib is not None:
            _lib.indexer_attention_destroy(h)


def indexer_attention_create(plan: Plan, Hq: int, Hkv: int, D: int, num_sel: int, block: int = 1,
                             dtype: int = IDX_BF16, kv_format: int = IDX_KV_DENSE,
                             num_slots: Optional[int] = None, page_size: int = 0,
                             scale: Optional[float] = None) -> Attention:
    """Attention over ``num_sel`` selected keys (or blocks of ``block`` keys) a row for the
    plan's batch (host only).  ``num_slots`` rows of k and v (default: the packed keys),
    ``scale`` 1/sqrt(D) by default."""
    spec = _AttentionSpec(Hq, Hkv, D, block, num_sel, dtype, kv_format,
                          plan.problem.total_keys if num_slots is None else num_slots, page_size,
                          max(D, 1) ** -0.5 if scale is None else scale)
    handle, ws = ctypes.c_void_p(), ctypes.c_size_t()
    _check("indexer_attention_create", lib().indexer_attention_create(
        plan.handle, ctypes.byref(spec), ctypes.byref(handle), ctypes.byref(ws)))
    return Attention(handle, ws.value, spec, plan.problem.total_rows, plan.problem.num_requests,
                     plan.max_keys)


def _packed(t):
    """Whether a row's elements are neighbours (a single one has any stride)."""
    return t.stride(1) == 1 or t.shape[1] <= 1


def _heads(name: str, t, shape, dtype):
    """Strides of a CUDA tensor of that shape and type (None: e4m3 codes or their bytes)."""
    if t.shape != shape or not t.is_cuda or \
            (t.dtype not in _E4M3 if dtype is None else t.dtype != dtype):
        raise ValueError(f"{name}: CUDA tensor {shape} of {dtype or 'e4m3 codes'} expected")
    st = t.stride()
    if st[2] != 1:
        raise ValueError(f"{name}: a contiguous last axis expected")
    return st


def _f32(name: str, t, shape):
    """Address of a contiguous fp32 CUDA tensor of that shape (0: none)."""
    if t is None:
        return 0
    if t.dtype != torch.float32 or t.shape != shape or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name}: contiguous fp32 CUDA tensor {shape} expected")
    return t.data_ptr()


def indexer_sparse_attention(attn: Attention, q, k, v, sel, compress_len, out, ws=None,
                             k_scale=None, v_scale=None, sel_count=None, page_table=None,
                             lse=None, stream=None):
    """Attention of ``q`` [rows, Hq, D] over the keys ``sel`` (int32 [rows, num_sel]) of ``k`` and
    ``v`` [num_slots, Hkv, D] into ``out`` (and ``lse`` fp32 [rows, Hq]); see the header."""
    kv_type = attn.dtype if attn.dense else None
    sq = _heads("q", q, attn.q_shape, attn.dtype)
    so = _heads("out", out, attn.q_shape, attn.dtype)
    sk = _heads("k", k, attn.kv_shape, kv_type)
    sv = _heads("v", v, attn.kv_shape, kv_type)
    if sel.dtype != torch.int32 or sel.shape != attn.sel_shape or not sel.is_cuda or \
            not _packed(sel):
        raise ValueError(f"sel: int32 CUDA tensor {attn.sel_shape} expected")
    table = ld_table = 0
    if page_table is not None:
        if page_table.dtype != torch.int32 or page_table.dim() != 2 or not page_table.is_cuda or \
                page_table.shape[0] != attn.requests or page_table.shape[1] < attn.pages or \
                not _packed(page_table):
            raise ValueError(f"page_table: int32 CUDA tensor [requests, {attn.pages} pages or more] "
                             "expected")
        table = page_table.data_ptr()
        ld_table = page_table.stride(0) if attn.requests > 1 else page_table.shape[1]
    io = _ATTENTION_IO(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
        _f32("k_scale", k_scale, attn.scale_shape), _f32("v_scale", v_scale, attn.scale_shape),
        sel.data_ptr(), _i32("sel_count", sel_count, attn.row_shape) or 0,
        _i32("compress_len", compress_len, attn.row_shape) or 0, table,
        _f32("lse", lse, attn.lse_shape), sq[0], sq[1], sk[0], sk[1], sv[0], sv[1], so[0], so[1],
        sel.stride(0) if attn.rows > 1 else attn.spec.num_sel, ld_table)
    rc = (_lib or lib()).indexer_sparse_attention(
        attn.handle, io, _ptr(ws), 0 if ws is None else ws.numel() * ws.element_size(),
        _stream(stream))
    if rc != IDX_OK:
        raise IndexerError("indexer_sparse_attention", rc)
    return out


def indexer_mask_blocks(plan: Plan, cand_mask, compress_len, block: int, blocks, count=None,
                        stream=None):
    """The candidate blocks of every mask row as a list: ``blocks`` int32 [rows, num_sel]
    (ascending, then -1) and ``count`` int32 [rows]."""
    rows = plan.problem.total_rows
    need = -(-plan.max_keys // block) if block > 0 else 0
    if cand_mask.dtype not in _MASK or not cand_mask.is_cuda or cand_mask.dim() != 2 or \
            cand_mask.shape[0] != rows or cand_mask.shape[1] < need or not _packed(cand_mask):
        raise ValueError(f"cand_mask: CUDA tensor [rows, {need} blocks or more] of bytes or truth values "
                         "expected")
    num_sel, shape = blocks.shape[-1], (rows,)
    rc = (_lib or lib()).indexer_mask_blocks(
        plan.handle, cand_mask.data_ptr(), cand_mask.stride(0) if rows > 1 else cand_mask.shape[1],
        _i32("compress_len", compress_len, shape), int(block),
        _i32("blocks", blocks, (rows, num_sel)), num_sel, _i32("count", count, shape),
        _stream(stream))
    if rc != IDX_OK:
        raise IndexerError("indexer_mask_blocks", rc)
    return blocks


class CausalAttention:
    """Owns an ``indexer_causal_t``; destroyed with the object."""

    def __init__(self, handle, workspace_bytes: int, spec: _CausalSpec, rows: int, requests: int,
                 max_keys: int):
        self.handle = handle
        self.workspace_bytes = workspace_bytes
        self.spec = spec
        self.rows = rows
        self.requests = requests
        self.pages = -(-max_keys // spec.page_size) if spec.page_size > 0 else 0
        # what the tensors of a call are compared with
        self.dtype = torch.bfloat16 if spec.dtype == IDX_BF16 else torch.float16
        self.kv_type = self.dtype if spec.kv_format == IDX_KV_DENSE else None
        self.row_shape = (rows,)
        self.q_shape = (rows, spec.Hq, spec.D)
        self.kv_shape = (spec.num_slots, spec.Hkv, spec.D)
        self.scale_shape = (spec.num_slots, spec.Hkv)
        self.lse_shape = (rows, spec.Hq)

    def info(self):
        n = [ctypes.c_int32() for _ in range(3)]
        _check("indexer_causal_attention_info",
               lib().indexer_causal_attention_info(self.handle, *map(ctypes.byref, n)))
        return dict(zip(("tiles", "blocks", "joined"), (x.value for x in n)))

    def __del__(self):
        h, self.handle = getattr(self, "handle", None), None
        if h is not None and _lib is not None:
            _lib.indexer_causal_attention_destroy(h)


def indexer_causal_attention_create(plan: Plan, Hq: int, Hkv: int, D: int, window: int = 0,
                                    sinks: int = 0, dtype: int = IDX_BF16,
                                    kv_format: int = IDX_KV_DENSE,
                                    num_slots: Optional[int] = None, page_size: int = 0,
                                    scale: Optional[float] = None) -> CausalAttention:
    """Causal attention of the plan's rows over their requests' cached keys (host only): all of
    them, or with ``window`` > 0 the last ``window`` and the first ``sinks``."""
    spec = _CausalSpec(Hq, Hkv, D, window, sinks, dtype, kv_format,
                       plan.problem.total_keys if num_slots is None else num_slots, page_size,
                       max(D, 1) ** -0.5 if scale is None else scale)
    handle, ws = ctypes.c_void_p(), ctypes.c_size_t()
    _check("indexer_causal_attention_create", lib().indexer_causal_attention_create(
        plan.handle, ctypes.byref(spec), ctypes.byref(handle), ctypes.byref(ws)))
    return CausalAttention(handle, ws.value, spec, plan.problem.total_rows,
                           plan.problem.num_requests, plan.max_keys)


def indexer_causal_attention(attn: CausalAttention, q, k, v, compress_len, out, ws=None,
                             k_scale=None, v_scale=None, page_table=None, lse=None, stream=None):
    """Attention of ``q`` [rows, Hq, D] over the keys below ``compress_len`` (int32 [rows]) of ``k``
    and ``v`` [num_slots, Hkv, D] into ``out`` (and ``lse`` fp32 [rows, Hq]); see the header."""
    sq = _heads("q", q, attn.q_shape, attn.dtype)
    so = _heads("out", out, attn.q_shape, attn.dtype)
    sk = _heads("k", k, attn.kv_shape, attn.kv_type)
    sv = _heads("v", v, attn.kv_shape, attn.kv_type)
    table = ld_table = 0
    if page_table is not None:
        if page_table.dtype != torch.int32 or page_table.dim() != 2 or not page_table.is_cuda or \
                page_table.shape[0] != attn.requests or page_table.shape[1] < attn.pages or \
                not _packed(page_table):
            raise ValueError(f"page_table: int32 CUDA tensor [requests, {attn.pages} pages or more] "
                             "expected")
        table = page_table.data_ptr()
        ld_table = page_table.stride(0) if attn.requests > 1 else page_table.shape[1]
    io = _CAUSAL_IO(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
        _f32("k_scale", k_scale, attn.scale_shape), _f32("v_scale", v_scale, attn.scale_shape),
        _i32("compress_len", compress_len, attn.row_shape) or 0, table,
        _f32("lse", lse, attn.lse_shape), sq[0], sq[1], sk[0], sk[1], sv[0], sv[1], so[0], so[1],
        ld_table)
    rc = (_lib or lib()).indexer_causal_attention(
        attn.handle, io, _ptr(ws), 0 if ws is None else ws.numel() * ws.element_size(),
        _stream(stream))
    if rc != IDX_OK:
        raise IndexerError("indexer_causal_attention", rc)
    return out


def _cache_rows(name: str, t, shape, dtype):
    """Strides of a cache of [num_slots, heads, D] elements (dtype None: e4m3 codes or bytes)."""
    if t.dim() != 3 or t.shape[1:] != shape or not t.is_cuda or \
            (t.dtype not in _E4M3 if dtype is None else t.dtype != dtype):
        raise ValueError(f"{name}: CUDA tensor [num_slots, {shape[0]}, {shape[1]}] of "
                         f"{dtype or 'e4m3 codes'} expected")
    st = t.stride()
    if st[2] != 1 and shape[1] > 1:
        raise ValueError(f"{name}: a contiguous last axis expected")
    # a single slot's or head's stride says nothing
    return st[0] if t.shape[0] > 1 else shape[0] * shape[1], st[1] if shape[0] > 1 else shape[1]


def indexer_cache_append(plan: Optional[Plan], k, v, k_cache, v_cache, positions,
                         rope: Optional[Rope] = None, page_table=None, page_size: int = 0,
                         slots=None, k_scale=None, v_scale=None, stream=None):
    """Write the batch's new ``k`` (turned by ``rope``) and ``v`` [rows, heads, D] into their caches
    [num_slots, heads, D]: of a 16-bit type, or e4m3 codes with ``k_scale`` and ``v_scale``
    [num_slots, heads].  Row t goes to its request's key ``positions[t]`` (int32 [rows]), through
    ``page_table`` [requests, pages] with ``page_size`` > 0, or to ``slots[t]``."""
    code, sk = _dense("k", k)
    vcode, sv = _dense("v", v)
    shape = k.shape
    rows, heads, D = shape
    if vcode != code or v.shape != shape:
        raise ValueError("v: a tensor of k's shape and type expected")
    if k_scale is None and v_scale is None:
        kind = k_cache.dtype
        cache_code = _DTYPES.get(kind, -1)
    else:
        kind, cache_code = None, IDX_CODES
    num_slots = k_cache.shape[0]
    kc, vc = _cache_rows("k_cache", k_cache, shape[1:], kind), \
        _cache_rows("v_cache", v_cache, shape[1:], kind)
    if v_cache.shape[0] != num_slots:
        raise ValueError("v_cache: as many slots as k_cache expected")
    if cache_code == IDX_CODES and (k_scale is None or v_scale is None):
        raise ValueError("k_scale and v_scale: both or none expected")
    scales = (num_slots, heads)
    table = ld_table = 0
    if page_size > 0 and slots is None:
        if plan is None or page_table is None:
            raise ValueError("page_size: a plan and its page_table expected")
        requests, pages = plan.problem.num_requests, -(-plan.max_keys // page_size)
        if page_table.dtype != torch.int32 or page_table.dim() != 2 or not page_table.is_cuda or \
                page_table.shape[0] != requests or page_table.shape[1] < pages or \
                not _packed(page_table):
            raise ValueError(f"page_table: int32 CUDA tensor [requests, {pages} pages or more] "
                             "expected")
        table = page_table.data_ptr()
        ld_table = page_table.stride(0) if requests > 1 else page_table.shape[1]
    elif page_table is not None and slots is None:
        raise ValueError("page_table: a page_size expected")
    io = _APPEND_IO(
        k.data_ptr(), v.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
        _f32("k_scale", k_scale, scales), _f32("v_scale", v_scale, scales),
        _i32("positions", positions, (rows,)) or 0, _i32("slots", slots, (rows,)) or 0, table,
        sk[0], sk[1], sv[0], sv[1], kc[0], kc[1], vc[0], vc[1], ld_table, rows, heads, D, code,
        cache_code, num_slots, page_size)
    rc = (_lib or lib()).indexer_cache_append(
        None if plan is None else plan.handle, None if rope is None else rope.handle, io,
        _stream(stream))
    if rc != IDX_OK:
        raise IndexerError("indexer_cache_append", rc)


_NO_PARTS = (0,) * IDX_MAX_PARTS


def indexer_attention_join(outs, lses, out=None, lse=None, sink=None, stream=None):
    """Join attention outputs ``outs`` [rows, heads, D] over disjoint keys by their log-sum-exps
    ``lses`` (fp32 [rows, heads]) into ``out`` (default: a new tensor of their type; may be one of
    them, as it is) and ``lse``; ``sink`` fp32 [heads]: the logit of attending to nothing."""
    n = len(outs)
    if n < 1 or n > IDX_MAX_PARTS or len(lses) != n:
        raise ValueError(f"outs, lses: 1 to {IDX_MAX_PARTS} parts each expected")
    first = outs[0]
    shape, dtype = first.shape, first.dtype
    if len(shape) != 3 or dtype not in _DTYPES:
        raise ValueError("outs: 3-d bf16, fp16 or fp32 CUDA tensors expected")
    rows, heads, D = shape
    ml = (rows, heads)
    parts, part_lses, row, head = [], [], [], []
    for o, l in zip(outs, lses):
        if o.shape != shape or o.dtype != dtype or not o.is_cuda:
            raise ValueError("outs: CUDA tensors of one shape and type expected")
        if l is None or l.dtype != torch.float32 or l.shape != ml or not l.is_cuda or \
                not l.is_contiguous():
            raise ValueError(f"lses: contiguous fp32 CUDA tensors {ml} expected")
        st = o.stride()
        if st[2] != 1 and D > 1:
            raise ValueError("outs: a contiguous last axis expected")
        parts.append(o.data_ptr())
        part_lses.append(l.data_ptr())
        row.append(st[0])
        head.append(st[1])
    if out is None:
        out = _new(stream, torch.empty, shape, dtype=dtype, device=first.device)
    ocode, so = _dense("out", out)
    if out.shape != shape:
        raise ValueError(f"out: [{rows}, {heads}, {D}] expected")
    pad = _NO_PARTS[n:]
    rc = (_lib or lib()).indexer_attention_join(
        _JOIN_IO(*parts, *pad, *part_lses, *pad, *row, *pad, *head, *pad, out.data_ptr(),
                 _f32("lse", lse, ml), _f32("sink", sink, (heads,)),
                 so[0] if rows > 1 else D, so[1] if heads > 1 else D,
                 n, rows, heads, D, _DTYPES[dtype], ocode), _stream(stream))
    if rc != IDX_OK:
        raise IndexerError("indexer_attention_join", rc)
    return out


def _matrix(name: str, t, shape, dtype):
    """Address and row stride of a CUDA matrix with neighbouring elements (0, 0: none)."""
    if t is None:
        return 0, 0
    if t.shape != shape or t.dtype != dtype or not t.is_cuda:
        raise ValueError(f"{name}: CUDA tensor {tuple(shape)} of {dtype} expected")
    st = t.stride()
    if st[1] != 1 and shape[1] > 1:
        raise ValueError(f"{name}: a contiguous last axis expected")
    return t.data_ptr(), st[0] if shape[0] > 1 else shape[1]


def indexer_rms_norm(x, weight=None, eps: float = 1e-6, residual=None, total=None, out=None,
                     codes=None, scales=None, stream=None):
    """Norm of ``x`` [rows, n] (plus ``residual``, the sum into ``total``) times ``weight`` [n] into
    ``out`` (default: a new tensor, unless ``codes`` are asked for) and, as e4m3, into ``codes``
    [rows, n] with ``scales`` fp32 [rows, n / group].  Returns ``out``."""
    shape, dtype = x.shape, x.dtype
    code = _DTYPES.get(dtype)
    if code is None or len(shape) != 2:
        raise ValueError("x: 2-d bf16, fp16 or fp32 CUDA tensor expected")
    rows, n = shape
    if out is None and codes is None:
        out = _new(stream, torch.empty, shape, dtype=dtype, device=x.device)
    px, sx = _matrix("x", x, shape, dtype)
    pr, sr = _matrix("residual", residual, shape, dtype)
    pt, st = _matrix("total", total, shape, dtype)
    po, so = _matrix("out", out, shape, dtype)
    pw, wcode = 0, code
    if weight is not None:
        wcode = _DTYPES.get(weight.dtype, -1)
        if weight.shape != shape[1:] or not weight.is_cuda or not weight.is_contiguous():
            raise ValueError(f"weight: contiguous CUDA tensor ({n},) expected")
        pw = weight.data_ptr()
    pc = ps = group = 0
    if codes is not None:
        if codes.dtype not in _E4M3 or codes.shape != shape or not codes.is_cuda or \
                not codes.is_contiguous():
            raise ValueError(f"codes: contiguous CUDA tensor {tuple(shape)} of e4m3 codes expected")
        groups = 0 if scales is None or scales.dim() != 2 else scales.shape[1]
        if groups < 1 or n % groups != 0:
            raise ValueError("scales: fp32 CUDA tensor [rows, n / group] expected")
        group = n // groups
        pc, ps = codes.data_ptr(), _f32("scales", scales, (rows, groups))
    elif scales is not None:
        raise ValueError("scales: codes expected")
    rc = (_lib or lib()).indexer_rms_norm(
        _NORM_IO(px, pr, pw, pt, po, pc, ps, sx, sr, st, so, rows, n, group, code, wcode, eps),
        _stream(stream))
    if rc != IDX_OK:
        raise IndexerError("indexer_rms_norm", rc)
    return out
