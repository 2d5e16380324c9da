"""Fused flash-style GQA attention for NVIDIA GB300 (sm_103a).

Thin Python binding over the C ABI in ``include/attn.h`` (``libattn_gb300.so``):
argument marshalling only (by ctypes; for the calls that are short on the GPU by the native
module ``_ops``). Every step of the computation runs in the library's
CUDA kernels; there is no CPU or PyTorch fallback, and importing a function whose
library is missing raises immediately.

PyTorch is used for device memory and streams: tensors are passed by data pointer,
outputs and workspaces are allocated with ``torch.empty`` when not supplied, and
work is queued on the current CUDA stream unless ``stream`` is given.

Entry points (same names as the C ABI):

* ``attn_fwd(q, k, v, ...)``          q [B,S,Hq,D], k/v [B,S,Hkv,D] -> (o, lse[B,Hq,S])
* ``attn_fwd_varlen(q, k, v, cu_seqlens, max_seqlen, ...)``  packed [T,H,D] -> (o, lse[Hq,T])
* ``attn_fwd_paged(q, k_cache, v_cache, block_table, seq_lens, cu_q, max_q_len, ...)``
  chunked prefill over a paged cache: packed new tokens [T,Hq,D] -> (o, lse[Hq,T])
* ``attn_bwd(q, k, v, o, lse, dO, ...)``  -> (dQ, dK, dV); dense or packed (cu_seqlens)
* ``attn_merge_lse(o_parts, lse_parts, ...)`` attention results over disjoint key sets -> (o, lse)
* ``attn_decode_paged(q, k_cache, v_cache, block_table, seq_lens, ...)`` -> (o, lse[B,Hq])
* ``attn_paged_plan(kv_lens, new_lens, free_pages, block_table, pages_held, free_used, total_new, ...)``
  pages, positions and cache slots of a serving step, from request lengths -> PagedPlan
* ``attn_qk_norm_rope(q, k, q_weight, k_weight, positions, cos_sin, ...)`` RMS norm of every head and
  rotary position encoding -> (q_out, k_out); ``attn_qk_norm_rope_bwd`` its gradient;
  ``attn_qk_norm_rope_paged`` the same with K and V written into the paged caches by slot -> q_out
* ``attn_tree_paged(q, k_cache, v_cache, block_table, seq_lens, cu_q, tree_mask, max_q_len, ...)``
  drafted token trees over a paged cache: packed rows [T,Hq,D] -> (o, lse[Hq,T])
* ``attn_workspace_size``, ``attn_bwd_sink_workspace_size``, ``attn_get_device_status``, ``attn_status_string``
* ``sink=`` of attn_fwd, attn_fwd_varlen, attn_fwd_paged, attn_bwd and attn_decode_paged: with a window, a sequence's first keys
  that stay visible past it
* ``attn_kv4_append(k, v, slots, kv_cache)`` keys and values into a paged cache of 4-bit codes, ``attn_kv4_unpack(kv_cache, pages)``
  its pages back as bf16, ``attn_decode_kv4(q, kv_cache, block_table, seq_lens, ...)`` decode over it -> (o, lse[B,Hq])
* ``attn_selftest_wait_timeout`` (exercises the bounded-wait failure reporting)
"""
from __future__ import annotations

import ctypes
import math
import os
import threading
from typing import Any, NamedTuple

__all__ = [
    "AttnError", "attn_fwd", "attn_fwd_varlen", "attn_fwd_paged", "attn_bwd", "attn_decode_paged", "attn_workspace_size",
    "attn_get_device_status", "attn_status_string", "library_path", "load_library",
    "attn_launch_count", "attn_profile_start", "attn_profile_stop", "attn_decode_paged_noalloc",
    "attn_selftest_wait_timeout", "attn_merge_lse", "attn_paged_plan", "PagedPlan", "attn_qk_norm_rope",
    "attn_qk_norm_rope_bwd", "attn_qk_norm_rope_paged", "attn_tree_paged", "attn_kv4_append", "attn_kv4_unpack", "attn_decode_kv4",
    "attn_bwd_sink_workspace_size",
    "ATTN_OP_FWD", "ATTN_OP_FWD_VARLEN", "ATTN_OP_BWD", "ATTN_OP_BWD_VARLEN", "ATTN_OP_DECODE_PAGED",
    "ATTN_OP_QK_NORM_ROPE_BWD", "ATTN_OP_TREE_PAGED", "ATTN_OP_DECODE_KV4",
]

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_HERE, "libattn_gb300.so")
_lock = threading.Lock()
_lib = None

ATTN_OP_FWD, ATTN_OP_FWD_VARLEN, ATTN_OP_BWD, ATTN_OP_BWD_VARLEN, ATTN_OP_DECODE_PAGED = 0, 1, 2, 3, 4
ATTN_OP_QK_NORM_ROPE_BWD, ATTN_OP_TREE_PAGED, ATTN_OP_DECODE_KV4 = 5, 6, 7
STATUS = {0: "ATTN_OK", 1: "ATTN_ERR_INVALID_ARG", 2: "ATTN_ERR_UNSUPPORTED", 3: "ATTN_ERR_MISALIGNED",
          4: "ATTN_ERR_WORKSPACE", 5: "ATTN_ERR_LAUNCH", 6: "ATTN_ERR_DEVICE_TIMEOUT", 7: "ATTN_ERR_DEVICE_BOUNDS",
          8: "ATTN_ERR_NO_DEVICE"}


class AttnError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {STATUS.get(status, status)}")
        self.status = status


def library_path() -> str:
    return _LIB_PATH


def load_library():
    """Load libattn_gb300.so (raises if it has not been built)."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(_LIB_PATH):
            raise RuntimeError(f"{_LIB_PATH} is missing: build it first (python -m attention_flash_gqa_gb300._build "
                               "or __graft_entry__.build()); there is no fallback implementation")
        lib = ctypes.CDLL(_LIB_PATH)
        P, I, F, Z = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
        lib.attn_fwd.argtypes = [P, P, P, P, P, I, I, I, I, I, F, I, I, P, Z, P]
        lib.attn_fwd_varlen.argtypes = [P, P, P, P, P, P, I, I, I, I, I, I, F, I, I, P, Z, P]
        lib.attn_fwd_paged.argtypes = [P, P, P, P, P, P, P, P, I, I, I, I, I, I, I, I, I, F, I, I, P]
        lib.attn_fwd_sink.argtypes = [P, P, P, P, P, I, I, I, I, I, F, I, I, I, P, Z, P]
        lib.attn_fwd_varlen_sink.argtypes = [P, P, P, P, P, P, I, I, I, I, I, I, F, I, I, I, P, Z, P]
        lib.attn_fwd_paged_sink.argtypes = [P, P, P, P, P, P, P, P, I, I, I, I, I, I, I, I, I, F, I, I, I, P]
        lib.attn_bwd_sink.argtypes = [P, P, P, P, P, P, P, P, P, I, I, I, I, I, F, I, I, I, P, I, I, P, Z, P]
        lib.attn_bwd_sink_workspace_size.argtypes = [I] * 8
        lib.attn_bwd_sink_workspace_size.restype = Z
        lib.attn_decode_paged_sink.argtypes = [P, P, P, P, P, P, P, I, I, I, I, I, I, I, F, I, I, P, Z, P]
        for f in (lib.attn_fwd_sink, lib.attn_fwd_varlen_sink, lib.attn_fwd_paged_sink, lib.attn_bwd_sink,
                  lib.attn_decode_paged_sink):
            f.restype = I
        lib.attn_merge_lse.argtypes = [P, P, P, P, I, I, I, I, I, P]
        lib.attn_merge_lse.restype = I
        lib.attn_bwd.argtypes = [P, P, P, P, P, P, P, P, P, I, I, I, I, I, F, I, I, P, I, I, P, Z, P]
        lib.attn_decode_paged.argtypes = [P, P, P, P, P, P, P, I, I, I, I, I, I, I, F, I, P, Z, P]
        lib.attn_workspace_size.argtypes = [I, I, I, I, I, I, I, I]
        lib.attn_workspace_size.restype = Z
        lib.attn_get_device_status.argtypes = [P]
        lib.attn_selftest_wait_timeout.argtypes = [I, P]
        lib.attn_status_string.argtypes = [I]
        lib.attn_status_string.restype = ctypes.c_char_p
        lib.attn_version.restype = I
        lib.attn_decode_paged_noalloc.argtypes = [P, P, P, P, P, P, P, I, I, I, I, I, I, I, F, I, P]
        lib.attn_decode_paged_noalloc.restype = I
        lib.attn_decode_paged_noalloc_max_bytes.restype = Z
        lib.attn_launch_count.restype = ctypes.c_ulonglong
        lib.attn_profile_start.restype = I
        lib.attn_profile_stop.argtypes = [ctypes.c_char_p, Z]
        lib.attn_profile_stop.restype = I
        LL = ctypes.c_longlong
        lib.attn_paged_plan.argtypes = [P] * 13 + [I] * 6 + [P]
        lib.attn_qk_norm_rope.argtypes = [P] * 8 + [I] * 6 + [LL, LL, F, F, I, I, P]
        lib.attn_qk_norm_rope_bwd.argtypes = [P] * 12 + [I] * 6 + [LL] * 4 + [F, F, I, I, P, Z, P]
        lib.attn_qk_norm_rope_paged.argtypes = [P] * 11 + [I] * 8 + [LL] * 3 + [F, F, I, I, P]
        lib.attn_tree_paged.argtypes = [P] * 10 + [I] * 10 + [F, I, P, Z, P]
        lib.attn_kv4_append.argtypes = [P] * 4 + [I] * 5 + [LL, LL, P]
        lib.attn_kv4_unpack.argtypes = [P] * 4 + [I] * 5 + [P]
        lib.attn_decode_kv4.argtypes = [P] * 6 + [I] * 7 + [F, I, I, P, Z, P]
        for f in (lib.attn_kv4_append, lib.attn_kv4_unpack, lib.attn_decode_kv4):
            f.restype = I
        for f in (lib.attn_paged_plan, lib.attn_qk_norm_rope, lib.attn_qk_norm_rope_bwd, lib.attn_qk_norm_rope_paged,
                  lib.attn_tree_paged):
            f.restype = I
        for f in (lib.attn_fwd, lib.attn_fwd_varlen, lib.attn_fwd_paged, lib.attn_bwd, lib.attn_decode_paged, lib.attn_get_device_status):
            f.restype = I
        _lib = lib
        return lib


def attn_status_string(status: int) -> str:
    return load_library().attn_status_string(int(status)).decode()


def attn_workspace_size(op: int, B: int = 0, Hq: int = 0, Hkv: int = 0, S: int = 0, D: int = 0, num_seqs: int = 0,
                        max_pages_per_seq: int = 0) -> int:
    return int(load_library().attn_workspace_size(op, B, Hq, Hkv, S, D, num_seqs, max_pages_per_seq))


def attn_bwd_sink_workspace_size(B: int, Hq: int, Hkv: int, S: int, D: int, num_seqs: int = 0, window: int = 0, sink: int = 0) -> int:
    """Bytes of attn_bwd's workspace for a window with sinks; packed sequences: B = 1, S = total tokens and num_seqs."""
    return int(load_library().attn_bwd_sink_workspace_size(B, Hq, Hkv, S, D, num_seqs, window, sink))


def attn_launch_count() -> int:
    """Kernel launches issued by the library in this process (monotonic)."""
    return int(load_library().attn_launch_count())


def attn_profile_start() -> None:
    """Bracket every library kernel launch with CUDA events from now on (clears old records)."""
    _check(load_library().attn_profile_start(), "attn_profile_start")


def attn_profile_stop() -> dict:
    """Stop profiling; returns {kernel name: (launches, total device ms)}."""
    buf = ctypes.create_string_buffer(1 << 14)
    n = load_library().attn_profile_stop(buf, len(buf))
    if n < 0:
        raise AttnError(-n, "attn_profile_stop")
    out = {}
    for line in buf.value.decode().splitlines():
        name, cnt, ms = line.split()
        out[name] = (int(cnt), float(ms))
    return out


def _stream_ptr(stream, device):
    import torch

    s = stream if stream is not None else torch.cuda.current_stream(device)
    return ctypes.c_void_p(s.cuda_stream)


def attn_get_device_status(stream=None) -> int:
    """Synchronise the stream and return (and clear) the device fault flags as a status code."""
    import torch

    return int(load_library().attn_get_device_status(_stream_ptr(stream, torch.cuda.current_device())))


def attn_selftest_wait_timeout(limit_ms: int = 100, stream=None) -> None:
    """Enqueue the bounded-wait self-test (a wait that nothing completes gives up after
    limit_ms and records ATTN_ERR_DEVICE_TIMEOUT); read it with attn_get_device_status()."""
    import torch

    _check(int(load_library().attn_selftest_wait_timeout(int(limit_ms), _stream_ptr(stream, torch.cuda.current_device()))),
           "attn_selftest_wait_timeout")


def _check(status: int, what: str):
    if status != 0:
        raise AttnError(status, what)


def _bf16(t, name):
    import torch

    if t.dtype != torch.bfloat16 or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous bfloat16 CUDA tensor")
    return ctypes.c_void_p(t.data_ptr())


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else None


def _on(stream, device):
    """Context of a call: what is allocated in it belongs to the stream that the call's kernels run on, and the library works on
    the current device."""
    import torch

    if stream is None:
        return torch.cuda.device(device)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(stream.cuda_stream, device=device)
    if stream.device != device:
        raise ValueError("stream is on another device than the tensors")
    return torch.cuda.stream(stream)


def _scratch(nbytes: int, device):
    """A workspace of one call's own (another stream or thread may be using the last one, and a graph keeps its own)."""
    import torch

    return torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)


def attn_fwd(q, k, v, o=None, lse=None, *, causal: bool = True, window: int = 0, scale: float | None = None,
             stream=None, sink: int = 0):
    """Forward of causal (optionally sliding-window) GQA attention, dense [B, S, H, D] layout. With a window the
    sequence's first ``sink`` keys (0 to 128) stay visible to every later query; K and V of its first 128 keys, whose tile is
    then read, must be finite."""
    if scale is None:
        scale = 1.0 / math.sqrt(q.shape[-1])
    if ops := _bound or _native_for(sink):
        return ops.fwd_sink(q, k, v, None, 0, o, lse, causal, int(window), sink or 0, scale, stream)
    import torch

    B, S, Hq, D = q.shape
    Hkv = k.shape[2]
    with _on(stream, q.device):
        if o is None:
            o = torch.empty_like(q)
        if lse is None:
            lse = torch.empty((B, Hq, S), dtype=torch.float32, device=q.device)
        rc = load_library().attn_fwd(_bf16(q, "q"), _bf16(k, "k"), _bf16(v, "v"), _bf16(o, "o"), _ptr(lse), B, Hq, Hkv,
                                     S, D, float(scale), int(causal), int(window), None, 0, _stream_ptr(stream, q.device))
    _check(rc, "attn_fwd")
    return o, lse


def attn_fwd_varlen(q, k, v, cu_seqlens, max_seqlen: int, o=None, lse=None, *, causal: bool = True, window: int = 0,
                    scale: float | None = None, stream=None, sink: int = 0):
    """Forward over packed sequences: q [T, Hq, D], k/v [T, Hkv, D], cu_seqlens int32 [n+1] on the device; ``sink`` as in
    attn_fwd, for each sequence."""
    if scale is None:
        scale = 1.0 / math.sqrt(q.shape[-1])
    if ops := _bound or _native_for(sink):
        return ops.fwd_sink(q, k, v, cu_seqlens, int(max_seqlen), o, lse, causal, int(window), sink or 0, scale, stream)
    import torch

    T, Hq, D = q.shape
    Hkv = k.shape[1]
    if cu_seqlens.dtype != torch.int32 or not cu_seqlens.is_cuda:
        raise ValueError("cu_seqlens must be an int32 CUDA tensor")
    with _on(stream, q.device):
        if o is None:
            o = torch.empty_like(q)
        if lse is None:
            lse = torch.empty((Hq, T), dtype=torch.float32, device=q.device)
        rc = load_library().attn_fwd_varlen(_bf16(q, "q"), _bf16(k, "k"), _bf16(v, "v"), _bf16(o, "o"), _ptr(lse),
                                            _ptr(cu_seqlens), cu_seqlens.numel() - 1, T, int(max_seqlen), Hq, Hkv, D,
                                            float(scale), int(causal), int(window), None, 0, _stream_ptr(stream, q.device))
    _check(rc, "attn_fwd_varlen")
    return o, lse


def attn_fwd_paged(q, k_cache, v_cache, block_table, seq_lens, cu_q, max_q_len: int, o=None, lse=None, *,
                   causal: bool = True, window: int = 0, scale: float | None = None, stream=None, sink: int = 0):
    """Chunked prefill: q [T,Hq,D] new tokens packed by cu_q, caches [pages,16,Hkv,D], block_table int32
    [R,max_pages], seq_lens int32 [R] (cached tokens including the new ones), cu_q int32 [R+1]; ``sink`` as in
    attn_fwd, for each request."""
    import torch

    T, Hq, D = q.shape
    num_pages, page_size, Hkv, _ = k_cache.shape
    scale = float(scale if scale is not None else 1.0 / math.sqrt(D))
    for t, n in ((block_table, "block_table"), (seq_lens, "seq_lens"), (cu_q, "cu_q")):
        if t.dtype != torch.int32 or not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{n} must be a contiguous int32 CUDA tensor")
    with _on(stream if o is None or lse is None else None, q.device):
        if o is None:
            o = torch.empty_like(q)
        if lse is None:
            lse = torch.empty((Hq, T), dtype=torch.float32, device=q.device)
        rc = load_library().attn_fwd_paged_sink(
            _bf16(q, "q"), _bf16(k_cache, "k_cache"), _bf16(v_cache, "v_cache"), _ptr(block_table), _ptr(seq_lens),
            _ptr(cu_q), _bf16(o, "o"), _ptr(lse), cu_q.numel() - 1, T, int(max_q_len), Hq, Hkv, D, page_size,
            block_table.shape[1], num_pages, scale, int(causal), int(window), int(sink), _stream_ptr(stream, q.device))
    _check(rc, "attn_fwd_paged")
    return o, lse


def attn_merge_lse(o_parts, lse_parts, o=None, lse=None, *, stream=None):
    """Combine results over disjoint key sets: o_parts [P,B,S,H,D] (or [P,T,H,D]) bf16, lse_parts
    [P,B,H,S] (or [P,H,T]) fp32 -> (o, lse) in the forward's layouts. o / lse may be o_parts[0] /
    lse_parts[0] (in-place running merge)."""
    import torch

    packed = o_parts.dim() == 4
    if packed:
        P, S, H, D = o_parts.shape
        B = 1
    else:
        P, B, S, H, D = o_parts.shape
    if lse_parts.dtype != torch.float32 or not lse_parts.is_cuda or not lse_parts.is_contiguous():
        raise ValueError("lse_parts must be a contiguous float32 CUDA tensor")
    if tuple(lse_parts.shape) != ((P, H, S) if packed else (P, B, H, S)):
        raise ValueError("lse_parts shape does not match o_parts")
    with _on(stream if o is None or lse is None else None, o_parts.device):
        if o is None:
            o = torch.empty(o_parts.shape[1:], dtype=torch.bfloat16, device=o_parts.device)
        if lse is None:
            lse = torch.empty(lse_parts.shape[1:], dtype=torch.float32, device=o_parts.device)
        rc = load_library().attn_merge_lse(_bf16(o_parts, "o_parts"), _ptr(lse_parts), _bf16(o, "o"), _ptr(lse), P, B,
                                           S, H, D, _stream_ptr(stream, o_parts.device))
    _check(rc, "attn_merge_lse")
    return o, lse


def attn_bwd(q, k, v, o, lse, dO, dq=None, dk=None, dv=None, *, causal: bool = True, window: int = 0,
             scale: float | None = None, cu_seqlens=None, max_seqlen: int = 0, workspace=None, stream=None, sink: int = 0):
    """Gradients (dQ, dK, dV). Dense [B,S,H,D] when cu_seqlens is None, else packed [T,H,D]; ``sink`` as in the forward."""
    if scale is None:
        scale = 1.0 / math.sqrt(q.shape[-1])
    if ops := _bound or _native_for(sink):
        return ops.bwd_sink(q, k, v, o, lse, dO, dq, dk, dv, causal, int(window), sink or 0, scale, cu_seqlens, int(max_seqlen), workspace, stream)
    import torch

    if cu_seqlens is None:
        B, S, Hq, D = q.shape
        Hkv = k.shape[2]
        nseq = 0
    else:
        B, (S, Hq, D) = 1, q.shape
        Hkv = k.shape[1]
        nseq = cu_seqlens.numel() - 1
    with _on(stream, q.device):
        dq = torch.empty_like(q) if dq is None else dq
        dk = torch.empty_like(k) if dk is None else dk
        dv = torch.empty_like(v) if dv is None else dv
        need = attn_workspace_size(ATTN_OP_BWD if cu_seqlens is None else ATTN_OP_BWD_VARLEN, B, Hq, Hkv, S, D, nseq)
        if workspace is None:
            workspace = _scratch(need, q.device)
        rc = load_library().attn_bwd(_bf16(q, "q"), _bf16(k, "k"), _bf16(v, "v"), _bf16(o, "o"), _ptr(lse),
                                     _bf16(dO, "dO"), _bf16(dq, "dQ"), _bf16(dk, "dK"), _bf16(dv, "dV"), B, Hq, Hkv, S, D,
                                     float(scale), int(causal), int(window), _ptr(cu_seqlens), nseq, int(max_seqlen),
                                     _ptr(workspace), workspace.numel() * workspace.element_size(),
                                     _stream_ptr(stream, q.device))
    _check(rc, "attn_bwd")
    return dq, dk, dv


def attn_decode_paged(q, k_cache, v_cache, block_table, seq_lens, o=None, lse=None, *, scale: float | None = None,
                      window: int = 0, workspace=None, stream=None, sink: int = 0):
    """Single-token decode: q [B,Hq,D], caches [pages,16,Hkv,D], block_table int32 [B,max_pages], seq_lens int32 [B];
    window > 0: the query sees only the last `window` keys, and the request's first `sink` ones (0 to 128)."""
    if scale is None:
        scale = 1.0 / math.sqrt(q.shape[-1])
    if ops := _bound or _native_for(sink):
        return ops.decode_paged_sink(q, k_cache, v_cache, block_table, seq_lens, o, lse, scale, int(window), sink or 0, workspace, stream)
    import torch

    B, Hq, D = q.shape
    num_pages, page_size, Hkv, _ = k_cache.shape
    for t, n in ((block_table, "block_table"), (seq_lens, "seq_lens")):
        if t.dtype != torch.int32 or not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{n} must be a contiguous int32 CUDA tensor")
    with _on(stream, q.device):
        if o is None:
            o = torch.empty_like(q)
        if lse is None:
            lse = torch.empty((B, Hq), dtype=torch.float32, device=q.device)
        need = attn_workspace_size(ATTN_OP_DECODE_PAGED, B, Hq, Hkv, 0, D)
        if workspace is None:
            workspace = _scratch(need, q.device)
        rc = load_library().attn_decode_paged(_bf16(q, "q"), _bf16(k_cache, "k_cache"), _bf16(v_cache, "v_cache"),
                                              _ptr(block_table), _ptr(seq_lens), _bf16(o, "o"), _ptr(lse), B, Hq, Hkv, D,
                                              page_size, block_table.shape[1], num_pages, float(scale), int(window),
                                              _ptr(workspace),
                                              workspace.numel() * workspace.element_size(), _stream_ptr(stream, q.device))
    _check(rc, "attn_decode_paged")
    return o, lse


def attn_decode_paged_noalloc(q, k_cache, v_cache, block_table, seq_lens, o, lse, *, scale: float | None = None,
                              window: int = 0, stream=None):
    """attn_decode_paged without a workspace: the library's built-in scratch buffer is used.

    For callers that cannot allocate device memory on their decode path, so the outputs
    ``o`` [B,Hq,D] and ``lse`` [B,Hq] must be supplied by the caller. It takes no sinks. Calls that overlap
    on the GPU share the buffer and race; see include/attn.h for the size limit.
    """
    import torch

    B, Hq, D = q.shape
    num_pages, page_size, Hkv, _ = k_cache.shape
    scale = float(scale if scale is not None else 1.0 / math.sqrt(D))
    for t, n in ((block_table, "block_table"), (seq_lens, "seq_lens")):
        if t.dtype != torch.int32 or not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{n} must be a contiguous int32 CUDA tensor")
    with torch.cuda.device(q.device):  # the library works on the current device
        rc = load_library().attn_decode_paged_noalloc(
            _bf16(q, "q"), _bf16(k_cache, "k_cache"), _bf16(v_cache, "v_cache"), _ptr(block_table), _ptr(seq_lens),
            _bf16(o, "o"), _ptr(lse), B, Hq, Hkv, D, page_size, block_table.shape[1], num_pages, scale, int(window),
            _stream_ptr(stream, q.device))
    _check(rc, "attn_decode_paged_noalloc")
    return o, lse


class PagedPlan(NamedTuple):
    """What attn_paged_plan writes (int32 tensors)."""

    seq_lens: Any     # [R] cached tokens including the new ones
    cu_q: Any         # [R + 1] first row of each request
    positions: Any    # [total_new] position of each row
    slots: Any        # [total_new] cache slot of each row, -1: none
    pages_held: Any   # [R] pages in each block-table row
    free_used: Any    # [1] pages taken of the free list
    admitted: Any     # [1] requests served


_bound = None


_unbound = False  # _native() has failed


def _native():
    """The native part of the binding (csrc/py_ops.cpp): many calls are short on the GPU, so the argument
    checks, output allocation and C call of each are one function of it. Outputs and workspaces that are not given
    belong to the stream of the call (or to the graph being captured): calls on different streams, or in
    different graphs, never share them."""
    global _bound
    if _bound is None:
        import torch  # noqa: F401  (the module uses torch's own library)

        load_library()
        from . import _build

        built_for = _build.ops_tag()
        if built_for is not None and built_for != _build.torch_tag():
            raise RuntimeError(f"attention_flash_gqa_gb300/_ops.so was built for {built_for}, not {_build.torch_tag()}: build it "
                               "again (python -m attention_flash_gqa_gb300._build or __graft_entry__.build())")
        try:
            from . import _ops as ops
        except ImportError as e:
            raise RuntimeError("attention_flash_gqa_gb300/_ops.so is missing or does not fit this torch: build it "
                               "(python -m attention_flash_gqa_gb300._build or __graft_entry__.build())") from e
        ops.load(_LIB_PATH, AttnError, PagedPlan)
        _bound = ops
    return _bound


def _native_for(sink):
    """_native(), or None where it is missing and a call without sinks goes to the C library from here."""
    global _unbound
    if sink:
        return _native()
    if not _unbound:
        try:
            return _native()
        except RuntimeError:
            _unbound = True
    return None


def attn_paged_plan(kv_lens, new_lens, free_pages, block_table, pages_held, free_used, total_new: int, *, num_pages: int,
                    page_size: int = 16, out: PagedPlan | None = None, stream=None) -> PagedPlan:
    """The plan of a serving step over a paged cache, from lengths on the device (all int32).

    kv_lens, new_lens, pages_held [R]: cached tokens, tokens to add and pages held of every request;
    free_pages [F] page ids to hand out in order, free_used [1] how many are taken already; block_table
    [R, max_pages], whose rows get the new pages in place; total_new: rows of positions and slots (a
    step of varying size may pass more than it fills: the rest gets slot -1). ``out`` gives the
    tensors to write; its seq_lens, pages_held and free_used may be kv_lens, pages_held and free_used
    themselves (a state kept in place). See include/attn.h for admission and refusals.
    """
    return (_bound or _native()).paged_plan(kv_lens, new_lens, free_pages, block_table, pages_held, free_used, total_new, num_pages,
                                          page_size, out, stream)


def attn_qk_norm_rope(q, k, q_weight, k_weight, positions, cos_sin, q_out=None, k_out=None, *, eps: float = 1e-6,
                      weight_offset: float = 0.0, interleaved: bool = False, stream=None):
    """RMS norm of every query and key head, then the rotary position encoding -> (q_out, k_out).

    q [T,Hq,D], k [T,Hkv,D] (or [B,S,H,D]) bf16, possibly slices of a fused projection; q_weight, k_weight
    [D] bf16 or fp32 (None: no weight), applied as weight_offset + w; positions int32 [T]; cos_sin fp32
    [max_pos, rot_dim], cos then sin of the rot_dim/2 angles of each position (None: no rotation).
    """
    return (_bound or _native()).norm_rope(q, k, q_weight, k_weight, positions, cos_sin, q_out, k_out, eps, weight_offset,
                                         interleaved, stream)


def attn_qk_norm_rope_bwd(dq_out, dk_out, q, k, q_weight, k_weight, positions, cos_sin, dq=None, dk=None, *,
                          eps: float = 1e-6, weight_offset: float = 0.0, interleaved: bool = False, workspace=None,
                          stream=None):
    """Gradient of attn_qk_norm_rope -> (dq, dk, dq_weight, dk_weight); the weight gradients are fp32 [D].

    dq_out, dk_out: gradients of its results (contiguous bf16); the rest as passed to the forward.
    dq / dk may be given, as slices of a fused projection's gradient too.
    """
    return (_bound or _native()).norm_rope_bwd(dq_out, dk_out, q, k, q_weight, k_weight, positions, cos_sin, dq, dk, eps,
                                             weight_offset, interleaved, workspace, stream)


def attn_qk_norm_rope_paged(q, k, v, q_weight, k_weight, positions, slots, cos_sin, k_cache, v_cache, q_out=None, *,
                            eps: float = 1e-6, weight_offset: float = 0.0, interleaved: bool = False, stream=None):
    """attn_qk_norm_rope for serving: returns q_out; k (normed and turned) and v go into the paged caches
    [pages,16,Hkv,D] in place, each token at its slot (int32 [T], of attn_paged_plan; -1: padding)."""
    return (_bound or _native()).norm_rope_paged(q, k, v, q_weight, k_weight, positions, slots, cos_sin, k_cache, v_cache, q_out, eps,
                                               weight_offset, interleaved, stream)


def attn_tree_paged(q, k_cache, v_cache, block_table, seq_lens, cu_q, tree_mask, max_q_len: int, o=None, lse=None, *,
                    positions=None, window: int = 0, scale: float | None = None, workspace=None, stream=None):
    """Attention of drafted token trees over a paged cache -> (o, lse[Hq,T]).

    q [T,Hq,D]: the drafted tokens of all requests packed by cu_q int32 [R+1], the last of their
    seq_lens int32 [R] cached tokens; tree_mask int32 [T, words]: bit d of a row (word d // 32) set where it
    sees its request's drafted token d; every row sees the context before the drafted tokens, with
    window > 0 only the keys less than `window` behind its position (positions int32 [T]). Among the drafted
    tokens the mask alone decides: for a windowed layer whose trees are deeper than the window, clear the bits of
    the ancestors `window` or more positions back. There are no sinks past the window here.
    """
    if scale is None:
        scale = 1.0 / math.sqrt(q.shape[-1])
    return (_bound or _native()).tree_paged(q, k_cache, v_cache, block_table, seq_lens, cu_q, tree_mask, max_q_len, o, lse, positions,
                                          window, scale, workspace, stream)


def attn_kv4_append(k, v, slots, kv_cache, *, page_size: int = 16, stream=None) -> None:
    """Keys and values into a paged cache in 4 bits, in place: k, v [T,Hkv,D] (or [B,S,H,D]) bf16, possibly slices of a fused
    projection, slots int32 [T] (of attn_paged_plan; -1: padding), kv_cache uint8 [pages,Hkv,18,D].

    32 dims of a token are held as n * s, n = -8 .. 7 and s a bf16 number of 5 significant bits; see include/attn.h.
    """
    (_bound or _native()).kv4_append(k, v, slots, kv_cache, page_size, stream)


def attn_kv4_unpack(kv_cache, pages, k_pages=None, v_pages=None, *, page_size: int = 16, stream=None):
    """Pages of a 4-bit cache as bf16, exactly -> (k_pages, v_pages) [n,16,Hkv,D]: what attn_fwd_paged and attn_tree_paged read, with a
    block table of 0 .. n-1. pages int32 [n] (-1: that page of the results is left as it is, in new ones as it was allocated)."""
    return (_bound or _native()).kv4_unpack(kv_cache, pages, k_pages, v_pages, page_size, stream)


def attn_decode_kv4(q, kv_cache, block_table, seq_lens, o=None, lse=None, *, scale: float | None = None, window: int = 0, sink: int = 0,
                    page_size: int = 16, workspace=None, stream=None):
    """Single-token decode over a 4-bit cache -> (o, lse[B,Hq]): q [B,Hq,D], kv_cache uint8 [pages,Hkv,18,D], block_table int32
    [B,max_pages], seq_lens int32 [B]; window > 0: only the last `window` keys are seen, and the first `sink` ones."""
    if scale is None:
        scale = 1.0 / math.sqrt(q.shape[-1])
    return (_bound or _native()).decode_kv4(q, kv_cache, block_table, seq_lens, o, lse, scale, window, sink, page_size, workspace, stream)
