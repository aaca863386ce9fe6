"""Decode-step top-K sparse attention on GB300 (sm_103a).

Thin ctypes binding over ``libtsa.so`` (C ABI in ``include/tsa.h``).  The
functions keep the library's names (``sparse_attn_decode``, ``lse_merge``,
``retopk_*``) and only marshal arguments: every step of the computation runs
in the library's CUDA kernels.  PyTorch supplies device memory and streams.

Importing this package loads the library; if it is missing it is built with
nvcc, and if that fails the import raises -- there is no fallback path.
"""
from __future__ import annotations

import ctypes as C
import math
import os
import struct
import threading
from typing import Optional

import torch

from . import build as _build

__all__ = [
    "TsaError", "lib", "KV", "kv_contiguous", "kv_paged", "decode_workspace_size",
    "sparse_attn_decode", "lse_merge", "ReTopK", "library_path", "set_stage_events",
    "set_trace", "read_trace", "kernel_launches", "sparse_attn_decode_noalloc",
    "noalloc_scratch_bytes", "RopeTable", "rope", "KV8", "kv8_append", "kv8_read",
    "attn_decode_workspace", "kv8_attn_decode", "window_attn_decode",
    "window_attn_prefill_workspace", "window_attn_prefill", "shared_attn_decode",
    "shared_attn_decode_workspace", "Pages", "pages_alloc", "pages_free", "pages_fork",
    "pages_compact", "pages_copy",
]

TSA_OK = 0
_ERRORS = {-1: "TSA_ERR_INVALID_ARG", -2: "TSA_ERR_WORKSPACE", -3: "TSA_ERR_CUDA",
           -4: "TSA_ERR_STATE", -5: "TSA_ERR_DEVICE_CHECK", -6: "TSA_ERR_TIMEOUT"}


class TsaError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"{_ERRORS.get(code, code)}: {msg}")
        self.code = code


class _KvStruct(C.Structure):
    _fields_ = [("k", C.c_void_p), ("v", C.c_void_p), ("page_table", C.c_void_p),
                ("page_size", C.c_int32), ("max_pages", C.c_int32), ("l_cap", C.c_int64)]


class _RopeSpec(C.Structure):
    _fields_ = [("theta", C.c_double), ("factor", C.c_double), ("low", C.c_double),
                ("high", C.c_double), ("amplitude", C.c_double), ("orig_len", C.c_int64),
                ("max_pos", C.c_int64), ("rot_dim", C.c_int32), ("layout", C.c_int32),
                ("scaling", C.c_int32)]


class _RopeStruct(C.Structure):
    _fields_ = [("table", C.c_void_p), ("max_pos", C.c_int64), ("rot_dim", C.c_int32),
                ("layout", C.c_int32)]


class _RopeAxes(C.Structure):
    _fields_ = [("n", C.c_int32), ("order", C.c_int32), ("rates", C.c_int32),
                ("pairs", C.c_int32 * 4)]


class _PagesStruct(C.Structure):
    _fields_ = [("table", C.c_void_p), ("refs", C.c_void_p), ("B", C.c_int32),
                ("max_pages", C.c_int32), ("n_pages", C.c_int32), ("page_size", C.c_int32)]


class _PageBuf(C.Structure):
    _fields_ = [("data", C.c_void_p), ("bytes", C.c_int64)]


class _RowsStruct(C.Structure):
    _fields_ = [("data", C.c_void_p), ("stride_t", C.c_int64), ("stride_h", C.c_int64)]


class _Kv8Struct(C.Structure):
    _fields_ = [("k", C.c_void_p), ("v", C.c_void_p), ("k_scale", C.c_void_p),
                ("v_scale", C.c_void_p), ("page_table", C.c_void_p), ("status", C.c_void_p),
                ("l_cap", C.c_int64), ("page_size", C.c_int32), ("max_pages", C.c_int32),
                ("n_pages", C.c_int32), ("block", C.c_int32), ("format", C.c_int32)]


_lock = threading.Lock()
_lib = None


def library_path() -> str:
    return _build.LIB


def lib():
    """Load libtsa.so (building it first if it is missing or stale)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            path = _build.build()
            L = C.CDLL(path)
            P, i32, i64, f32, sz = C.c_void_p, C.c_int, C.c_int64, C.c_float, C.c_size_t
            L.tsa_last_error.restype = C.c_char_p
            L.tsa_version.restype = C.c_char_p
            L.tsa_decode_workspace_size.argtypes = [i32, i32, i32, i32, i64, i32, i32, i32]
            L.tsa_decode_workspace_size.restype = sz
            L.sparse_attn_decode.argtypes = [P, P, P, i32, i32, i32, i32, i32, i32, i32, f32,
                                             P, P, P, P, P, sz, P]
            L.lse_merge.argtypes = [P, P, P, P, P, P, i32, i32, P]
            L.sparse_attn_decode_noalloc.argtypes = [P, P, P, i32, i32, i32, i32, i32, i32,
                                                     i32, f32, P, P, P, P, P]
            L.tsa_noalloc_scratch_bytes.restype = sz
            L.retopk_state_size.argtypes = [i32, i32, i32, i32]
            L.retopk_state_size.restype = sz
            L.retopk_create.argtypes = [C.POINTER(P), i32, i32, i32, i32, i32, i32, i32, f32,
                                        i32, i64, P, sz]
            L.retopk_init.argtypes = [P, P, P, P, P]
            L.retopk_workspace_size.argtypes = [P]
            L.retopk_workspace_size.restype = sz
            L.retopk_step.argtypes = [P, P, P, i64, f32, P, P, P, P, P, P, P, sz, P]
            L.retopk_batched_workspace_size.argtypes = [P, i32]
            L.retopk_batched_workspace_size.restype = sz
            L.retopk_step_batched.argtypes = [P, i32, P, P, P, f32, P, P, P, P, P, P, P, sz, P]
            L.retopk_get_counters.argtypes = [P, C.POINTER(i64), C.POINTER(C.c_int32)]
            L.retopk_set_counters.argtypes = [P, i64, C.c_int32]
            L.retopk_destroy.argtypes = [P]
            L.tsa_set_stage_events.argtypes = [C.POINTER(P), i32]
            L.tsa_set_trace.argtypes = [P, sz]
            L.tsa_kernel_launches.restype = C.c_ulonglong
            L.tsa_workspace_status.argtypes = [P, i32, P]
            L.sparse_attn_decode_shard.argtypes = [P, P, i64, i64, i64, i32, i32, i32, i32, i32,
                                                   i32, f32, P, P, P, P, P, sz, P]
            L.tsa_attend_set_workspace_size.argtypes = [i32, i32, i32]
            L.tsa_attend_set_workspace_size.restype = sz
            L.attend_set.argtypes = [P, P, i32, i32, i32, i32, P, P, i32, f32, P, P, P, sz, P]
            L.retopk_prefill_workspace_size.argtypes = [i32, i32, i32, i32, i64, i32]
            L.retopk_prefill_workspace_size.restype = sz
            L.retopk_prefill_supports.argtypes = [P, P, i64, i32, i32, i32, i32, i32, f32, P, P,
                                                  P, sz, P]
            L.tsa_inject_scan_stall.argtypes = [C.c_longlong]
            L.tsa_quantize_keys.argtypes = [P, P, P, i32, i32, i32, i64, i32, P]
            L.tsa_decode_q8_workspace_size.argtypes = [i32, i32, i32, i32, i64, i32, i32, i32]
            L.tsa_decode_q8_workspace_size.restype = sz
            L.sparse_attn_decode_q8.argtypes = [P, P, P, i32, P, i32, i32, i32, i32, i32, i32,
                                                i32, f32, P, P, P, P, P, sz, P]
            L.tsa_rope_table_size.argtypes = [i32, i64]
            L.tsa_rope_table_size.restype = sz
            L.tsa_rope_table.argtypes = [P, P, sz, P, P]
            L.rope_apply.argtypes = [P, P, i32, P, P, i32, i64, i32, P, P, i32, P]
            L.kv8_append.argtypes = [P, P, P, P, i64, i32, P, i32, i32, i32, P, P, P]
            L.kv8_read.argtypes = [P, P, P, P, i64, i32, P, i32, i32, i32, P]
            L.tsa_rope_table_axes.argtypes = [P, P, P, sz, P, P]
            L.rope_apply_axes.argtypes = [P, P, i32, P, P, i32, i64, i32, P, i64, P, P, i32, P]
            L.kv8_append_axes.argtypes = [P, P, P, P, i64, i32, P, i32, i32, i32, P, P, P, i64, P]
            L.tsa_pages_workspace_size.argtypes = [i32, i32, i32]
            L.tsa_pages_workspace_size.restype = sz
            for fn in (L.pages_alloc, L.pages_free):
                fn.argtypes = [P, P, P, P, sz, P]
            L.pages_fork.argtypes = [P, P, P, P, i32, P, P, P, sz, P]
            L.pages_compact.argtypes = [P, P, P, P, P, sz, P]
            L.pages_copy.argtypes = [P, i32, i32, P, P, P, i32, P, P]
            L.tsa_shared_attn_workspace_size.argtypes = [i32, i32, i32, i32, i32]
            L.tsa_shared_attn_workspace_size.restype = sz
            for fn in (L.shared_attn_decode, L.kv8_shared_attn_decode):
                fn.argtypes = [P, P, P, i32, P, P, i32, i32, i32, i32, f32, P, i32, P, P, sz, P]
            L.tsa_attn_decode_workspace_size.argtypes = [i32, i32, i32, i32]
            L.tsa_attn_decode_workspace_size.restype = sz
            for fn in (L.kv8_attn_decode, L.window_attn_decode):
                fn.argtypes = [P, P, P, i32, i32, i32, i32, i64, i64, f32, P, P, P, sz, P]
            L.window_attn_prefill_workspace_size.argtypes = [i32, i32, i32, i32, i32, i64, i64,
                                                             i64]
            L.window_attn_prefill_workspace_size.restype = sz
            L.window_attn_prefill.argtypes = [P, P, P, i64, i32, P, i32, i32, i32, i32, i64, i64,
                                              f32, P, P, P, sz, P]
            _lib = L
    return _lib


def _check(rc: int) -> None:
    if rc != TSA_OK:
        raise TsaError(rc, lib().tsa_last_error().decode())


def _p(t: Optional[torch.Tensor]):
    return None if t is None else C.c_void_p(t.data_ptr())


def _stream(stream) -> C.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return C.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _want(t: torch.Tensor, dtype, name: str):
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def kernel_launches() -> int:
    """Kernels the library has launched in this process so far."""
    return int(lib().tsa_kernel_launches())


def set_stage_events(events) -> None:
    """Per-stage timing: a list of 4 torch.cuda.Event(enable_timing=True) (or None).

    Later calls on this thread record them before the first launch and after
    the scan, the selection and the attention kernel, on the call's stream."""
    if not events:
        _check(lib().tsa_set_stage_events(None, 0))
        return
    arr = (C.c_void_p * len(events))(*[C.c_void_p(e.cuda_event) for e in events])
    _check(lib().tsa_set_stage_events(arr, len(events)))


def set_trace(buf: Optional[torch.Tensor]) -> None:
    """Per-CTA kernel timeline into a uint8 device tensor (see include/tsa.h);
    the first 4 bytes count records and must be zeroed by the caller."""
    if buf is None:
        _check(lib().tsa_set_trace(None, 0))
    else:
        _check(lib().tsa_set_trace(_p(buf), buf.numel()))


def read_trace(buf: torch.Tensor):
    """Decode a trace buffer into a list of dicts (kernel, cta, sm, t0..t3)."""
    import numpy as np
    raw = buf.cpu().numpy()
    n = int(raw[:4].view(np.uint32)[0])
    cap = (raw.size - 64) // 48
    rec = raw[64:64 + 48 * min(n, cap)].view(np.uint32).reshape(-1, 12)
    out = []
    for r in rec:
        t = r[4:12].view(np.uint64)
        out.append({"kernel": int(r[0]), "cta": int(r[1]), "sm": int(r[2]),
                    "info": int(r[3]), "t": [int(x) for x in t]})
    return out


def _page_bufs(*pools: torch.Tensor) -> bytes:
    """The tsa_page_buf of every pool of pages, [n_pages][...] (as their bytes)."""
    return b"".join(struct.pack("=qq", p.data_ptr(), p.nbytes // max(1, p.shape[0]))
                    for p in pools)


class KV:
    """A layer's KV cache as the library sees it (keeps the tensors alive)."""

    def __init__(self, k, v, page_table=None, page_size=0):
        _want(k, torch.bfloat16, "k")
        _want(v, torch.bfloat16, "v")
        if v.shape != k.shape:
            raise ValueError(f"v must have k's shape {tuple(k.shape)}, got {tuple(v.shape)}")
        for t, name in ((v, "v"), (page_table, "page_table")):
            if t is not None and t.device != k.device:
                raise ValueError(f"{name} is on {t.device}, k on {k.device}")
        self.k, self.v, self.page_table = k, v, page_table
        self._bufs = _page_bufs(k, v)
        if page_table is None:
            if k.dim() != 4:
                raise ValueError("contiguous k must be [B][Hkv][l_cap][d]")
            self.B, self.Hkv, self.l_cap, self.d = k.shape
            self.struct = _KvStruct(k.data_ptr(), v.data_ptr(), None, 0, 0, self.l_cap)
        else:
            _want(page_table, torch.int32, "page_table")
            if k.dim() != 4:
                raise ValueError("paged k must be [pages][Hkv][page_size][d]")
            _, self.Hkv, ps, self.d = k.shape
            self.B, max_pages = page_table.shape
            self.l_cap = max_pages * ps
            self.struct = _KvStruct(k.data_ptr(), v.data_ptr(), page_table.data_ptr(), ps,
                                    max_pages, self.l_cap)


def kv_contiguous(k: torch.Tensor, v: torch.Tensor) -> KV:
    return KV(k, v)


def kv_paged(k_pages: torch.Tensor, v_pages: torch.Tensor, page_table: torch.Tensor) -> KV:
    return KV(k_pages, v_pages, page_table)


def decode_workspace_size(B, Hq, Hkv, d, l_cap, K, n_init, n_recent) -> int:
    return int(lib().tsa_decode_workspace_size(B, Hq, Hkv, d, l_cap, K, n_init, n_recent))


def sparse_attn_decode(q: torch.Tensor, kv: KV, lens: torch.Tensor, K: int, n_init: int,
                       n_recent: int, scale: Optional[float] = None,
                       out: Optional[torch.Tensor] = None,
                       lse_out: Optional[torch.Tensor] = None,
                       topk_idx: Optional[torch.Tensor] = None,
                       topk_score: Optional[torch.Tensor] = None,
                       workspace: Optional[torch.Tensor] = None, stream=None):
    """One decode step over every sequence and query head (see include/tsa.h).

    q: bf16 [B][Hq][d] on the device; lens: int32 [B] on the device.
    workspace: uint8, zero-filled before its first use and then reused as
    is (each call leaves it ready for the next); None allocates a fresh one.
    Returns (out, lse_out, topk_idx, topk_score) (the optional ones may be None).
    """
    _want(q, torch.bfloat16, "q")
    _want(lens, torch.int32, "lens")
    B, Hq, d = q.shape
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        out = torch.empty((B, Hq, d), dtype=torch.float32, device=q.device)
    if workspace is None:
        nb = decode_workspace_size(B, Hq, kv.Hkv, d, kv.l_cap, K, n_init, n_recent)
        workspace = torch.zeros(max(nb, 256), dtype=torch.uint8, device=q.device)
    _check(lib().sparse_attn_decode(
        _p(q), C.byref(kv.struct), _p(lens), B, Hq, kv.Hkv, d, K, n_init, n_recent,
        float(scale), _p(out), _p(lse_out), _p(topk_idx), _p(topk_score), _p(workspace),
        workspace.numel() * workspace.element_size(), _stream(stream)))
    return out, lse_out, topk_idx, topk_score


class _Kq8Struct(C.Structure):
    _fields_ = [("codes", C.c_void_p), ("scale", C.c_void_p), ("err", C.c_void_p)]


class KeyCodes:
    """The int8 copy of a cache's keys (see tsa_kq8 in include/tsa.h): codes
    with the row geometry of kv.k (one byte per element, offset binary),
    per-(sequence, KV head, channel) scales and error bounds."""

    def __init__(self, kv: "KV", B: Optional[int] = None):
        dev = kv.k.device
        self.B = kv.B if B is None else B
        self.codes = torch.empty(kv.k.shape, dtype=torch.uint8, device=dev)
        self.scale = torch.zeros((self.B, kv.Hkv, kv.d), dtype=torch.float32, device=dev)
        self.err = torch.zeros((self.B, kv.Hkv, kv.d), dtype=torch.float32, device=dev)
        self.struct = _Kq8Struct(self.codes.data_ptr(), self.scale.data_ptr(),
                                 self.err.data_ptr())


def quantize_keys(kv: "KV", codes: KeyCodes, lens: torch.Tensor, fit: bool = True,
                  n_tail: int = 0, stream=None) -> KeyCodes:
    """Fit scales and code rows [0, lens[b]) (fit), or code the last n_tail
    rows of each sequence with the stored scales."""
    _want(lens, torch.int32, "lens")
    _check(lib().tsa_quantize_keys(C.byref(kv.struct), C.byref(codes.struct), _p(lens),
                                   codes.B, kv.Hkv, kv.d, int(n_tail), 1 if fit else 0,
                                   _stream(stream)))
    return codes


def decode_q8_workspace_size(B, Hq, Hkv, d, l_cap, K, n_init, n_recent) -> int:
    return int(lib().tsa_decode_q8_workspace_size(B, Hq, Hkv, d, l_cap, K, n_init, n_recent))


def sparse_attn_decode_q8(q: torch.Tensor, kv: KV, codes: KeyCodes, lens: torch.Tensor, K: int,
                          n_init: int, n_recent: int, n_new: int = 0,
                          scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                          lse_out: Optional[torch.Tensor] = None,
                          topk_idx: Optional[torch.Tensor] = None,
                          topk_score: Optional[torch.Tensor] = None,
                          workspace: Optional[torch.Tensor] = None, stream=None):
    """sparse_attn_decode through the key codes (same results; the last n_new
    rows of each sequence are coded first).  The workspace is a q8 one."""
    _want(q, torch.bfloat16, "q")
    _want(lens, torch.int32, "lens")
    B, Hq, d = q.shape
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        out = torch.empty((B, Hq, d), dtype=torch.float32, device=q.device)
    if workspace is None:
        nb = decode_q8_workspace_size(B, Hq, kv.Hkv, d, kv.l_cap, K, n_init, n_recent)
        workspace = torch.zeros(max(nb, 256), dtype=torch.uint8, device=q.device)
    _check(lib().sparse_attn_decode_q8(
        _p(q), C.byref(kv.struct), C.byref(codes.struct), int(n_new), _p(lens), B, Hq, kv.Hkv,
        d, K, n_init, n_recent, float(scale), _p(out), _p(lse_out), _p(topk_idx),
        _p(topk_score), _p(workspace), workspace.numel() * workspace.element_size(),
        _stream(stream)))
    return out, lse_out, topk_idx, topk_score


def sparse_attn_decode_noalloc(q: torch.Tensor, kv: KV, lens: torch.Tensor, K: int,
                               n_init: int, n_recent: int, scale: Optional[float] = None,
                               out: Optional[torch.Tensor] = None,
                               lse_out: Optional[torch.Tensor] = None,
                               topk_idx: Optional[torch.Tensor] = None,
                               topk_score: Optional[torch.Tensor] = None, stream=None):
    """sparse_attn_decode with the library's own fixed scratch array instead
    of a workspace (for callers that cannot allocate while decoding; limits
    and concurrency rules in include/tsa.h).  The output buffers are the
    caller's: pass them to allocate nothing here either."""
    _want(q, torch.bfloat16, "q")
    _want(lens, torch.int32, "lens")
    B, Hq, d = q.shape
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        out = torch.empty((B, Hq, d), dtype=torch.float32, device=q.device)
    _check(lib().sparse_attn_decode_noalloc(
        _p(q), C.byref(kv.struct), _p(lens), B, Hq, kv.Hkv, d, K, n_init, n_recent,
        float(scale), _p(out), _p(lse_out), _p(topk_idx), _p(topk_score), _stream(stream)))
    return out, lse_out, topk_idx, topk_score


def noalloc_scratch_bytes() -> int:
    return int(lib().tsa_noalloc_scratch_bytes())


def decode_shard(q: torch.Tensor, kv: "KV", shard_len: int, pos_offset: int, global_len: int,
                 K: int, n_init: int, n_recent: int, scale=None, out=None, lse_out=None,
                 topk_idx=None, topk_score=None, workspace=None, stream=None):
    """One shard [pos_offset, pos_offset + shard_len) of a sequence of
    global_len positions (q bf16 [Hq][128]): local top-K (local row indices)
    and attention over the shard's window rows and that top-K."""
    _want(q, torch.bfloat16, "q")
    Hq, d = q.shape
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        out = torch.empty((Hq, d), dtype=torch.float32, device=q.device)
    if workspace is None:
        n = decode_workspace_size(1, Hq, kv.Hkv, d, kv.l_cap, K, n_init, n_recent)
        workspace = torch.zeros(n, dtype=torch.uint8, device=q.device)
    _check(lib().sparse_attn_decode_shard(_p(q), C.byref(kv.struct), int(shard_len),
                                          int(pos_offset), int(global_len), Hq, kv.Hkv, d, K,
                                          n_init, n_recent, float(scale), _p(out), _p(lse_out),
                                          _p(topk_idx), _p(topk_score), _p(workspace),
                                          workspace.numel(), _stream(stream)))
    return out


def attend_set(q: torch.Tensor, kv: "KV", positions: torch.Tensor, counts: torch.Tensor,
               scale=None, out=None, lse_out=None, workspace=None, stream=None):
    """Attention over given rows: q bf16 [B][Hq][128], positions int32
    [B][Hq][M], counts int32 [B][Hq]; returns out fp32 [B][Hq][128]."""
    _want(q, torch.bfloat16, "q")
    _want(positions, torch.int32, "positions")
    _want(counts, torch.int32, "counts")
    B, Hq, d = q.shape
    M = positions.shape[-1]
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        out = torch.empty((B, Hq, d), dtype=torch.float32, device=q.device)
    if workspace is None:
        n = int(lib().tsa_attend_set_workspace_size(B, Hq, M))
        workspace = torch.zeros(n, dtype=torch.uint8, device=q.device)
    _check(lib().attend_set(_p(q), C.byref(kv.struct), B, Hq, kv.Hkv, d, _p(positions),
                            _p(counts), M, float(scale), _p(out), _p(lse_out), _p(workspace),
                            workspace.numel(), _stream(stream)))
    return out


def prefill_workspace_size(C, Hq, Hkv, d, l_cap, K) -> int:
    return int(lib().retopk_prefill_workspace_size(C, Hq, Hkv, d, l_cap, K))


def prefill_supports(q_prefill: torch.Tensor, kv: "KV", L0: int, K: int, scale=None,
                     supports=None, counts=None, workspace=None, stream=None):
    """Exact causal top-K of the last C prefill queries (q_prefill bf16
    [C][Hq][128], query c at position L0 - C + c) over their prefixes, in one
    call: returns (supports int32 [C][Hq][K] padded with -1, counts int32
    [C][Hq])."""
    _want(q_prefill, torch.bfloat16, "q_prefill")
    Cn, Hq, d = q_prefill.shape
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    dev = q_prefill.device
    if supports is None:
        supports = torch.empty((Cn, Hq, K), dtype=torch.int32, device=dev)
    if counts is None:
        counts = torch.empty((Cn, Hq), dtype=torch.int32, device=dev)
    if workspace is None:
        n = prefill_workspace_size(Cn, Hq, kv.Hkv, d, kv.l_cap, K)
        workspace = torch.zeros(n, dtype=torch.uint8, device=dev)
    _check(lib().retopk_prefill_supports(_p(q_prefill), C.byref(kv.struct), int(L0), Cn, Hq,
                                         kv.Hkv, d, K, float(scale), _p(supports), _p(counts),
                                         _p(workspace), workspace.numel(), _stream(stream)))
    return supports, counts


def workspace_status(workspace: torch.Tensor, clear: bool = True, stream=None) -> int:
    """Device-side status of a decode or ReTopK workspace (synchronises the
    stream): 0, TSA_ERR_TIMEOUT (-6) or TSA_ERR_DEVICE_CHECK (-5)."""
    return int(lib().tsa_workspace_status(_p(workspace), 1 if clear else 0, _stream(stream)))


def inject_scan_stall(wait_limit_ns: int) -> None:
    """Fault injection for tests: the next call's key scan gives up a wait
    after wait_limit_ns (its first CTA withholds a tile copy)."""
    _check(lib().tsa_inject_scan_stall(int(wait_limit_ns)))


def lse_merge(o_a, lse_a, o_b, lse_b, o_out=None, lse_out=None, stream=None):
    """Eq. 4-5 merge of two (o, lse) partials: o fp32 [rows][d], lse fp32 [rows]."""
    rows, d = o_a.shape
    if o_out is None:
        o_out = torch.empty_like(o_a)
    if lse_out is None:
        lse_out = torch.empty_like(lse_a)
    for t, n in ((o_a, "o_a"), (o_b, "o_b"), (o_out, "o_out"), (lse_a, "lse_a"),
                 (lse_b, "lse_b"), (lse_out, "lse_out")):
        _want(t, torch.float32, n)
    _check(lib().lse_merge(_p(o_a), _p(lse_a), _p(o_b), _p(lse_b), _p(o_out), _p(lse_out),
                           rows, d, _stream(stream)))
    return o_out, lse_out


class ReTopK:
    """ReTopK per-layer state (query-support FIFO per head) on the device."""

    def __init__(self, Hq, Hkv, d, K, C_, R, W, tau, T_r, max_len, device="cuda"):
        n = int(lib().retopk_state_size(Hq, d, K, C_))
        if n == 0:
            raise TsaError(-1, "invalid ReTopK sizes")
        self.state = torch.zeros(n, dtype=torch.uint8, device=device)
        self.handle = C.c_void_p()
        _check(lib().retopk_create(C.byref(self.handle), Hq, Hkv, d, K, C_, R, W, float(tau),
                                   T_r, max_len, _p(self.state), n))
        self.Hq, self.Hkv, self.d, self.K, self.C, self.R, self.W = Hq, Hkv, d, K, C_, R, W
        self.cand_cap = R * K + W
        self.workspace = torch.zeros(int(lib().retopk_workspace_size(self.handle)),
                                     dtype=torch.uint8, device=device)

    def __del__(self):
        try:
            if self.handle:
                lib().retopk_destroy(self.handle)
                self.handle = C.c_void_p()
        except Exception:
            pass

    def init(self, prefill_q, prefill_supports, prefill_counts, stream=None):
        _want(prefill_q, torch.bfloat16, "prefill_q")
        _want(prefill_supports, torch.int32, "prefill_supports")
        _want(prefill_counts, torch.int32, "prefill_counts")
        _check(lib().retopk_init(self.handle, _p(prefill_q), _p(prefill_supports),
                                 _p(prefill_counts), _stream(stream)))

    def step(self, q, kv: KV, length: int, scale=None, out=None, support_out=None,
             path_out=None, mcand_out=None, cand_out=None, lse_out=None, stream=None):
        _want(q, torch.bfloat16, "q")
        if scale is None:
            scale = 1.0 / math.sqrt(self.d)
        if out is None:
            out = torch.empty((self.Hq, self.d), dtype=torch.float32, device=q.device)
        _check(lib().retopk_step(self.handle, _p(q), C.byref(kv.struct), int(length),
                                 float(scale), _p(out), _p(support_out), _p(path_out),
                                 _p(mcand_out), _p(cand_out), _p(lse_out), _p(self.workspace),
                                 self.workspace.numel(), _stream(stream)))
        return out

    @staticmethod
    def batched_workspace_size(proto: "ReTopK", n_max: int) -> int:
        return int(lib().retopk_batched_workspace_size(proto.handle, n_max))

    @staticmethod
    def step_batched(handles, q, kv: KV, lens, scale=None, out=None, support_out=None,
                     path_out=None, mcand_out=None, cand_out=None, lse_out=None,
                     workspace=None, stream=None):
        """One step of len(handles) sequences, each with its own state: q bf16
        [n][Hq][128], kv with the n sequences in call order, lens (host ints)."""
        _want(q, torch.bfloat16, "q")
        n = len(handles)
        Hq, d = handles[0].Hq, handles[0].d
        if scale is None:
            scale = 1.0 / math.sqrt(d)
        if out is None:
            out = torch.empty((n, Hq, d), dtype=torch.float32, device=q.device)
        if workspace is None:
            workspace = torch.zeros(ReTopK.batched_workspace_size(handles[0], n),
                                    dtype=torch.uint8, device=q.device)
        hs = (C.c_void_p * n)(*[h.handle.value for h in handles])
        ls = (C.c_int64 * n)(*[int(x) for x in lens])
        _check(lib().retopk_step_batched(hs, n, _p(q), C.byref(kv.struct), ls, float(scale),
                                         _p(out), _p(support_out), _p(path_out), _p(mcand_out),
                                         _p(cand_out), _p(lse_out), _p(workspace),
                                         workspace.numel(), _stream(stream)))
        return out

    def counters(self):
        t, h = C.c_int64(), C.c_int32()
        _check(lib().retopk_get_counters(self.handle, C.byref(t), C.byref(h)))
        return t.value, h.value

    def set_counters(self, t: int, fifo_head: int) -> None:
        _check(lib().retopk_set_counters(self.handle, t, fifo_head))


# --------------------------------------------- cache-side operators
_ROPE_SCALING = {"none": 0, "linear": 1, "ntk": 2, "by_parts": 3, "yarn": 4}
_ROPE_LAYOUT = {"half": 0, "interleaved": 1}
_ROPE_ORDER = {"blocks": 0, "turns": 1}
_ROPE_RATES = {"joint": 0, "own": 1}
_KV8_FORMAT = {"int8": 0, "e4m3": 1}


def _gpu(*named) -> torch.device:
    """The one CUDA device that the given (tensor, name) pairs live on."""
    dev = None
    for t, name in named:
        if t is None:
            continue
        d = t.device
        if dev is None:
            if d.type != "cuda":
                raise ValueError(f"{name} must be a CUDA tensor")
            dev = d
        elif d != dev:
            raise ValueError(f"{name} is on {d}, not on {dev}: it must be a CUDA tensor there")
    return dev


# The current device and the raw handle of its current stream: the public
# calls (torch.cuda.current_device, current_stream) take several times as long,
# which a decode step's call would notice.
_device_now = getattr(torch._C, "_cuda_getDevice", None)
_stream_now = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _run_on(dev: torch.device, stream, fn, *args) -> None:
    """fn(*args, stream) with dev current; stream None: dev's current one."""
    i = dev.index
    if stream is None:
        handle = _stream_now(i)
    else:
        handle = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    if i == _device_now():
        rc = fn(*args, handle)
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, handle)
    if rc:
        _check(rc)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _new(stream, dev: torch.device, shape, dtype, zero: bool = False) -> torch.Tensor:
    """A tensor made on the stream that the call runs on."""
    make = torch.zeros if zero else torch.empty
    if stream is None:
        return make(shape, dtype=dtype, device=dev)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(getattr(stream, "cuda_stream", stream)), device=dev)
    with torch.cuda.stream(stream):
        return make(shape, dtype=dtype, device=dev)


_pack_rows = struct.Struct("=qqq").pack  # tsa_rows


def _rows(t: torch.Tensor, name: str) -> bytes:
    """The tsa_rows of a bf16 [tokens][heads][128] tensor (as its bytes: a
    quarter of the time of a ctypes structure)."""
    if t.dtype != torch.bfloat16:
        raise TypeError(f"{name} must be {torch.bfloat16}, got {t.dtype}")
    st = t.stride()
    if len(st) != 3 or st[2] != 1:
        raise ValueError(f"{name} must be [tokens][heads][128] with contiguous rows")
    return _pack_rows(t.data_ptr(), st[0], st[1])


def _count(n, what: str) -> int:
    """A number of tokens as the library's 32 bits hold it (ctypes cuts silently)."""
    n = int(n)
    if not 0 <= n < 1 << 31:
        raise ValueError(f"{what} = {n}: must be in [0, 2^31)")
    return n


def _offsets(cu, T: int, max_n, B: int, what: str) -> int:
    """The most tokens of a sequence (max_n, or T / B without offsets)."""
    if cu is None:
        if B and T % B:
            raise ValueError(f"{T} tokens do not divide over {B} sequences: pass offsets")
        if max_n is not None and max_n * B != T:
            raise ValueError(f"{what} = {max_n}: {T} tokens of {B} sequences without offsets")
        return T // B if B else 0
    _want(cu, torch.int32, "offsets")
    if cu.shape != (B + 1,):
        raise ValueError(f"offsets must be int32 [{B + 1}], got {tuple(cu.shape)}")
    if max_n is None:
        raise ValueError(f"{what} is needed with offsets")
    return _count(max_n, what)


class RopeTable:
    """The angles of a rotary embedding on the device (tsa_rope_table).

    layout: "half" (pairs i, i + rot_dim/2) or "interleaved" (2i, 2i + 1);
    scaling: "none", "linear", "ntk", "by_parts" or "yarn" (see include/tsa.h)
    with `factor` and `orig_len`; low, high and amplitude default to the kind's.

    sections: pairs of every axis (two to four numbers that add up to rot_dim / 2, or
    one) where tokens have positions on several axes; order: "blocks" (axis after
    axis) or "turns" (dealt in turn); rates: "joint" (of the whole table) or "own" (of
    each axis by itself).  See tsa_rope_axes in include/tsa.h.
    """

    def __init__(self, rot_dim: int, max_pos: int, theta: float = 10000.0, layout: str = "half",
                 scaling: Optional[str] = None, factor: float = 1.0, orig_len: int = 0,
                 low: float = 0.0, high: float = 0.0, amplitude: float = 0.0, device="cuda",
                 stream=None, sections=None, order: str = "blocks", rates: str = "joint"):
        if layout not in _ROPE_LAYOUT:
            raise ValueError(f"layout {layout!r}: one of {sorted(_ROPE_LAYOUT)}")
        if (scaling or "none") not in _ROPE_SCALING:
            raise ValueError(f"scaling {scaling!r}: one of {sorted(_ROPE_SCALING)}")
        for what, val, known in (("order", order, _ROPE_ORDER), ("rates", rates, _ROPE_RATES)):
            if val not in known:
                raise ValueError(f"{what} {val!r}: one of {sorted(known)}")
        self.sections = None if sections is None else tuple(int(x) for x in sections)
        self._axes = None
        if self.sections is not None:
            if not 1 <= len(self.sections) <= 4:
                raise ValueError(f"sections {self.sections}: one to four axes")
            pairs = (C.c_int32 * 4)(*[_count(x, "sections") for x in self.sections])
            self._axes = C.byref(_RopeAxes(len(self.sections), _ROPE_ORDER[order],
                                           _ROPE_RATES[rates], pairs))
        n = int(lib().tsa_rope_table_size(int(rot_dim), int(max_pos)))
        if n == 0:
            raise TsaError(-1, f"invalid rotation sizes (rot_dim {rot_dim}, max_pos {max_pos})")
        spec = _RopeSpec(theta, factor, low, high, amplitude, int(orig_len), int(max_pos),
                         int(rot_dim), _ROPE_LAYOUT[layout], _ROPE_SCALING[scaling or "none"])
        self.rot_dim, self.max_pos, self.layout = int(rot_dim), int(max_pos), layout
        self.struct = _RopeStruct()
        self._ref = C.byref(self.struct)
        dev = torch.device(device)
        if dev.type == "cuda" and dev.index is None:
            dev = torch.device("cuda", torch.cuda.current_device())
        self.table = _new(stream, dev, (n,), torch.uint8)
        self.device = self.table.device
        if self._axes is None:
            _run_on(_gpu((self.table, "table")), stream, lib().tsa_rope_table, C.byref(spec),
                    _ptr(self.table), n, self._ref)
        else:
            _run_on(_gpu((self.table, "table")), stream, lib().tsa_rope_table_axes, C.byref(spec),
                    self._axes, _ptr(self.table), n, self._ref)


def _axis_positions(positions: torch.Tensor, table: RopeTable, T: int) -> int:
    """Whether positions are [axes][T] (then their stride), or [T] (then -1)."""
    if positions.dim() == 1:
        _want(positions, torch.int32, "positions")
        if positions.shape != (T,):
            raise ValueError(f"positions must be int32 [{T}], got {tuple(positions.shape)}")
        return -1
    if positions.dtype != torch.int32:
        raise TypeError(f"positions must be {torch.int32}, got {positions.dtype}")
    if table is None or table.sections is None:
        raise ValueError("positions of several axes need a RopeTable with sections")
    A = len(table.sections)
    if positions.shape != (A, T):
        raise ValueError(f"positions must be int32 [{A}][{T}] (or [{T}]), got "
                         f"{tuple(positions.shape)}")
    if T > 1 and positions.stride(1) != 1:
        raise ValueError("positions must have contiguous rows")
    return positions.stride(0)


def rope(q: torch.Tensor, positions: torch.Tensor, table: RopeTable,
         k: Optional[torch.Tensor] = None, q_out: Optional[torch.Tensor] = None,
         k_out: Optional[torch.Tensor] = None, inverse: bool = False, stream=None):
    """Rotates q bf16 [T][Hq][128] (and k [T][Hkv][128]) by positions int32 [T], or
    [axes][T] with a table of several axes.

    Rows may be strided (a slice of a fused projection); q_out=q rotates in
    place.  Returns (q_out, k_out)."""
    dev = q.device
    if positions.device != dev or table.device != dev or not q.is_cuda or \
            k is not None and k.device != dev or q_out is not None or k_out is not None:
        _gpu((q, "q"), (positions, "positions"), (k, "k"), (q_out, "q_out"), (k_out, "k_out"),
             (table.table, "table"))
    T, Hq, d = q.shape
    stride = _axis_positions(positions, table, T)
    if q_out is None:
        q_out = _new(stream, dev, (T, Hq, d), torch.bfloat16)
    elif q_out.shape != q.shape:
        raise ValueError("q_out must have q's shape")
    Hkv, ks, kos = 0, None, None
    if k is not None:
        if k.shape[0] != T or k.shape[2] != d or k_out is not None and k_out.shape != k.shape:
            raise ValueError("k and k_out must be [tokens][heads][128] with q's tokens")
        if k_out is None:
            k_out = _new(stream, dev, k.shape, torch.bfloat16)
        Hkv, ks, kos = k.shape[1], _rows(k, "k"), _rows(k_out, "k_out")
    elif k_out is not None:
        raise ValueError("k_out without k")
    if stride < 0:
        _run_on(dev, stream, lib().rope_apply, _rows(q, "q"), _rows(q_out, "q_out"),
                Hq, ks, kos, Hkv, T, d, _ptr(positions), table._ref, 1 if inverse else 0)
    else:
        _run_on(dev, stream, lib().rope_apply_axes, _rows(q, "q"), _rows(q_out, "q_out"),
                Hq, ks, kos, Hkv, T, d, _ptr(positions), stride, table._ref, table._axes,
                1 if inverse else 0)
    return q_out, k_out


class KV8:
    """An 8-bit KV cache as the library sees it (tsa_kv8 in include/tsa.h).

    k, v: uint8 codes [B][Hkv][l_cap][128], or [pages][Hkv][page_size][128]
    with page_table int32 [B][max_pages]; k_scale, v_scale: fp32 with one
    entry per block of rows, [...][Hkv][rows / block].  status: optional int32
    word (256-byte aligned) for workspace_status."""

    def __init__(self, k, v, k_scale, v_scale, fmt: str = "int8", page_table=None, status=None):
        if fmt not in _KV8_FORMAT:
            raise ValueError(f"fmt {fmt!r}: one of {sorted(_KV8_FORMAT)}")
        for t, name in ((k, "k"), (v, "v")):
            _want(t, torch.uint8, name)
        for t, name in ((k_scale, "k_scale"), (v_scale, "v_scale")):
            _want(t, torch.float32, name)
        if k.dim() != 4 or k.shape != v.shape:
            raise ValueError("k and v must have one shape [B or pages][Hkv][rows][128]")
        n, self.Hkv, rows, self.d = k.shape
        if k_scale.shape != v_scale.shape or k_scale.dim() != 3 or \
                k_scale.shape[:2] != k.shape[:2] or not k_scale.shape[2] or \
                rows % k_scale.shape[2]:
            raise ValueError("scales must be [B or pages][Hkv][rows / block]")
        self.device = _gpu((k, "k"), (v, "v"), (k_scale, "k_scale"), (v_scale, "v_scale"),
                           (page_table, "page_table"), (status, "status"))
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.page_table, self.status, self.fmt = page_table, status, fmt
        self._bufs = _page_bufs(k, v, k_scale, v_scale)
        self._status = _ptr(status)
        self.block = rows // k_scale.shape[2]
        if page_table is None:
            self.B, self.l_cap, ps, mp, n_pages = n, rows, 0, 0, 0
        else:
            _want(page_table, torch.int32, "page_table")
            self.B, mp = page_table.shape
            self.l_cap, ps, n_pages = mp * rows, rows, n
        if status is not None:
            _want(status, torch.int32, "status")
        self.struct = _Kv8Struct(
            k.data_ptr(), v.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(),
            None if page_table is None else page_table.data_ptr(),
            None if status is None else status.data_ptr(), self.l_cap, ps, mp, n_pages,
            self.block, _KV8_FORMAT[fmt])
        self._ref = C.byref(self.struct)

    @classmethod
    def contiguous(cls, B: int, Hkv: int, l_cap: int, block: int = 64, fmt: str = "int8",
                   device="cuda") -> "KV8":
        """A contiguous cache of zeros with a status word."""
        return cls._made(B, Hkv, l_cap, block, fmt, None, device)

    @classmethod
    def paged(cls, pages: int, Hkv: int, page_size: int, page_table: torch.Tensor,
              block: int = 16, fmt: str = "int8") -> "KV8":
        """A pool of pages of zeros with a status word."""
        return cls._made(pages, Hkv, page_size, block, fmt, page_table, page_table.device)

    @classmethod
    def _made(cls, n, Hkv, rows, block, fmt, page_table, device):
        if rows % block:
            raise ValueError(f"block {block} does not divide {rows} rows")
        code = [torch.full((n, Hkv, rows, 128), 128 if fmt == "int8" else 0, dtype=torch.uint8,
                           device=device) for _ in range(2)]
        scale = [torch.zeros((n, Hkv, rows // block), dtype=torch.float32, device=device)
                 for _ in range(2)]
        status = torch.zeros(64, dtype=torch.int32, device=device)
        return cls(*code, *scale, fmt=fmt, page_table=page_table, status=status)


def _cache_batch(cache, lens: torch.Tensor) -> int:
    _want(lens, torch.int32, "lens")
    if cache.d != 128:
        raise ValueError(f"cache rows have {cache.d} elements: only 128 is compiled")
    B = lens.shape[0]
    if lens.dim() != 1 or B > cache.B:
        raise ValueError(f"lens must be int32 [B] with B <= {cache.B}, the cache's sequences")
    return B


def kv8_append(cache: KV8, k_new: torch.Tensor, v_new: torch.Tensor, lens: torch.Tensor,
               cu_new: Optional[torch.Tensor] = None, max_new: Optional[int] = None,
               rope: Optional[RopeTable] = None, positions: Optional[torch.Tensor] = None,
               stream=None) -> KV8:
    """Writes new tokens' rows (bf16 [T][Hkv][128], strided allowed) at the
    last positions before lens[b], quantised, the keys rotated if `rope` is
    given (at positions int32 [T], [axes][T] with a table of several axes, or their
    own).  Ragged with cu_new int32 [B+1] and max_new, else T / B tokens a sequence."""
    B = _cache_batch(cache, lens)
    dev = _gpu((cache.k, "cache"), (k_new, "k_new"), (v_new, "v_new"), (lens, "lens"),
               (cu_new, "cu_new"), (positions, "positions"), (rope.table if rope else None, "rope"))
    T = k_new.shape[0]
    if k_new.shape != (T, cache.Hkv, cache.d) or v_new.shape != k_new.shape:
        raise ValueError(f"k_new and v_new must be [T][{cache.Hkv}][{cache.d}]")
    stride = -1 if positions is None else _axis_positions(positions, rope, T)
    n = _offsets(cu_new, T, max_new, B, "max_new")
    if stride < 0:
        _run_on(dev, stream, lib().kv8_append, cache._ref, _rows(k_new, "k_new"),
                _rows(v_new, "v_new"), _ptr(cu_new), T, n, _ptr(lens), B, cache.Hkv, cache.d,
                rope._ref if rope else None, _ptr(positions))
    else:
        _run_on(dev, stream, lib().kv8_append_axes, cache._ref, _rows(k_new, "k_new"),
                _rows(v_new, "v_new"), _ptr(cu_new), T, n, _ptr(lens), B, cache.Hkv, cache.d,
                rope._ref, rope._axes, _ptr(positions), stride)
    return cache


def kv8_read(cache: KV8, lens: torch.Tensor, n: Optional[int] = None,
             cu: Optional[torch.Tensor] = None, T: Optional[int] = None,
             k_out: Optional[torch.Tensor] = None, v_out: Optional[torch.Tensor] = None,
             stream=None):
    """The last rows before lens[b] back in bf16: n of every sequence, or
    cu[b+1] - cu[b] <= n of sequence b (T tokens in all, known to the host).
    Returns (k_out, v_out), [T][Hkv][128]."""
    B = _cache_batch(cache, lens)
    if n is None or (cu is not None and T is None and k_out is None):
        raise ValueError("pass n, and T (or k_out and v_out) with offsets")
    if T is None:
        T = B * n if cu is None else k_out.shape[0]
    dev = _gpu((cache.k, "cache"), (lens, "lens"), (cu, "cu"), (k_out, "k_out"), (v_out, "v_out"))
    shape = (T, cache.Hkv, cache.d)
    if k_out is None:
        k_out = _new(stream, dev, shape, torch.bfloat16)
    if v_out is None:
        v_out = _new(stream, dev, shape, torch.bfloat16)
    if k_out.shape != shape or v_out.shape != shape:
        raise ValueError(f"k_out and v_out must be {list(shape)}")
    n = _offsets(cu, T, n, B, "n")
    _run_on(dev, stream, lib().kv8_read, cache._ref, _rows(k_out, "k_out"),
            _rows(v_out, "v_out"), _ptr(cu), T, n, _ptr(lens), B, cache.Hkv, cache.d)
    return k_out, v_out


def attn_decode_workspace(B: int, Hq: int, Hkv: int, d: int = 128, device="cuda") -> torch.Tensor:
    """A zeroed workspace of kv8_attn_decode and window_attn_decode."""
    n = int(lib().tsa_attn_decode_workspace_size(B, Hq, Hkv, d))
    return torch.zeros(max(n, 256), dtype=torch.uint8, device=device)


def _attn_decode(fn, ref, q, cache, lens, n_init, n_recent, scale, out, lse_out, workspace,
                 stream):
    B = _cache_batch(cache, lens)
    _want(q, torch.bfloat16, "q")
    Bq, Hq, d = q.shape
    if Bq != B:
        raise ValueError(f"q has {Bq} sequences, lens {B}")
    dev = q.device
    if cache.k.device != dev or lens.device != dev or not q.is_cuda or \
            lse_out is not None and lse_out.device != dev or out is not None or \
            workspace is not None and workspace.device != dev:
        _gpu((q, "q"), (cache.k, "cache"), (lens, "lens"), (out, "out"), (lse_out, "lse_out"),
             (workspace, "workspace"))
    if scale is None:
        scale = d ** -0.5
    if out is None:
        out = _new(stream, dev, (B, Hq, d), torch.float32)
    elif out.shape != q.shape:
        raise ValueError("out must have q's shape")
    else:
        _want(out, torch.float32, "out")
    if lse_out is not None:
        _want(lse_out, torch.float32, "lse_out")
        if lse_out.shape != (B, Hq):
            raise ValueError(f"lse_out must be fp32 [{B}][{Hq}]")
    if workspace is None:
        n = int(lib().tsa_attn_decode_workspace_size(B, Hq, cache.Hkv, d))
        workspace = _new(stream, dev, (max(n, 256),), torch.uint8, zero=True)
    _run_on(dev, stream, fn, _ptr(q), ref, _ptr(lens), B, Hq, cache.Hkv, d, int(n_init),
            cache.l_cap if n_recent is None else int(n_recent), float(scale), _ptr(out),
            _ptr(lse_out), _ptr(workspace), workspace.nbytes)
    return out, lse_out


def kv8_attn_decode(q: torch.Tensor, cache: KV8, lens: torch.Tensor, n_init: int = 0,
                    n_recent: Optional[int] = None, scale: Optional[float] = None,
                    out: Optional[torch.Tensor] = None, lse_out: Optional[torch.Tensor] = None,
                    workspace: Optional[torch.Tensor] = None, stream=None):
    """One decode step of attention over the 8-bit cache: q bf16 [B][Hq][128],
    all rows (n_recent None) or the sinks and the window.  Returns (out fp32
    [B][Hq][128], lse_out)."""
    return _attn_decode(lib().kv8_attn_decode, cache._ref, q, cache, lens, n_init, n_recent,
                        scale, out, lse_out, workspace, stream)


def window_attn_decode(q: torch.Tensor, kv: KV, lens: torch.Tensor, n_init: int,
                       n_recent: Optional[int], scale: Optional[float] = None,
                       out: Optional[torch.Tensor] = None,
                       lse_out: Optional[torch.Tensor] = None,
                       workspace: Optional[torch.Tensor] = None, stream=None):
    """One decode step over a bf16 cache, the first n_init and the last
    n_recent rows visible (None: all).  Returns (out fp32, lse_out), a partial
    that lse_merge takes."""
    return _attn_decode(lib().window_attn_decode, C.byref(kv.struct), q, kv, lens, n_init,
                        n_recent, scale, out, lse_out, workspace, stream)


def window_attn_prefill_workspace(B: int, Hq: int, Hkv: int, max_q: int, l_cap: int, n_init: int,
                                  n_recent: Optional[int], d: int = 128,
                                  device="cuda") -> torch.Tensor:
    """A zeroed workspace of window_attn_prefill for these sizes."""
    n = int(lib().window_attn_prefill_workspace_size(
        B, Hq, Hkv, d, _count(max_q, "max_q"), l_cap, n_init, l_cap if n_recent is None else n_recent))
    return torch.zeros(max(n, 256), dtype=torch.uint8, device=device)


def window_attn_prefill(q: torch.Tensor, kv: KV, lens: torch.Tensor, n_init: int,
                        n_recent: Optional[int], cu_q: Optional[torch.Tensor] = None,
                        max_q: Optional[int] = None, scale: Optional[float] = None,
                        out: Optional[torch.Tensor] = None,
                        lse_out: Optional[torch.Tensor] = None,
                        workspace: Optional[torch.Tensor] = None, stream=None):
    """Many new tokens per sequence over a bf16 cache that holds them: q bf16
    [T][Hq][128] (strided allowed), ragged with cu_q int32 [B+1] and max_q, else
    T / B tokens a sequence.  Returns (out bf16 [T][Hq][128], lse_out)."""
    B = _cache_batch(kv, lens)
    T, Hq, d = q.shape
    dev = _gpu((q, "q"), (kv.k, "kv"), (lens, "lens"), (cu_q, "cu_q"), (out, "out"),
               (lse_out, "lse_out"), (workspace, "workspace"))
    n = _offsets(cu_q, T, max_q, B, "max_q")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        out = _new(stream, dev, (T, Hq, d), torch.bfloat16)
    elif out.shape != q.shape:
        raise ValueError("out must have q's shape")
    else:
        _want(out, torch.bfloat16, "out")
    if lse_out is not None:
        _want(lse_out, torch.float32, "lse_out")
        if lse_out.shape != (T, Hq):
            raise ValueError(f"lse_out must be fp32 [{T}][{Hq}]")
    nr = kv.l_cap if n_recent is None else int(n_recent)
    if workspace is None:
        nb = int(lib().window_attn_prefill_workspace_size(B, Hq, kv.Hkv, d, n, kv.l_cap,
                                                          int(n_init), nr))
        workspace = _new(stream, dev, (max(nb, 256),), torch.uint8, zero=True)
    _run_on(dev, stream, lib().window_attn_prefill, _rows(q, "q"), C.byref(kv.struct),
            _ptr(cu_q), T, n, _ptr(lens), B, Hq, kv.Hkv, d, int(n_init), nr, float(scale),
            _ptr(out), _ptr(lse_out), _ptr(workspace), workspace.nbytes)
    return out, lse_out


def shared_attn_decode_workspace(B: int, N: int, Hq: int, Hkv: int, d: int = 128,
                                 device="cuda") -> torch.Tensor:
    """A zeroed workspace of shared_attn_decode for N groups."""
    n = int(lib().tsa_shared_attn_workspace_size(B, N, Hq, Hkv, d))
    return torch.zeros(max(n, 256), dtype=torch.uint8, device=device)


def shared_attn_decode(q: torch.Tensor, cache, lens: torch.Tensor, cu_group: torch.Tensor,
                       shared: torch.Tensor, scale: Optional[float] = None,
                       out: Optional[torch.Tensor] = None,
                       lse_out: Optional[torch.Tensor] = None,
                       workspace: Optional[torch.Tensor] = None, stream=None):
    """One decode step of a batch in groups that share their first rows: sequences
    [cu_group[n], cu_group[n+1]) (int32 [N+1]) begin with the same shared[n] rows (int32
    [N]), which are read once a group.  q: bf16 [B][Hq][128]; cache: a KV or a KV8.
    Returns (out [B][Hq][128], fp32 unless a bf16 one is passed, lse_out)."""
    B = _cache_batch(cache, lens)
    _want(q, torch.bfloat16, "q")
    Bq, Hq, d = q.shape
    if Bq != B:
        raise ValueError(f"q has {Bq} sequences, lens {B}")
    _want(cu_group, torch.int32, "cu_group")
    _want(shared, torch.int32, "shared")
    N = shared.numel()
    if shared.dim() != 1 or cu_group.shape != (N + 1,):
        raise ValueError("cu_group must be int32 [N + 1], shared int32 [N]")
    dev = _gpu((q, "q"), (cache.k, "cache"), (lens, "lens"), (cu_group, "cu_group"),
               (shared, "shared"), (out, "out"), (lse_out, "lse_out"), (workspace, "workspace"))
    if scale is None:
        scale = d ** -0.5
    if out is None:
        out = _new(stream, dev, (B, Hq, d), torch.float32)
    elif out.shape != q.shape or out.dtype not in (torch.float32, torch.bfloat16) or \
            not out.is_contiguous():
        raise ValueError("out must be a contiguous fp32 or bf16 tensor of q's shape")
    if lse_out is not None:
        _want(lse_out, torch.float32, "lse_out")
        if lse_out.shape != (B, Hq):
            raise ValueError(f"lse_out must be fp32 [{B}][{Hq}]")
    if workspace is None:
        n = int(lib().tsa_shared_attn_workspace_size(B, N, Hq, cache.Hkv, d))
        workspace = _new(stream, dev, (max(n, 256),), torch.uint8, zero=True)
    fn, ref = (lib().kv8_shared_attn_decode, cache._ref) if isinstance(cache, KV8) else \
        (lib().shared_attn_decode, C.byref(cache.struct))
    _run_on(dev, stream, fn, _ptr(q), ref, _ptr(lens), B, _ptr(cu_group), _ptr(shared), N, Hq,
            cache.Hkv, d, float(scale), _ptr(out), 1 if out.dtype == torch.bfloat16 else 0,
            _ptr(lse_out), _ptr(workspace), workspace.nbytes)
    return out, lse_out


class Pages:
    """Which pages of a pool the sequences have (tsa_pages in include/tsa.h).

    table: int32 [B][max_pages], the page table of the layers' caches (entries without a
    page are -1); refs: int32 [n_pages], how many entries name a page (0: free).  Calls on
    one Pages must be ordered on a stream; workspace_status(pages.workspace) tells what
    they flagged."""

    def __init__(self, table: torch.Tensor, refs: torch.Tensor, page_size: int):
        _want(table, torch.int32, "table")
        _want(refs, torch.int32, "refs")
        if table.dim() != 2 or refs.dim() != 1:
            raise ValueError("table must be int32 [B][max_pages], refs int32 [n_pages]")
        self.device = _gpu((table, "table"), (refs, "refs"))
        self.table, self.refs, self.page_size = table, refs, int(page_size)
        self.B, self.max_pages = table.shape
        self.n_pages = refs.numel()
        n = int(lib().tsa_pages_workspace_size(self.B, self.max_pages, self.n_pages))
        self.workspace = torch.zeros(max(n, 256), dtype=torch.uint8, device=self.device)
        self._ws, self._ws_bytes = self.workspace.data_ptr(), self.workspace.nbytes
        self.struct = _PagesStruct(table.data_ptr(), refs.data_ptr(), self.B, self.max_pages,
                                   self.n_pages, self.page_size)
        self._ref = C.byref(self.struct)

    @classmethod
    def empty(cls, B: int, max_pages: int, n_pages: int, page_size: int,
              device="cuda") -> "Pages":
        """All pages free, no sequence with any."""
        return cls(torch.full((B, max_pages), -1, dtype=torch.int32, device=device),
                   torch.zeros(n_pages, dtype=torch.int32, device=device), page_size)

    def _run(self, fn, stream, *args):
        _run_on(self.device, stream, fn, self._ref, *args, self._ws, self._ws_bytes)

    def _ints(self, n: int, **named):
        """The int32 [n] tensors given (or None) on the pages' device, as pointers."""
        out = []
        for name, t in named.items():
            if t is None:
                out.append(None)
                continue
            if t.dtype != torch.int32:
                raise TypeError(f"{name} must be {torch.int32}, got {t.dtype}")
            if t.shape != (n,) or not t.is_contiguous():
                raise ValueError(f"{name} must be contiguous int32 [{n}], got {tuple(t.shape)}")
            if t.device != self.device:
                _gpu((self.table, "pages"), (t, name))
            out.append(t.data_ptr())
        return out


def pages_alloc(pages: Pages, lo: torch.Tensor, hi: torch.Tensor, stream=None) -> Pages:
    """Gives sequence b a free page (the lowest ones) for every entry that holds a
    position of [lo[b], hi[b]) and has none."""
    pages._run(lib().pages_alloc, stream, *pages._ints(pages.B, lo=lo, hi=hi))
    return pages


def pages_free(pages: Pages, lo: torch.Tensor, hi: torch.Tensor, stream=None) -> Pages:
    """Takes from sequence b the pages that lie in positions [lo[b], hi[b]) altogether."""
    pages._run(lib().pages_free, stream, *pages._ints(pages.B, lo=lo, hi=hi))
    return pages


def pages_fork(pages: Pages, parents: torch.Tensor, children: torch.Tensor, lens: torch.Tensor,
               src: Optional[torch.Tensor] = None, dst: Optional[torch.Tensor] = None,
               stream=None):
    """Sequence children[i] becomes the first lens[i] positions of parents[i]: whole
    pages are shared, a partial last one gets a page of its own.  Returns (src, dst),
    int32 [n], the pages that pages_copy has to copy (-1: none)."""
    n = parents.numel()
    if src is None or dst is None:
        new = _new(stream, pages.device, (2, n), torch.int32).unbind(0)
        src, dst = new[0] if src is None else src, new[1] if dst is None else dst
    p = pages._ints(n, parents=parents, children=children, lens=lens, src=src, dst=dst)
    pages._run(lib().pages_fork, stream, p[0], p[1], p[2], n, p[3], p[4])
    return src, dst


def pages_compact(pages: Pages, src: Optional[torch.Tensor] = None,
                  dst: Optional[torch.Tensor] = None, count: Optional[torch.Tensor] = None,
                  stream=None):
    """Moves the pages in use to the front of the pool (tables and counts; the rows are
    moved by pages_copy).  Returns (src, dst, count): int32 [n_pages // 2] twice, padded
    with -1, and int32 [1]."""
    n = pages.n_pages // 2
    if src is None or dst is None:
        new = _new(stream, pages.device, (2, n), torch.int32).unbind(0)
        src, dst = new[0] if src is None else src, new[1] if dst is None else dst
    if count is None:
        count = _new(stream, pages.device, (1,), torch.int32)
    pages._run(lib().pages_compact, stream, *pages._ints(n, src=src, dst=dst),
               *pages._ints(1, count=count))
    return src, dst, count


def pages_copy(caches, src: torch.Tensor, dst: torch.Tensor,
               count: Optional[torch.Tensor] = None, stream=None,
               pages: Optional[Pages] = None) -> None:
    """Copies page src[i] over page dst[i] (int32 [n], -1: none) in every cache given (a
    paged KV or KV8, or a list of them, of one pool size); count: int32 [1], how many
    pairs count.  Pages outside the pool are skipped, and flagged in the first status word
    among the caches, or, where none has one (bf16 caches), in the workspace of `pages`."""
    if not isinstance(caches, (list, tuple)):
        caches = (caches,)
    n = src.numel()
    for t, name, size in ((src, "src", n), (dst, "dst", n), (count, "count", 1)):
        if t is not None:
            _want(t, torch.int32, name)
            if t.shape != (size,):
                raise ValueError(f"{name} must be int32 [{size}], got {tuple(t.shape)}")
    if not caches:
        return
    n_pages, dev, status = caches[0].k.shape[0], src.device, None
    for c in caches:
        if c.page_table is None:
            raise ValueError("pages_copy needs paged caches")
        if c.k.shape[0] != n_pages:
            raise ValueError("the caches' pools must have the same number of pages")
        if c.k.device != dev:
            _gpu((src, "src"), (c.k, "a cache"))
        status = status or getattr(c, "_status", None)
    if pages is not None:
        if pages.device != dev:
            _gpu((src, "src"), (pages.table, "pages"))
        status = status or pages._ws
    if dst.device != dev or dev.type != "cuda" or count is not None and count.device != dev:
        _gpu((src, "src"), (dst, "dst"), (count, "count"))
    if n_pages == 0:
        return
    bufs = b"".join([c._bufs for c in caches])
    _run_on(dev, stream, lib().pages_copy, bufs, len(bufs) // 16, n_pages, src.data_ptr(),
            dst.data_ptr(), _ptr(count), n, status)
