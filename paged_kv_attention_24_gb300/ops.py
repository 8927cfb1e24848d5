"""Thin ctypes binding over libmsgl_attn (argument marshalling only).

Every function here converts torch tensors to raw device pointers and host
scalars, calls the C ABI declared in ``include/msgl_attn.h`` with the
current CUDA stream, and turns a non-OK status into :class:`MsglError`.
All compute happens in the library's CUDA kernels; there is no CPU or
PyTorch fallback, and calling anything here without the built library
raises immediately.  The step tables, the prefix groups, the shared-prefix
decode, the rotary store, the draft verification and the page calls, whose
kernels are short, marshal their arguments in a native extension over the
same C ABI (``csrc/python/binding.cpp``).
"""
from __future__ import annotations

import ctypes
import importlib.util
import math
import os
import threading
from typing import NamedTuple, Optional

import torch

from .build import binding_path

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "_build", "libmsgl_attn.so")

MSGL_OK = 0
STATUS_NAMES = {0: "OK", 1: "INVALID_ARG", 2: "UNSUPPORTED", 3: "CUDA", 4: "OUT_OF_RANGE",
                5: "TIMEOUT", 6: "WORKSPACE"}
DEVERR_SLOT_RANGE = 0x1
DEVERR_PAGE_RANGE = 0x2
DEVERR_LENGTH = 0x4
DEVERR_POSITION = 0x8
DEVERR_TIMEOUT = 0x10
DEVERR_APPEND_SLOT = 0x20
DEVERR_GROUP = 0x40
DEVERR_NO_PAGES = 0x80
DEVERR_ROW = 0x100
DEVERR_TOKEN = 0x200
DEVERR_PROBS = 0x400


class MsglError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"msgl status {STATUS_NAMES.get(status, status)}: {message}")
        self.status = status


class _Pool(ctypes.Structure):
    _fields_ = [("k_pool", ctypes.c_void_p), ("v_pool", ctypes.c_void_p),
                ("num_slots", ctypes.c_int64), ("page_size", ctypes.c_int32),
                ("num_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32)]


class _Pages(ctypes.Structure):
    _fields_ = [("page_ids", ctypes.c_void_p), ("stride", ctypes.c_int32),
                ("width", ctypes.c_int32)]


class _ExtendBatch(ctypes.Structure):
    _fields_ = [("pages", _Pages), ("q", ctypes.c_void_p), ("prefix_lens", ctypes.c_void_p),
                ("ext_lens", ctypes.c_void_p), ("cu_ext", ctypes.c_void_p), ("positions", ctypes.c_void_p),
                ("num_reqs", ctypes.c_int32), ("total_tokens", ctypes.c_int32),
                ("max_ext_len", ctypes.c_int32), ("max_seq_len", ctypes.c_int32),
                ("o", ctypes.c_void_p), ("lse", ctypes.c_void_p)]


class _DecodeBatch(ctypes.Structure):
    _fields_ = [("pages", _Pages), ("q", ctypes.c_void_p), ("seq_lens", ctypes.c_void_p),
                ("num_reqs", ctypes.c_int32), ("max_seq_len", ctypes.c_int32),
                ("o", ctypes.c_void_p), ("lse", ctypes.c_void_p)]


class _StepOut(ctypes.Structure):
    _fields_ = [("page_ids", ctypes.c_void_p), ("stride", ctypes.c_int32), ("width", ctypes.c_int32),
                ("seq_lens", ctypes.c_void_p), ("cu_ext", ctypes.c_void_p), ("positions", ctypes.c_void_p),
                ("out_loc", ctypes.c_void_p), ("pages_taken", ctypes.c_void_p),
                ("total_tokens", ctypes.c_int32)]


class _Rope(ctypes.Structure):
    _fields_ = [("turns", ctypes.c_void_p), ("axes", ctypes.c_void_p), ("num_pairs", ctypes.c_int32),
                ("num_axes", ctypes.c_int32), ("adjacent", ctypes.c_int32), ("factor", ctypes.c_float)]


class _NewTokens(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("q_out", ctypes.c_void_p),
                ("q_stride", ctypes.c_int64), ("k_stride", ctypes.c_int64), ("v_stride", ctypes.c_int64),
                ("out_stride", ctypes.c_int64), ("positions", ctypes.c_void_p), ("axis_stride", ctypes.c_int64),
                ("out_loc", ctypes.c_void_p), ("n_tokens", ctypes.c_int32), ("num_q_heads", ctypes.c_int32)]


class _DraftBatch(ctypes.Structure):
    _fields_ = [("target", ctypes.c_void_p), ("draft", ctypes.c_void_p), ("target_stride", ctypes.c_int64),
                ("draft_stride", ctypes.c_int64), ("vocab", ctypes.c_int32), ("is_bf16", ctypes.c_int32),
                ("tokens", ctypes.c_void_p), ("cu_ext", ctypes.c_void_p), ("accept_u", ctypes.c_void_p),
                ("sample_u", ctypes.c_void_p), ("cached_lens", ctypes.c_void_p), ("num_reqs", ctypes.c_int32),
                ("total_tokens", ctypes.c_int32), ("accepted", ctypes.c_void_p), ("out_tokens", ctypes.c_void_p),
                ("kv_lens", ctypes.c_void_p)]


class _ForkOut(ctypes.Structure):
    _fields_ = [("copy_src", ctypes.c_void_p), ("copy_dst", ctypes.c_void_p), ("copy_tokens", ctypes.c_void_p),
                ("pages_taken", ctypes.c_void_p)]


class _CompactOut(ctypes.Structure):
    _fields_ = [("page_ids", ctypes.c_void_p), ("stride", ctypes.c_int32), ("remap", ctypes.c_void_p),
                ("src", ctypes.c_void_p), ("dst", ctypes.c_void_p), ("num_moves", ctypes.c_void_p),
                ("num_used", ctypes.c_void_p)]


_lib = None
_lock = threading.Lock()

P, I32, I64, SZ, F32 = (ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t,
                        ctypes.c_float)
PP = ctypes.POINTER(_Pool)
PT = ctypes.POINTER(_Pages)

SIGNATURES = {
    "msgl_store_kv": ([PP, P, P, P, I32, P, P], ctypes.c_int),
    "msgl_extend_workspace_size": ([I32, I32, I32, I32, I32, I32], SZ),
    "msgl_attn_extend": ([PP, PT, P, I32, P, P, P, P, I32, I32, I32, I32, F32, P, P, P, SZ, P, P],
                         ctypes.c_int),
    "msgl_decode_workspace_size": ([I32, I32, I32, I32, I32], SZ),
    "msgl_attn_decode": ([PP, PT, P, I32, P, I32, I32, F32, P, P, P, SZ, P, P], ctypes.c_int),
    "msgl_attn_decode_append": ([PP, PT, P, I32, P, P, P, P, I32, I32, F32, P, P, P, SZ, P, P], ctypes.c_int),
    "msgl_attn_decode_noalloc": ([PP, PT, P, I32, P, I32, I32, F32, P, P, P, P], ctypes.c_int),
    "msgl_attn_mixed": ([PP, ctypes.POINTER(_ExtendBatch), ctypes.POINTER(_DecodeBatch), I32, F32, P, SZ, P, P],
                        ctypes.c_int),
    "msgl_step_tables": ([I64, I32, P, I32, I32, I32, P, P, P, I32, P, I32, ctypes.POINTER(_StepOut), P, P],
                         ctypes.c_int),
    "msgl_shared_prefixes": ([PT, P, I32, I32, I32, I32, P, P, P, P], ctypes.c_int),
    "msgl_decode_shared_workspace_size": ([I32, I32, I32, I32, I32], SZ),
    "msgl_attn_decode_shared": ([PP, PT, P, I32, P, P, P, I32, I32, I32, F32, P, P, P, SZ, P, P], ctypes.c_int),
    "msgl_rope_store_kv": ([PP, ctypes.POINTER(_NewTokens), ctypes.POINTER(_Rope), P, P, F32, P, P], ctypes.c_int),
    "msgl_verify_drafts": ([ctypes.POINTER(_DraftBatch), P, P], ctypes.c_int),
    "msgl_fork_requests": ([I64, I32, P, I32, I32, I32, P, P, P, I32, P, I32, ctypes.POINTER(_ForkOut), P, P],
                           ctypes.c_int),
    "msgl_copy_pages": ([PP, I32, P, P, P, I32, P, P, P], ctypes.c_int),
    "msgl_page_map_workspace_size": ([I64, I32], SZ),
    "msgl_free_pages": ([I64, I32, P, I32, I32, I32, P, P, I32, P, P, P, P, SZ, P, P], ctypes.c_int),
    "msgl_compact_pages": ([I64, I32, P, I32, I32, I32, P, P, I32, P, ctypes.POINTER(_CompactOut), P, SZ, P, P],
                           ctypes.c_int),
    "msgl_selftest_wait_timeout": ([P, I64, P], ctypes.c_int),
    "msgl_read_status": ([P, ctypes.POINTER(ctypes.c_uint32), P], ctypes.c_int),
    "msgl_status_string": ([ctypes.c_int], ctypes.c_char_p),
    "msgl_last_error": ([], ctypes.c_char_p),
    "msgl_abi_version": ([], I32),
    "msgl_check_store_meta": ([I64, P, I32], ctypes.c_int),
    "msgl_check_extend_meta": ([I64, I32, P, I32, I32, P, P, P, P, I32, I32, I32, I32], ctypes.c_int),
    "msgl_check_decode_meta": ([I64, I32, P, I32, I32, P, I32, I32], ctypes.c_int),
    "msgl_check_step_meta": ([I64, I32, P, I32, I32, I32, P, P, P, I32, P, I32, I32], ctypes.c_int),
    "msgl_check_groups_meta": ([I64, I32, P, I32, I32, P, P, P, I32, I32], ctypes.c_int),
    "msgl_check_fork_meta": ([I64, I32, P, I32, I32, I32, P, P, P, I32, P, I32], ctypes.c_int),
    "msgl_check_copy_meta": ([I64, I32, P, P, P, I32], ctypes.c_int),
    "msgl_check_held_meta": ([I64, I32, P, I32, I32, I32, P, P, I32], ctypes.c_int),
    "msgl_check_draft_meta": ([I32, P, P, P, P, I32, I32], ctypes.c_int),
}


def load(path: Optional[str] = None):
    """Load the library (once).  Raises if it has not been built."""
    global _lib
    with _lock:
        if _lib is not None and path is None:
            return _lib
        p = path or LIB_PATH
        if not os.path.exists(p):
            raise RuntimeError(f"libmsgl_attn is not built ({p} missing); run "
                               "`python -c 'import __graft_entry__ as g; g.build()'`")
        lib = ctypes.CDLL(p)
        for name, (args, res) in SIGNATURES.items():
            fn = getattr(lib, name)
            fn.argtypes = args
            fn.restype = res
        if path is None:
            _lib = lib
        return lib


def _check(rc: int, what: str):
    if rc != MSGL_OK:
        msg = load().msgl_last_error().decode(errors="replace")
        raise MsglError(rc, f"{what}: {msg}")


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _need(t: torch.Tensor, name: str, dtype: torch.dtype):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


class KVPool:
    """A layer's unified KV pool: bf16 K and V tensors [num_slots, Hkv, 128]."""

    def __init__(self, k_pool: torch.Tensor, v_pool: torch.Tensor, page_size: int):
        _need(k_pool, "k_pool", torch.bfloat16)
        _need(v_pool, "v_pool", torch.bfloat16)
        if k_pool.shape != v_pool.shape or k_pool.dim() != 3:
            raise ValueError("k_pool and v_pool must both be [num_slots, Hkv, D]")
        self.k, self.v, self.page_size = k_pool, v_pool, int(page_size)

    @property
    def num_kv_heads(self) -> int:
        return int(self.k.shape[1])

    def c(self) -> _Pool:
        return _Pool(self.k.data_ptr(), self.v.data_ptr(), self.k.shape[0], self.page_size,
                     self.k.shape[1], self.k.shape[2])


def _pages(page_table: torch.Tensor) -> _Pages:
    _need(page_table, "page_table", torch.int32)
    if page_table.dim() != 2:
        raise ValueError("page_table must be [num_reqs, width]")
    return _Pages(page_table.data_ptr(), page_table.shape[1], page_table.shape[1])


def new_status(device=None) -> torch.Tensor:
    return torch.zeros(1, dtype=torch.int32, device=device or "cuda")


def store_kv(pool: KVPool, k: torch.Tensor, v: torch.Tensor, out_loc: torch.Tensor,
             status: Optional[torch.Tensor] = None, stream=None) -> None:
    """pool.k[out_loc[t]] = k[t]; pool.v[out_loc[t]] = v[t] (bit-exact)."""
    _need(k, "k", torch.bfloat16)
    _need(v, "v", torch.bfloat16)
    _need(out_loc, "out_loc", torch.int32)
    pc = pool.c()
    rc = load().msgl_store_kv(ctypes.byref(pc), _ptr(k), _ptr(v), _ptr(out_loc), int(out_loc.shape[0]),
                              _ptr(status), _stream(stream))
    _check(rc, "msgl_store_kv")


def decode_workspace_size(num_reqs: int, hq: int, hkv: int, max_seq_len: int, head_dim: int = 128) -> int:
    return int(load().msgl_decode_workspace_size(num_reqs, hq, hkv, head_dim, max_seq_len))


def extend_workspace_size(num_reqs: int, total_tokens: int, hq: int, hkv: int, max_seq_len: int,
                          head_dim: int = 128) -> int:
    return int(load().msgl_extend_workspace_size(num_reqs, total_tokens, hq, hkv, head_dim, max_seq_len))


def _workspace(nbytes: int, device) -> Optional[torch.Tensor]:
    if nbytes == 0:
        return None
    return torch.empty(nbytes, dtype=torch.uint8, device=device)


def attn_decode(pool: KVPool, q: torch.Tensor, page_table: torch.Tensor, seq_lens: torch.Tensor,
                max_seq_len: int, scale: float, out: Optional[torch.Tensor] = None,
                lse: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                status: Optional[torch.Tensor] = None, stream=None):
    """One query row per request over all its pages; returns (o bf16 [B,Hq,D], lse fp32 [B,Hq])."""
    _need(q, "q", torch.bfloat16)
    _need(seq_lens, "seq_lens", torch.int32)
    B, hq, d = q.shape
    out = torch.empty_like(q) if out is None else out
    lse = torch.empty(B, hq, dtype=torch.float32, device=q.device) if lse is None else lse
    _need(out, "out", torch.bfloat16)
    _need(lse, "lse", torch.float32)
    if workspace is None:
        workspace = _workspace(decode_workspace_size(B, hq, pool.num_kv_heads, max_seq_len, d), q.device)
    pc, pt = pool.c(), _pages(page_table)
    rc = load().msgl_attn_decode(
        ctypes.byref(pc), ctypes.byref(pt), _ptr(q), hq, _ptr(seq_lens), B, int(max_seq_len),
        float(scale), _ptr(out), _ptr(lse), _ptr(workspace),
        0 if workspace is None else workspace.numel() * workspace.element_size(), _ptr(status),
        _stream(stream))
    _check(rc, "msgl_attn_decode")
    return out, lse


def attn_extend(pool: KVPool, q: torch.Tensor, page_table: torch.Tensor, prefix_lens: torch.Tensor,
                ext_lens: torch.Tensor, cu_ext: torch.Tensor, max_ext_len: int, max_seq_len: int,
                scale: float, positions: Optional[torch.Tensor] = None,
                out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                workspace: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
                stream=None):
    """Chunked prefill over cached prefix + causal chunk; returns (o [T,Hq,D], lse [T,Hq])."""
    _need(q, "q", torch.bfloat16)
    for name, t in (("prefix_lens", prefix_lens), ("ext_lens", ext_lens), ("cu_ext", cu_ext)):
        _need(t, name, torch.int32)
    if positions is not None:
        _need(positions, "positions", torch.int32)
    T, hq, d = q.shape
    B = int(prefix_lens.shape[0])
    out = torch.empty_like(q) if out is None else out
    lse = torch.empty(T, hq, dtype=torch.float32, device=q.device) if lse is None else lse
    _need(out, "out", torch.bfloat16)
    _need(lse, "lse", torch.float32)
    if workspace is None:
        workspace = _workspace(extend_workspace_size(B, T, hq, pool.num_kv_heads, max_seq_len, d), q.device)
    pc, pt = pool.c(), _pages(page_table)
    rc = load().msgl_attn_extend(
        ctypes.byref(pc), ctypes.byref(pt), _ptr(q), hq, _ptr(prefix_lens), _ptr(ext_lens),
        _ptr(cu_ext), _ptr(positions), B, T, int(max_ext_len), int(max_seq_len), float(scale),
        _ptr(out), _ptr(lse), _ptr(workspace),
        0 if workspace is None else workspace.numel() * workspace.element_size(), _ptr(status),
        _stream(stream))
    _check(rc, "msgl_attn_extend")
    return out, lse


def attn_decode_append(pool: KVPool, q: torch.Tensor, k_new: torch.Tensor, v_new: torch.Tensor,
                       new_loc: torch.Tensor, page_table: torch.Tensor, seq_lens: torch.Tensor,
                       max_seq_len: int, scale: float, out: Optional[torch.Tensor] = None,
                       lse: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                       status: Optional[torch.Tensor] = None, stream=None):
    """Store each request's current-token K/V at new_loc and decode, in one launch."""
    _need(q, "q", torch.bfloat16)
    _need(k_new, "k_new", torch.bfloat16)
    _need(v_new, "v_new", torch.bfloat16)
    _need(new_loc, "new_loc", torch.int32)
    _need(seq_lens, "seq_lens", torch.int32)
    B, hq, d = q.shape
    out = torch.empty_like(q) if out is None else out
    lse = torch.empty(B, hq, dtype=torch.float32, device=q.device) if lse is None else lse
    _need(out, "out", torch.bfloat16)
    _need(lse, "lse", torch.float32)
    if workspace is None:
        workspace = _workspace(decode_workspace_size(B, hq, pool.num_kv_heads, max_seq_len, d), q.device)
    pc, pt = pool.c(), _pages(page_table)
    rc = load().msgl_attn_decode_append(
        ctypes.byref(pc), ctypes.byref(pt), _ptr(q), hq, _ptr(k_new), _ptr(v_new), _ptr(new_loc),
        _ptr(seq_lens), B, int(max_seq_len), float(scale), _ptr(out), _ptr(lse), _ptr(workspace),
        0 if workspace is None else workspace.numel() * workspace.element_size(), _ptr(status),
        _stream(stream))
    _check(rc, "msgl_attn_decode_append")
    return out, lse


def attn_mixed(pool: KVPool, scale: float,
               ext_q: torch.Tensor, ext_page_table: torch.Tensor, prefix_lens: torch.Tensor,
               ext_lens: torch.Tensor, cu_ext: torch.Tensor, max_ext_len: int, max_ext_seq_len: int,
               dec_q: torch.Tensor, dec_page_table: torch.Tensor, seq_lens: torch.Tensor, max_dec_seq_len: int,
               positions: Optional[torch.Tensor] = None, ext_out=None, ext_lse=None, dec_out=None, dec_lse=None,
               workspace: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None, stream=None):
    """The extend batch and the decode batch of one forward in one call (msgl_attn_mixed).

    Same results as :func:`attn_extend` and :func:`attn_decode`; returns
    ((o_ext, lse_ext), (o_dec, lse_dec)).
    """
    _need(ext_q, "ext_q", torch.bfloat16)
    _need(dec_q, "dec_q", torch.bfloat16)
    for name, t in (("prefix_lens", prefix_lens), ("ext_lens", ext_lens), ("cu_ext", cu_ext),
                    ("seq_lens", seq_lens)):
        _need(t, name, torch.int32)
    if positions is not None:
        _need(positions, "positions", torch.int32)
    T, hq, d = ext_q.shape
    B = int(dec_q.shape[0])
    if dec_q.shape[1] != hq:
        raise ValueError("ext_q and dec_q must have the same number of q heads")
    ext_out = torch.empty_like(ext_q) if ext_out is None else ext_out
    ext_lse = torch.empty(T, hq, dtype=torch.float32, device=ext_q.device) if ext_lse is None else ext_lse
    dec_out = torch.empty_like(dec_q) if dec_out is None else dec_out
    dec_lse = torch.empty(B, hq, dtype=torch.float32, device=dec_q.device) if dec_lse is None else dec_lse
    for name, t, dt in (("ext_out", ext_out, torch.bfloat16), ("ext_lse", ext_lse, torch.float32),
                        ("dec_out", dec_out, torch.bfloat16), ("dec_lse", dec_lse, torch.float32)):
        _need(t, name, dt)
    if workspace is None:
        workspace = _workspace(mixed_workspace_size(B, T, int(prefix_lens.shape[0]), hq, pool.num_kv_heads,
                                                    max_ext_seq_len, max_dec_seq_len, d), dec_q.device)
    eb = _ExtendBatch(_pages(ext_page_table), ext_q.data_ptr(), prefix_lens.data_ptr(), ext_lens.data_ptr(),
                      cu_ext.data_ptr(), None if positions is None else positions.data_ptr(),
                      int(prefix_lens.shape[0]), T, int(max_ext_len), int(max_ext_seq_len),
                      ext_out.data_ptr(), ext_lse.data_ptr())
    db = _DecodeBatch(_pages(dec_page_table), dec_q.data_ptr(), seq_lens.data_ptr(), B, int(max_dec_seq_len),
                      dec_out.data_ptr(), dec_lse.data_ptr())
    pc = pool.c()
    rc = load().msgl_attn_mixed(ctypes.byref(pc), ctypes.byref(eb), ctypes.byref(db), hq, float(scale),
                                _ptr(workspace),
                                0 if workspace is None else workspace.numel() * workspace.element_size(),
                                _ptr(status), _stream(stream))
    _check(rc, "msgl_attn_mixed")
    return (ext_out, ext_lse), (dec_out, dec_lse)


def mixed_workspace_size(dec_reqs: int, ext_tokens: int, ext_reqs: int, hq: int, hkv: int,
                         max_ext_seq_len: int, max_dec_seq_len: int, head_dim: int = 128) -> int:
    """Workspace bytes of :func:`attn_mixed`: the decode's (rounded up to 256) plus the extend's."""
    dec = decode_workspace_size(dec_reqs, hq, hkv, max_dec_seq_len, head_dim) if dec_reqs > 0 else 0
    ext = extend_workspace_size(ext_reqs, ext_tokens, hq, hkv, max_ext_seq_len, head_dim) if ext_reqs > 0 else 0
    return (dec + 255) // 256 * 256 + ext


NOALLOC_SCRATCH_BYTES = 32 << 20


def attn_decode_noalloc(pool: KVPool, q: torch.Tensor, page_table: torch.Tensor,
                        seq_lens: torch.Tensor, max_seq_len: int, scale: float,
                        out: torch.Tensor, lse: torch.Tensor,
                        status: Optional[torch.Tensor] = None, stream=None):
    """Decode with the library's built-in scratch instead of a workspace.

    For callers that must not allocate device memory: the caller passes the
    output buffers, and the library allocates nothing.  Same results as
    :func:`attn_decode`.
    """
    _need(q, "q", torch.bfloat16)
    _need(seq_lens, "seq_lens", torch.int32)
    _need(out, "out", torch.bfloat16)
    _need(lse, "lse", torch.float32)
    B, hq, _ = q.shape
    pc, pt = pool.c(), _pages(page_table)
    rc = load().msgl_attn_decode_noalloc(
        ctypes.byref(pc), ctypes.byref(pt), _ptr(q), hq, _ptr(seq_lens), B, int(max_seq_len),
        float(scale), _ptr(out), _ptr(lse), _ptr(status), _stream(stream))
    _check(rc, "msgl_attn_decode_noalloc")
    return out, lse


# ------------------------------------------------- step tables and shared prefixes

class StepTables(NamedTuple):
    """The outputs of :func:`step_tables` (all int32): keep one and pass it as ``out`` to reuse its buffers."""
    page_table: torch.Tensor   # [B, width] page ids; entries past a request's last page are left as they were
    seq_lens: torch.Tensor     # [B]      cached + new tokens
    cu_ext: torch.Tensor       # [B + 1]  prefix sums of the new tokens
    positions: torch.Tensor    # [T]      absolute position of each new token
    out_loc: torch.Tensor      # [T]      pool slot of each new token (-1: none)
    pages_taken: torch.Tensor  # [1]      how many of the free pages are now in use


_native = None


def _binding():
    """The native binding of the calls below (csrc/python/binding.cpp); raises if it has not been built."""
    global _native
    load()
    path = binding_path()
    if not os.path.exists(path):
        raise RuntimeError(f"the native binding is not built ({path} missing); run "
                           "`python -c 'import __graft_entry__ as g; g.build()'`")
    spec = importlib.util.spec_from_file_location("_msgl_binding", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    _native = module
    return module


def _handle(stream):
    return None if stream is None else stream.cuda_stream


def step_tables(req_table: torch.Tensor, cached_lens: torch.Tensor, new_lens: Optional[torch.Tensor],
                free_pages: torch.Tensor, num_slots: int, page_size: int, total_tokens: Optional[int] = None,
                width: Optional[int] = None, req_rows: Optional[torch.Tensor] = None,
                out: Optional[StepTables] = None, status: Optional[torch.Tensor] = None, stream=None) -> StepTables:
    """Block tables and slot maps of one step from its request lengths (msgl_step_tables).

    ``req_table`` int32 [rows, W] holds the page ids of every running request and gets
    this step's new pages, taken from the front of ``free_pages``; request b is row
    ``req_rows[b]`` (b when None), has ``cached_lens[b]`` tokens and gets ``new_lens[b]``
    more (one each when None).  ``total_tokens`` and ``width`` size the outputs when
    ``out`` is not given (W columns by default).  No output may overlap an input: a loop
    whose ``cached_lens`` are the last step's ``seq_lens`` keeps two ``out`` and takes
    them in turn.  ``out.page_table`` may be ``req_table`` itself when ``req_rows`` is None.
    """
    if out is None:
        if total_tokens is None:
            raise ValueError("step_tables needs total_tokens or out")
        B, T, dev = cached_lens.shape[0], int(total_tokens), cached_lens.device

        def i32(*shape):
            return torch.empty(*shape, dtype=torch.int32, device=dev)
        out = StepTables(i32(B, req_table.shape[1] if width is None else int(width)).fill_(-1), i32(B), i32(B + 1),
                         i32(T), i32(T), i32(1))
        if stream is not None:
            for t in out:
                t.record_stream(stream)
            stream.wait_stream(torch.cuda.current_stream(dev))   # behind the fill
    else:
        if total_tokens is not None and total_tokens != out[3].shape[0]:
            raise ValueError("total_tokens must match out")
        if width is not None and width != out[0].shape[1]:
            raise ValueError("width must match out")
    page_table, seq_lens, cu_ext, positions, out_loc, pages_taken = out
    rc = (_native or _binding()).step_tables(req_table, cached_lens, new_lens, free_pages, num_slots, page_size,
                                             req_rows, page_table, seq_lens, cu_ext, positions, out_loc, pages_taken,
                                             status, _handle(stream))
    if rc is not None:
        _check(rc, "msgl_step_tables")
    return out


def shared_prefixes(page_table: torch.Tensor, seq_lens: torch.Tensor, page_size: int, max_seq_len: int,
                    min_shared: int, group_start: Optional[torch.Tensor] = None,
                    shared_lens: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None, stream=None):
    """Groups of neighbouring requests over the same leading pages (msgl_shared_prefixes).

    Returns (group_start int32 [B], shared_lens int32 [B]), the group arguments of
    :func:`attn_decode_shared`.
    """
    r = (_native or _binding()).shared_prefixes(page_table, seq_lens, page_size, max_seq_len, min_shared, group_start,
                                                shared_lens, status, _handle(stream))
    if type(r) is int:
        _check(r, "msgl_shared_prefixes")
    return r


def decode_shared_workspace_size(num_reqs: int, hq: int, hkv: int, max_seq_len: int, head_dim: int = 128) -> int:
    return int(load().msgl_decode_shared_workspace_size(num_reqs, hq, hkv, head_dim, max_seq_len))


SHARING = {"auto": 0, "always": 1, "never": 2}


def attn_decode_shared(pool: KVPool, q: torch.Tensor, page_table: torch.Tensor, seq_lens: torch.Tensor,
                       group_start: torch.Tensor, shared_lens: torch.Tensor, max_seq_len: int, scale: float,
                       out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                       workspace: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None, stream=None,
                       sharing: str = "auto"):
    """:func:`attn_decode` with the keys that a group of requests shares read once for all of them.

    ``group_start[b]`` is the first row of b's group (neighbouring rows) and
    ``shared_lens[b]`` the leading keys the group has in common, read through the first
    row's pages (:func:`shared_prefixes` finds both).  ``sharing`` = "always" or "never"
    settles whether a group's rows go through its shared keys together, which "auto"
    does where the batch's lengths and groups make it pay.  A row's last bits depend on
    the rest of the batch in all three (its keys are cut into pieces by the sums over all
    rows); the same arguments give the same bits.  Returns (o bf16 [B,Hq,D], lse fp32
    [B,Hq]).
    """
    r = (_native or _binding()).attn_decode_shared(pool.k, pool.v, pool.page_size, q, page_table, seq_lens, group_start,
                                                   shared_lens, max_seq_len, scale, out, lse, workspace, status,
                                                   _handle(stream), SHARING[sharing])
    if type(r) is int:
        _check(r, "msgl_attn_decode_shared")
    return r


# ------------------------------- rotary store, drafts, pages between the steps

class Rope:
    """How heads turn by position: made once, an argument of :func:`rope_store_kv`.

    ``inv_freq``: radians per position of each of a head's pairs (8, 16, .. 64 of them; any
    scaling of positions or frequencies is the caller's, in 64 bits).  ``axes``: the row
    of ``positions`` that a pair goes by (all 0 when None): ``[0] * 16 + [1] * 24 + [2] * 24`` for
    sections of time, height and width, ``[0, 1, 2] * 16 + ..`` for interleaved ones.  Pair j is
    dims j and j + pairs, or 2j and 2j + 1 when ``adjacent``; later dims do not turn.
    ``factor`` scales what turns.  The frequencies are kept on ``device`` (the current CUDA device
    when None), where the tensors of the calls have to be.
    """

    def __init__(self, inv_freq, axes=None, adjacent: bool = False, factor: float = 1.0, device=None):
        freq = [float(f) for f in (inv_freq.tolist() if isinstance(inv_freq, torch.Tensor) else inv_freq)]
        axes = [0] * len(freq) if axes is None else [int(a) for a in axes]
        if not freq or len(freq) > 64 or len(freq) % 8:
            raise ValueError("inv_freq must have 8, 16, .. 64 entries")
        if not all(math.isfinite(f) for f in freq) or not math.isfinite(factor):
            raise ValueError("inv_freq and factor must be finite")
        if len(axes) != len(freq) or min(axes) < 0 or max(axes) > 3:
            raise ValueError("axes must have an entry in [0, 3] for each of inv_freq")
        # a fraction of a turn in 64 bits: whole turns of an integer position drop out of the product
        turns = [int(math.fmod(f / (2 * math.pi), 1.0) * 2.0 ** 64) % 2 ** 64 for f in freq]
        self.turns = torch.tensor([t - 2 ** 64 if t >> 63 else t for t in turns], dtype=torch.int64,
                                  device="cuda" if device is None else device)
        self.axes, self.adjacent, self.factor = bytes(axes), bool(adjacent), float(factor)


def rope_store_kv(pool: KVPool, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, positions: torch.Tensor,
                  out_loc: torch.Tensor, rope: Rope, q_out: Optional[torch.Tensor] = None,
                  q_norm: Optional[torch.Tensor] = None, k_norm: Optional[torch.Tensor] = None, eps: float = 1e-6,
                  status: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """:func:`store_kv` of k and v with k turned by position on the way, and q turned into q_out, which it returns.

    q [T,Hq,D], k and v [T,Hkv,D] may be columns of one tensor (tokens any multiple of 8
    elements apart); ``q_out`` may be q itself.  ``positions`` int32 [T] or [axes, T].  ``q_norm`` and
    ``k_norm`` bf16 [D] norm each head first.  A token with out_loc -1 is none (padding): its row of
    q_out is not written, whatever its other rows hold.
    """
    r = (_native or _binding()).rope_store_kv(pool.k, pool.v, pool.page_size, q, k, v, positions, out_loc, rope.turns,
                                              rope.axes, rope.adjacent, rope.factor, q_out, q_norm, k_norm, eps, status,
                                              _handle(stream))
    if type(r) is int:
        _check(r, "msgl_rope_store_kv")
    return r


class Verified(NamedTuple):
    """The outputs of :func:`verify_drafts` (all int32): keep one and pass it as ``out`` to reuse its buffers."""
    accepted: torch.Tensor     # [B]  drafts that stand
    tokens: torch.Tensor       # [T]  a request's rows: its accepted drafts, the new token, -1
    kv_lens: torch.Tensor      # [B]  tokens whose K/V are kept: the next step's cached_lens


def verify_drafts(target_probs: torch.Tensor, draft_probs: Optional[torch.Tensor], tokens: torch.Tensor,
                  cu_ext: torch.Tensor, accept_u: torch.Tensor, sample_u: torch.Tensor,
                  cached_lens: Optional[torch.Tensor] = None, out: Optional[Verified] = None,
                  status: Optional[torch.Tensor] = None, stream=None) -> Verified:
    """Drafted tokens accepted or replaced by the target's probabilities (msgl_verify_drafts).

    Request b's rows of a step, ``cu_ext[b]`` to ``cu_ext[b+1] - 1``, were fed its last token and its
    drafts (``tokens`` int32 [T]).  ``target_probs`` and ``draft_probs`` float32 or bfloat16 [T, vocab]: row r is the
    distribution that token r + 1 is held against, and was drawn from (``draft_probs`` None: drafts
    that were not drawn at random).  ``accept_u`` [T] and ``sample_u`` [B] are float32 numbers in
    [0, 1).  ``out.kv_lens`` may be ``cached_lens`` itself, which a loop then goes on with.
    """
    a, x, n = (None, None, None) if out is None else out
    r = (_native or _binding()).verify_drafts(target_probs, draft_probs, tokens, cu_ext, accept_u, sample_u, cached_lens,
                                              a, x, n, status, _handle(stream))
    if type(r) is int:
        _check(r, "msgl_verify_drafts")
    return out if r is None else Verified(*r)


class Forked(NamedTuple):
    """The outputs of :func:`fork_requests` (all int32); the first three are arguments of :func:`copy_pages`."""
    src: torch.Tensor          # [N]  page to copy, -1 where none is
    dst: torch.Tensor          # [N]
    tokens: torch.Tensor       # [N]  tokens on it
    pages_taken: torch.Tensor  # [1]  how many places among the free pages were given out (to refused forks too)


def fork_requests(req_table: torch.Tensor, parent_rows: torch.Tensor, child_rows: torch.Tensor, lens: torch.Tensor,
                  free_pages: torch.Tensor, num_slots: int, page_size: int, out: Optional[Forked] = None,
                  status: Optional[torch.Tensor] = None, stream=None) -> Forked:
    """Row ``child_rows[i]`` of ``req_table`` continues the first ``lens[i]`` tokens of row ``parent_rows[i]``.

    Whole pages are shared; a partly filled last one is replaced by a page from the front of
    ``free_pages`` and has to be copied (msgl_fork_requests): ``copy_pages(pools, f.src, f.dst, f.tokens)``.
    """
    s, d, n, t = (None,) * 4 if out is None else out
    r = (_native or _binding()).fork_requests(req_table, parent_rows, child_rows, lens, free_pages, num_slots, page_size,
                                              s, d, n, t, status, _handle(stream))
    if type(r) is int:
        _check(r, "msgl_fork_requests")
    return out if r is None else Forked(*r)


def copy_pages(pools, src: torch.Tensor, dst: torch.Tensor, tokens: Optional[torch.Tensor] = None,
               count: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None, stream=None) -> None:
    """Pages ``src[i]`` to ``dst[i]`` in every pool (a :class:`KVPool` or a sequence of them, one a layer).

    ``tokens`` int32 [N]: only the first of a page's slots; ``count`` int32 [1]: only the first pairs.
    Pairs of -1 are passed over (msgl_copy_pages).
    """
    if isinstance(pools, KVPool):
        pools = (pools,)
    rc = (_native or _binding()).copy_pages(pools, src, dst, tokens, count, status, _handle(stream))
    if rc is not None:
        _check(rc, "msgl_copy_pages")


class FreePages(NamedTuple):
    """The outputs of :func:`free_pages` (int32)."""
    pages: torch.Tensor        # [num_pages]  ids in ascending order, -1 behind them
    num_free: torch.Tensor     # [1]


def page_map_workspace_size(num_slots: int, page_size: int) -> int:
    """Workspace bytes of :func:`free_pages` and :func:`compact_pages`."""
    return int(load().msgl_page_map_workspace_size(num_slots, page_size))


def free_pages(req_table: torch.Tensor, lens: torch.Tensor, num_slots: int, page_size: int,
               req_rows: Optional[torch.Tensor] = None, held: Optional[torch.Tensor] = None,
               out: Optional[FreePages] = None, workspace: Optional[torch.Tensor] = None,
               status: Optional[torch.Tensor] = None, stream=None) -> FreePages:
    """The pages that no request holds (msgl_free_pages): the ``free_pages`` of :func:`step_tables` and
    :func:`fork_requests`.

    Request b holds the pages of its first ``lens[b]`` tokens in row ``req_rows[b]`` (b when
    None; -1: padding).  ``held`` uint8 or bool [num_pages]: pages in use beside them.
    """
    p, c = (None, None) if out is None else out
    r = (_native or _binding()).free_pages(req_table, lens, num_slots, page_size, req_rows, held, p, c, workspace,
                                           status, _handle(stream))
    if type(r) is int:
        _check(r, "msgl_free_pages")
    return out if r is None else FreePages(*r)


class Compaction(NamedTuple):
    """The outputs of :func:`compact_pages` (int32)."""
    page_table: torch.Tensor   # [rows, W]       the requests' rows with the new ids
    remap: torch.Tensor        # [num_pages]     a page's new id, -1 for a free one
    src: torch.Tensor          # [num_pages//2]  the moves, -1 behind them
    dst: torch.Tensor          # [num_pages//2]
    num_moves: torch.Tensor    # [1]
    num_used: torch.Tensor     # [1]             pages in use


def compact_pages(req_table: torch.Tensor, lens: torch.Tensor, num_slots: int, page_size: int,
                  req_rows: Optional[torch.Tensor] = None, held: Optional[torch.Tensor] = None,
                  out: Optional[Compaction] = None, workspace: Optional[torch.Tensor] = None,
                  status: Optional[torch.Tensor] = None, stream=None) -> Compaction:
    """Moves the requests' pages to the front of the pool (msgl_compact_pages).

    The table is rewritten in place unless ``out`` has another; the pages themselves move by
    ``copy_pages(pools, c.src, c.dst, count=c.num_moves)``.  Requests and ``held`` (pages that stay where they
    are) as in :func:`free_pages`.
    """
    t, m, s, d, n, u = (req_table,) + (None,) * 5 if out is None else out
    r = (_native or _binding()).compact_pages(req_table, lens, num_slots, page_size, req_rows, held, t, m, s, d, n, u,
                                              workspace, status, _handle(stream))
    if type(r) is int:
        _check(r, "msgl_compact_pages")
    return out if r is None else Compaction(req_table, *r)


def selftest_wait_timeout(status: torch.Tensor, budget_cycles: int = 10_000_000, stream=None) -> None:
    """Run the bounded-wait self-test; the status word then holds DEVERR_TIMEOUT."""
    rc = load().msgl_selftest_wait_timeout(_ptr(status), int(budget_cycles), _stream(stream))
    _check(rc, "msgl_selftest_wait_timeout")


def read_status(status: torch.Tensor, stream=None) -> int:
    """Synchronise and return the device status word's bits (through the C ABI)."""
    flags = ctypes.c_uint32(0)
    rc = load().msgl_read_status(_ptr(status), ctypes.byref(flags), _stream(stream))
    if rc not in (0, 4, 5):
        _check(rc, "msgl_read_status")
    return int(flags.value)


# ------------------------------------------------------------ metadata checks (host)

def _host_i32(t):
    """A host int32 copy of a tensor (any device) or None, plus its ctypes pointer."""
    if t is None:
        return None, None
    a = t.detach().to("cpu", torch.int32).contiguous()
    return a, ctypes.c_void_p(a.data_ptr())


def check_store_meta(out_loc: torch.Tensor, num_slots: int):
    """Copies out_loc back and checks it: every slot in range, none twice.  Raises MsglError."""
    a, p = _host_i32(out_loc)
    _check(load().msgl_check_store_meta(int(num_slots), p, a.numel()), "msgl_check_store_meta")


def _table(page_table: torch.Tensor):
    a, p = _host_i32(page_table)
    if a.dim() == 1:
        a = a.reshape(1, -1)
    return a, p, int(a.shape[1])


def check_extend_meta(num_slots: int, page_size: int, page_table: torch.Tensor, prefix_lens: torch.Tensor,
                      ext_lens: torch.Tensor, cu_ext: torch.Tensor, positions: Optional[torch.Tensor],
                      max_ext_len: int, max_seq_len: int):
    """Copies an extend step's metadata back and checks it (lengths, positions, pages).  Raises MsglError."""
    pt, ptp, w = _table(page_table)
    pre, prep = _host_i32(prefix_lens)
    ext, extp = _host_i32(ext_lens)
    cu, cup = _host_i32(cu_ext)
    pos, posp = _host_i32(positions)
    if cu.numel() != pre.numel() + 1 or ext.numel() != pre.numel():
        raise ValueError("cu_ext must have num_reqs + 1 entries and ext_lens num_reqs")
    total = int(pos.numel()) if pos is not None else int(cu[-1])
    _check(load().msgl_check_extend_meta(int(num_slots), int(page_size), ptp, w, w, prep, extp, cup, posp,
                                         pre.numel(), total, int(max_ext_len), int(max_seq_len)),
           "msgl_check_extend_meta")


def check_decode_meta(num_slots: int, page_size: int, page_table: torch.Tensor, seq_lens: torch.Tensor,
                      max_seq_len: int):
    """Copies a decode step's metadata back and checks it (lengths, pages).  Raises MsglError."""
    pt, ptp, w = _table(page_table)
    seq, seqp = _host_i32(seq_lens)
    _check(load().msgl_check_decode_meta(int(num_slots), int(page_size), ptp, w, w, seqp, seq.numel(),
                                         int(max_seq_len)), "msgl_check_decode_meta")


def check_step_meta(num_slots: int, page_size: int, req_table: torch.Tensor, req_rows: Optional[torch.Tensor],
                    cached_lens: torch.Tensor, new_lens: Optional[torch.Tensor], free_pages: torch.Tensor,
                    total_tokens: int):
    """Copies a step's request lengths and tables back and checks them (rows, pages, sizes).  Raises MsglError."""
    rt, rtp, w = _table(req_table)
    rows, rowsp = _host_i32(req_rows)
    c, cp = _host_i32(cached_lens)
    n, np_ = _host_i32(new_lens)
    f, fp = _host_i32(free_pages)
    for name, t in (("req_rows", rows), ("new_lens", n)):
        if t is not None and t.numel() != c.numel():
            raise ValueError(f"{name} must have one entry per request")
    _check(load().msgl_check_step_meta(int(num_slots), int(page_size), rtp, rt.numel() // w if w else 0, w, w, rowsp,
                                       cp, np_, c.numel(), fp, f.numel(), int(total_tokens)), "msgl_check_step_meta")


def check_groups_meta(num_slots: int, page_size: int, page_table: torch.Tensor, seq_lens: torch.Tensor,
                      group_start: torch.Tensor, shared_lens: torch.Tensor, max_seq_len: int):
    """Copies a shared-prefix decode's metadata back and checks it (groups, lengths, pages).  Raises MsglError."""
    pt, ptp, w = _table(page_table)
    seq, seqp = _host_i32(seq_lens)
    first, firstp = _host_i32(group_start)
    shared, sharedp = _host_i32(shared_lens)
    if first.numel() != seq.numel() or shared.numel() != seq.numel():
        raise ValueError("group_start and shared_lens must have one entry per request")
    _check(load().msgl_check_groups_meta(int(num_slots), int(page_size), ptp, w, w, firstp, sharedp, seqp, seq.numel(),
                                         int(max_seq_len)), "msgl_check_groups_meta")


def check_fork_meta(num_slots: int, page_size: int, req_table: torch.Tensor, parent_rows: torch.Tensor,
                    child_rows: torch.Tensor, lens: torch.Tensor, free_pages: torch.Tensor):
    """Copies the forks' rows, lengths and tables back and checks them.  Raises MsglError."""
    rt, rtp, w = _table(req_table)
    a, ap = _host_i32(parent_rows)
    b, bp = _host_i32(child_rows)
    n, np_ = _host_i32(lens)
    f, fp = _host_i32(free_pages)
    if b.numel() != a.numel() or n.numel() != a.numel():
        raise ValueError("child_rows and lens must have an entry for each of parent_rows")
    _check(load().msgl_check_fork_meta(int(num_slots), int(page_size), rtp, rt.numel() // w if w else 0, w, w, ap, bp,
                                       np_, a.numel(), fp, f.numel()), "msgl_check_fork_meta")


def check_copy_meta(num_slots: int, page_size: int, src: torch.Tensor, dst: torch.Tensor,
                    tokens: Optional[torch.Tensor] = None):
    """Copies the pairs of pages back and checks them.  Raises MsglError."""
    s, sp = _host_i32(src)
    d, dp = _host_i32(dst)
    n, np_ = _host_i32(tokens)
    if d.numel() != s.numel() or (n is not None and n.numel() != s.numel()):
        raise ValueError("dst and tokens must have an entry for each of src")
    _check(load().msgl_check_copy_meta(int(num_slots), int(page_size), sp, dp, np_, s.numel()), "msgl_check_copy_meta")


def check_held_meta(num_slots: int, page_size: int, req_table: torch.Tensor, lens: torch.Tensor,
                    req_rows: Optional[torch.Tensor] = None):
    """Copies what :func:`free_pages` and :func:`compact_pages` go by back and checks it.  Raises MsglError."""
    rt, rtp, w = _table(req_table)
    n, np_ = _host_i32(lens)
    r, rp = _host_i32(req_rows)
    if r is not None and r.numel() != n.numel():
        raise ValueError("req_rows must have one entry per request")
    _check(load().msgl_check_held_meta(int(num_slots), int(page_size), rtp, rt.numel() // w if w else 0, w, w, rp, np_,
                                       n.numel()), "msgl_check_held_meta")


def check_draft_meta(vocab: int, tokens: torch.Tensor, cu_ext: torch.Tensor, accept_u: torch.Tensor,
                     sample_u: torch.Tensor):
    """Copies a draft batch's tokens, rows and random numbers back and checks them.  Raises MsglError."""
    t, tp = _host_i32(tokens)
    cu, cup = _host_i32(cu_ext)
    a = accept_u.detach().to("cpu", torch.float32).contiguous()
    s = sample_u.detach().to("cpu", torch.float32).contiguous()
    if a.numel() != t.numel() or cu.numel() != s.numel() + 1:
        raise ValueError("accept_u must be [T], and cu_ext [B + 1] for sample_u [B]")
    _check(load().msgl_check_draft_meta(int(vocab), tp, cup, ctypes.c_void_p(a.data_ptr()),
                                        ctypes.c_void_p(s.data_ptr()), s.numel(), t.numel()), "msgl_check_draft_meta")
