"""Gated delta rule on GB300 (sm_103a): a thin Python binding of libgdr.so.

Every function here only marshals arguments into the C ABI declared in
include/gdr.h (same names); all arithmetic runs in the library's CUDA kernels.
PyTorch is used for device memory and streams only.  There is no CPU path:
if the compiled library is missing, every call raises.
"""

from __future__ import annotations

import ctypes
import functools
import os
import threading
from typing import Optional

__all__ = [
    "GdrError", "gdr_dims", "lib", "library_path",
    "gdr_prefill_chunked", "gdr_prefill_workspace_bytes", "gdr_prefill_chunked_static",
    "gdr_prefill_segmented", "gdr_prefill_segmented_workspace_bytes", "gdr_prefill_segments_hint",
    "gdr_decode_step", "gdr_decode_step_overlapped", "gdr_decode_step_gated", "gdr_gated_rmsnorm",
    "gdr_prefill_with_decode",
    "gdr_verify_block", "gdr_verify_commit",
    "gdr_state_snapshot", "gdr_state_restore", "gdr_device_error", "gdr_selftest_wait_timeout", "gdr_status_string",
    "gdr_attn_append", "gdr_attn_prefill", "gdr_attn_decode", "gdr_attn_decode_workspace_bytes",
    "gdr_verify_tree", "gdr_verify_tree_commit",
    "gdr_attn_append_tree", "gdr_attn_decode_tree", "gdr_attn_decode_tree_workspace_bytes", "gdr_attn_commit_tree",
    "gdr_attn_dims", "gdr_rows", "gdr_kv_cache",
    "GDR_F32", "GDR_BF16", "GDR_F16", "GDR_FLAG_QK_L2NORM", "GDR_FLAG_BETA_LOGITS",
]

GDR_OK, GDR_ERR_INVALID_ARG, GDR_ERR_UNSUPPORTED, GDR_ERR_CUDA, GDR_ERR_DEVICE_TIMEOUT = range(5)
GDR_F32, GDR_BF16, GDR_F16 = 0, 1, 2
GDR_FLAG_QK_L2NORM, GDR_FLAG_BETA_LOGITS = 1, 2

_HERE = os.path.dirname(os.path.abspath(__file__))
_lock = threading.Lock()
_lib = None


def library_path() -> str:
    return os.path.join(_HERE, "libgdr.so")


class GdrError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {gdr_status_string(status)}")


class gdr_dims(ctypes.Structure):
    _fields_ = [
        ("h_qk", ctypes.c_int32), ("h_v", ctypes.c_int32),
        ("d_k", ctypes.c_int32), ("d_v", ctypes.c_int32),
        ("chunk", ctypes.c_int32), ("in_dtype", ctypes.c_int32),
        ("out_dtype", ctypes.c_int32), ("scale", ctypes.c_float),
        ("flags", ctypes.c_int32),
    ]


class gdr_attn_dims(ctypes.Structure):
    _fields_ = [
        ("h_q", ctypes.c_int32), ("h_kv", ctypes.c_int32), ("d", ctypes.c_int32),
        ("dtype", ctypes.c_int32), ("scale", ctypes.c_float),
    ]


class gdr_rows(ctypes.Structure):
    _fields_ = [("ptr", ctypes.c_void_p), ("token_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64)]


class gdr_kv_cache(ctypes.Structure):
    _fields_ = [
        ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
        ("page_stride", ctypes.c_int64), ("token_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64),
        ("page_table", ctypes.c_void_p), ("table_stride", ctypes.c_int64),
        ("n_pages", ctypes.c_int32), ("page_size", ctypes.c_int32), ("max_pages", ctypes.c_int32),
    ]


_P = ctypes.c_void_p
_ROWS = ctypes.POINTER(gdr_rows)
_SIGS = {
    "gdr_abi_version": ([], ctypes.c_int32),
    "gdr_status_string": ([ctypes.c_int], ctypes.c_char_p),
    "gdr_prefill_workspace_bytes": ([ctypes.POINTER(gdr_dims), ctypes.c_int32, ctypes.c_int64],
                                    ctypes.c_size_t),
    "gdr_prefill_chunked": ([ctypes.POINTER(gdr_dims), ctypes.c_int32, _P, ctypes.c_int64,
                             _P, _P, _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P], ctypes.c_int),
    "gdr_prefill_chunked_static": ([ctypes.POINTER(gdr_dims), ctypes.c_int32, _P, ctypes.c_int64,
                                    _P, _P, _P, _P, _P, _P, _P, _P], ctypes.c_int),
    "gdr_prefill_static_workspace_capacity": ([], ctypes.c_size_t),
    "gdr_prefill_segmented": ([ctypes.POINTER(gdr_dims), ctypes.c_int32, _P, ctypes.c_int64,
                               _P, _P, _P, _P, _P, _P, _P, ctypes.c_int32, _P, ctypes.c_size_t, _P], ctypes.c_int),
    "gdr_prefill_segmented_workspace_bytes": ([ctypes.POINTER(gdr_dims), ctypes.c_int32, ctypes.c_int64,
                                               ctypes.c_int32], ctypes.c_size_t),
    "gdr_prefill_segments_hint": ([ctypes.POINTER(gdr_dims), ctypes.c_int32, ctypes.c_int64], ctypes.c_int32),
    "gdr_decode_step": ([ctypes.POINTER(gdr_dims), ctypes.c_int32, _P, _P, _P, _P, _P, _P, _P, _P],
                        ctypes.c_int),
    "gdr_decode_step_overlapped": ([ctypes.POINTER(gdr_dims), ctypes.c_int32, _P, _P, _P, _P, _P, _P, _P, _P],
                                   ctypes.c_int),
    "gdr_prefill_with_decode": ([ctypes.POINTER(gdr_dims), ctypes.c_int32, _P, ctypes.c_int64,
                                 _P, _P, _P, _P, _P, _P, _P, _P, ctypes.c_size_t, ctypes.c_int32,
                                 _P, _P, _P, _P, _P, _P, _P, _P], ctypes.c_int),
    "gdr_verify_block": ([ctypes.POINTER(gdr_dims), ctypes.c_int32, ctypes.c_int32,
                          _P, _P, _P, _P, _P, _P, _P, _P, _P, _P], ctypes.c_int),
    "gdr_verify_commit": ([ctypes.POINTER(gdr_dims), ctypes.c_int32, ctypes.c_int32,
                           _P, _P, _P, _P, _P, _P, _P], ctypes.c_int),
    "gdr_decode_step_gated": ([ctypes.POINTER(gdr_dims), ctypes.c_int32, _P, _P, _P, _P, _P, _P, _P, _P,
                               ctypes.c_float, _P, _P], ctypes.c_int),
    "gdr_gated_rmsnorm": ([ctypes.POINTER(gdr_dims), ctypes.c_int64, _P, _P, _P, ctypes.c_float, _P, _P],
                          ctypes.c_int),
    "gdr_state_snapshot": ([ctypes.POINTER(gdr_dims), ctypes.c_int32, _P, _P, _P], ctypes.c_int),
    "gdr_state_restore": ([ctypes.POINTER(gdr_dims), ctypes.c_int32, _P, _P, _P], ctypes.c_int),
    "gdr_attn_append": ([ctypes.POINTER(gdr_attn_dims), ctypes.c_int32, _P, ctypes.c_int64, _ROWS, _ROWS, _ROWS, _ROWS,
                         _ROWS, ctypes.POINTER(gdr_kv_cache), _P, _P, ctypes.c_int32, ctypes.c_int32, _P],
                        ctypes.c_int),
    "gdr_attn_prefill": ([ctypes.POINTER(gdr_attn_dims), ctypes.c_int32, _P, ctypes.c_int64, _ROWS, _ROWS, _ROWS,
                          _ROWS, _P, _P], ctypes.c_int),
    "gdr_attn_decode": ([ctypes.POINTER(gdr_attn_dims), ctypes.c_int32, ctypes.c_int32, _ROWS,
                         ctypes.POINTER(gdr_kv_cache), _P, _ROWS, _P, _P, ctypes.c_size_t, _P], ctypes.c_int),
    "gdr_attn_decode_workspace_bytes": ([ctypes.POINTER(gdr_attn_dims), ctypes.c_int32, ctypes.c_int32],
                                        ctypes.c_size_t),
    "gdr_verify_tree": ([ctypes.POINTER(gdr_dims), ctypes.c_int32, ctypes.c_int32, _P, _P, _P, _P, _P, _P, _P, _P, _P,
                         _P], ctypes.c_int),
    "gdr_verify_tree_commit": ([ctypes.POINTER(gdr_dims), ctypes.c_int32, ctypes.c_int32, _P, _P, _P, _P, _P, _P, _P],
                               ctypes.c_int),
    "gdr_attn_append_tree": ([ctypes.POINTER(gdr_attn_dims), ctypes.c_int32, ctypes.c_int32, _P, _ROWS, _ROWS, _ROWS,
                              _ROWS, _ROWS, ctypes.POINTER(gdr_kv_cache), _P, _P, ctypes.c_int32, ctypes.c_int32, _P],
                             ctypes.c_int),
    "gdr_attn_decode_tree": ([ctypes.POINTER(gdr_attn_dims), ctypes.c_int32, ctypes.c_int32, _P, _ROWS,
                              ctypes.POINTER(gdr_kv_cache), _P, _ROWS, _P, _P, ctypes.c_size_t, _P], ctypes.c_int),
    "gdr_attn_decode_tree_workspace_bytes": ([ctypes.POINTER(gdr_attn_dims), ctypes.c_int32, ctypes.c_int32],
                                             ctypes.c_size_t),
    "gdr_attn_commit_tree": ([ctypes.POINTER(gdr_attn_dims), ctypes.c_int32, ctypes.c_int32, _P, _P, ctypes.c_int32,
                              ctypes.c_int64, ctypes.POINTER(gdr_kv_cache), _P, _P, _P], ctypes.c_int),
    "gdr_device_error": ([_P, ctypes.POINTER(ctypes.c_int32)], ctypes.c_int),
    "gdr_selftest_wait_timeout": ([ctypes.c_int64, _P], ctypes.c_int),
}


def lib():
    """The loaded library (ctypes); raises if it has not been built."""
    global _lib
    with _lock:
        if _lib is None:
            path = library_path()
            if not os.path.exists(path):
                raise ImportError(
                    f"{path} is missing: build it with `python -m gated_deltanet_scan_gb300.build` "
                    "(there is no CPU fallback)")
            handle = ctypes.CDLL(path)
            for name, (argtypes, restype) in _SIGS.items():
                fn = getattr(handle, name)
                fn.argtypes = argtypes
                fn.restype = restype
            _lib = handle
    return _lib


def gdr_status_string(status: int) -> str:
    try:
        return lib().gdr_status_string(int(status)).decode()
    except ImportError:
        return f"gdr_status {status}"


def _check(status: int, where: str) -> None:
    if status != GDR_OK:
        raise GdrError(status, where)


# --- marshalling helpers (torch only for pointers, dtypes and streams) ----------

def _torch():
    import torch
    return torch


def _dtype_code(t) -> int:
    torch = _torch()
    if t.dtype == torch.bfloat16:
        return GDR_BF16
    if t.dtype == torch.float32:
        return GDR_F32
    raise TypeError(f"unsupported dtype {t.dtype}")


def _ptr(t) -> Optional[int]:
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return t.data_ptr()


def _stream_handle(stream, device) -> Optional[int]:
    torch = _torch()
    if stream is None:
        stream = torch.cuda.current_stream(device)
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def flags_of(qk_l2norm: bool = False, beta_logits: bool = False) -> int:
    return (GDR_FLAG_QK_L2NORM if qk_l2norm else 0) | (GDR_FLAG_BETA_LOGITS if beta_logits else 0)


def make_dims(q, v, o, chunk: int = 64, scale: float = 1.0, flags: int = 0) -> gdr_dims:
    """dims from q [T, H_qk, d_k], v [T, H_v, d_v] and o (its dtype is the output type)."""
    return gdr_dims(h_qk=q.shape[-2], h_v=v.shape[-2], d_k=q.shape[-1], d_v=v.shape[-1],
                    chunk=chunk, in_dtype=_dtype_code(q), out_dtype=_dtype_code(o),
                    scale=float(scale), flags=int(flags))


def gdr_prefill_workspace_bytes(q, v, o, n_seqs: int, t_total: int, *, chunk: int = 64,
                                scale: float = 1.0) -> int:
    """Device scratch bytes gdr_prefill_chunked needs (0 on the CUDA-core path)."""
    dims = make_dims(q, v, o, chunk, scale, 0)
    return int(lib().gdr_prefill_workspace_bytes(ctypes.byref(dims), int(n_seqs), int(t_total)))


def gdr_prefill_chunked(q, k, v, g, beta, state, o, cu_seqlens, *, chunk: int = 64,
                        scale: float = 1.0, qk_l2norm: bool = False, beta_logits: bool = False, t_total: Optional[int] = None, workspace=None,
                        stream=None) -> None:
    """Chunked prefill over packed sequences (see gdr_prefill_chunked in include/gdr.h).

    q, k [T, H_qk, d_k]; v [T, H_v, d_v]; g, beta [T, H_v] fp32;
    state [n, H_v, d_k, d_v] fp32 (in/out); o [T, H_v, d_v]; cu_seqlens int32 [n+1]
    on the device.  ``t_total`` defaults to q.shape[0].  ``workspace`` is a
    device tensor of at least gdr_prefill_workspace_bytes(...) bytes; when it is
    None, one is taken from torch's caching allocator for this call, on the
    stream the call runs on (``stream``), so that torch hands its memory to no
    other work before the call's kernels on that stream are done."""
    torch = _torch()
    dims = make_dims(q, v, o, chunk, scale, flags_of(qk_l2norm, beta_logits))
    n = cu_seqlens.shape[0] - 1
    T = q.shape[0] if t_total is None else int(t_total)
    need = int(lib().gdr_prefill_workspace_bytes(ctypes.byref(dims), n, T))
    if workspace is None and need > 0:
        # allocated while the call's stream is current: the caching allocator ties
        # the block to that stream, whatever stream is current in the caller
        s = stream if stream is not None else torch.cuda.current_stream(q.device)
        if isinstance(s, int):
            s = torch.cuda.ExternalStream(s, device=q.device)
        with torch.cuda.stream(s):
            workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    ws_ptr = _ptr(workspace) if workspace is not None else None
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    st = lib().gdr_prefill_chunked(
        ctypes.byref(dims), n, _ptr(cu_seqlens), T, _ptr(q), _ptr(k), _ptr(v), _ptr(g),
        _ptr(beta), _ptr(state), _ptr(o), ws_ptr, ws_bytes, _stream_handle(stream, q.device))
    _check(st, "gdr_prefill_chunked")


def gdr_prefill_chunked_static(q, k, v, g, beta, state, o, cu_seqlens, *, chunk: int = 64,
                               scale: float = 1.0, qk_l2norm: bool = False, beta_logits: bool = False,
                               t_total: Optional[int] = None, stream=None) -> None:
    """gdr_prefill_chunked with the library's fixed scratch array instead of a
    workspace (nothing is allocated; see include/gdr.h for its size limit)."""
    dims = make_dims(q, v, o, chunk, scale, flags_of(qk_l2norm, beta_logits))
    n = cu_seqlens.shape[0] - 1
    T = q.shape[0] if t_total is None else int(t_total)
    st = lib().gdr_prefill_chunked_static(
        ctypes.byref(dims), n, _ptr(cu_seqlens), T, _ptr(q), _ptr(k), _ptr(v), _ptr(g),
        _ptr(beta), _ptr(state), _ptr(o), _stream_handle(stream, q.device))
    _check(st, "gdr_prefill_chunked_static")


def gdr_prefill_segments_hint(q, v, o, n_seqs: int, t_total: int, *, chunk: int = 64, scale: float = 1.0) -> int:
    """Segments the two-level prefill would use on the current device (1: none)."""
    dims = make_dims(q, v, o, chunk, scale, 0)
    return int(lib().gdr_prefill_segments_hint(ctypes.byref(dims), int(n_seqs), int(t_total)))


def gdr_prefill_segmented_workspace_bytes(q, v, o, n_seqs: int, t_total: int, n_segments: int, *,
                                          chunk: int = 64, scale: float = 1.0) -> int:
    dims = make_dims(q, v, o, chunk, scale, 0)
    return int(lib().gdr_prefill_segmented_workspace_bytes(ctypes.byref(dims), int(n_seqs), int(t_total),
                                                           int(n_segments)))


def gdr_prefill_segmented(q, k, v, g, beta, state, o, cu_seqlens, n_segments: Optional[int] = None, *,
                          chunk: int = 64, scale: float = 1.0, qk_l2norm: bool = False, beta_logits: bool = False, t_total: Optional[int] = None, workspace=None,
                          stream=None) -> None:
    """Two-level (segment-parallel) prefill (see gdr_prefill_segmented in
    include/gdr.h): arguments as gdr_prefill_chunked; ``n_segments`` defaults to
    gdr_prefill_segments_hint.  Without ``workspace`` one is taken from torch's
    allocator on the call's stream."""
    torch = _torch()
    dims = make_dims(q, v, o, chunk, scale, flags_of(qk_l2norm, beta_logits))
    n = cu_seqlens.shape[0] - 1
    T = q.shape[0] if t_total is None else int(t_total)
    P = int(lib().gdr_prefill_segments_hint(ctypes.byref(dims), n, T)) if n_segments is None else int(n_segments)
    need = int(lib().gdr_prefill_segmented_workspace_bytes(ctypes.byref(dims), n, T, P))
    if workspace is None and need > 0:
        s = stream if stream is not None else torch.cuda.current_stream(q.device)
        if isinstance(s, int):
            s = torch.cuda.ExternalStream(s, device=q.device)
        with torch.cuda.stream(s):
            workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    ws_ptr = _ptr(workspace) if workspace is not None else None
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    st = lib().gdr_prefill_segmented(
        ctypes.byref(dims), n, _ptr(cu_seqlens), T, _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(state),
        _ptr(o), P, ws_ptr, ws_bytes, _stream_handle(stream, q.device))
    _check(st, "gdr_prefill_segmented")


def gdr_decode_step(q, k, v, g, beta, state, o, *, scale: float = 1.0, qk_l2norm: bool = False,
                    beta_logits: bool = False, stream=None) -> None:
    """One decode step for B sequences: q, k [B, H_qk, d]; v, o [B, H_v, d];
    g, beta [B, H_v]; state [B, H_v, d, d] updated in place."""
    dims = make_dims(q, v, o, 64, scale, flags_of(qk_l2norm, beta_logits))
    st = lib().gdr_decode_step(
        ctypes.byref(dims), q.shape[0], _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta),
        _ptr(state), _ptr(o), _stream_handle(stream, q.device))
    _check(st, "gdr_decode_step")


def gdr_prefill_with_decode(q, k, v, g, beta, state, o, cu_seqlens, dq, dk, dv, dg, dbeta, dstate, d_o, *,
                            scale: float = 1.0, qk_l2norm: bool = False, beta_logits: bool = False,
                            t_total: Optional[int] = None, workspace=None, stream=None) -> None:
    """A prefill (as gdr_prefill_chunked) and one decode step of another batch (as
    gdr_decode_step) in the same chunk-scan launch (see include/gdr.h)."""
    torch = _torch()
    dims = make_dims(q, v, o, 64, scale, flags_of(qk_l2norm, beta_logits))
    n = cu_seqlens.shape[0] - 1
    T = q.shape[0] if t_total is None else int(t_total)
    need = int(lib().gdr_prefill_workspace_bytes(ctypes.byref(dims), n, T))
    if workspace is None and need > 0:
        s = stream if stream is not None else torch.cuda.current_stream(q.device)
        if isinstance(s, int):
            s = torch.cuda.ExternalStream(s, device=q.device)
        with torch.cuda.stream(s):
            workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    ws_ptr = _ptr(workspace) if workspace is not None else None
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    st = lib().gdr_prefill_with_decode(
        ctypes.byref(dims), n, _ptr(cu_seqlens), T, _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(state),
        _ptr(o), ws_ptr, ws_bytes, dq.shape[0], _ptr(dq), _ptr(dk), _ptr(dv), _ptr(dg), _ptr(dbeta), _ptr(dstate),
        _ptr(d_o), _stream_handle(stream, q.device))
    _check(st, "gdr_prefill_with_decode")


def gdr_decode_step_overlapped(q, k, v, g, beta, state, o, *, scale: float = 1.0, qk_l2norm: bool = False,
                               beta_logits: bool = False, stream=None) -> None:
    """gdr_decode_step launched as a programmatic dependent of the kernel before it
    on the stream (see include/gdr.h): none of its inputs or states may be written
    by that kernel."""
    dims = make_dims(q, v, o, 64, scale, flags_of(qk_l2norm, beta_logits))
    st = lib().gdr_decode_step_overlapped(
        ctypes.byref(dims), q.shape[0], _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta),
        _ptr(state), _ptr(o), _stream_handle(stream, q.device))
    _check(st, "gdr_decode_step_overlapped")


RMSNORM_EPS = 1e-6  # the epsilon of the gated RMSNorm after the rule


def gdr_decode_step_gated(q, k, v, g, beta, state, z, weight, y, *, eps: float = RMSNORM_EPS, scale: float = 1.0,
                          qk_l2norm: bool = False, beta_logits: bool = False, stream=None) -> None:
    """gdr_decode_step with the gated RMSNorm fused: y = weight * o / sqrt(mean(o^2) + eps) * silu(z)
    per (sequence, V head) row; z [B, H_v, d] like v, weight [d] fp32, y like the output."""
    dims = make_dims(q, v, y, 64, scale, flags_of(qk_l2norm, beta_logits))
    st = lib().gdr_decode_step_gated(
        ctypes.byref(dims), q.shape[0], _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(state), _ptr(z),
        _ptr(weight), float(eps), _ptr(y), _stream_handle(stream, q.device))
    _check(st, "gdr_decode_step_gated")


def gdr_gated_rmsnorm(o, z, weight, y, *, eps: float = RMSNORM_EPS, stream=None) -> None:
    """y = weight * o / sqrt(mean(o^2) + eps) * silu(z) over the last axis of o [..., d]
    (o and y fp32 or bf16, z fp32 or bf16, weight [d] fp32)."""
    d = o.shape[-1]
    rows = o.numel() // d
    dims = gdr_dims(h_qk=1, h_v=1, d_k=d, d_v=d, chunk=64, in_dtype=_dtype_code(z), out_dtype=_dtype_code(o),
                    scale=1.0, flags=0)
    if y.dtype != o.dtype:
        raise TypeError("y must have o's dtype")
    st = lib().gdr_gated_rmsnorm(ctypes.byref(dims), rows, _ptr(o), _ptr(z), _ptr(weight), float(eps), _ptr(y),
                                 _stream_handle(stream, o.device))
    _check(st, "gdr_gated_rmsnorm")


def gdr_verify_block(q, k, v, g, beta, state, snapshot, o, n_tok: int, *, deltas=None, scale: float = 1.0,
                     qk_l2norm: bool = False, beta_logits: bool = False, stream=None) -> None:
    """n_tok (<= 16) draft tokens per sequence from the current state; the incoming
    state is copied to ``snapshot``.  Token rows are [n_seqs * n_tok, ...].  With
    ``deltas`` (fp32, shaped like v) each token's correction is kept for
    gdr_verify_commit."""
    dims = make_dims(q, v, o, 16, scale, flags_of(qk_l2norm, beta_logits))
    n = state.shape[0]
    st = lib().gdr_verify_block(
        ctypes.byref(dims), n, int(n_tok), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta),
        _ptr(state), _ptr(snapshot), _ptr(o), _ptr(deltas), _stream_handle(stream, state.device))
    _check(st, "gdr_verify_block")


def gdr_verify_commit(k, g, deltas, snapshot, state, accepted, n_tok: int, *, qk_l2norm: bool = False,
                      stream=None) -> None:
    """State after the accepted prefix of a verify block: accepted (int32 device
    tensor [n_seqs]) tokens per sequence, from the block's ``deltas`` and the
    ``snapshot`` it took; writes ``state``."""
    n, hv, dk, dv = state.shape
    dims = gdr_dims(h_qk=k.shape[1], h_v=hv, d_k=dk, d_v=dv, chunk=16,
                    in_dtype=_dtype_code(k), out_dtype=GDR_F32, scale=1.0, flags=flags_of(qk_l2norm))
    st = lib().gdr_verify_commit(
        ctypes.byref(dims), n, int(n_tok), _ptr(accepted), _ptr(k), _ptr(g), _ptr(deltas),
        _ptr(snapshot), _ptr(state), _stream_handle(stream, state.device))
    _check(st, "gdr_verify_commit")


def _state_dims(state) -> gdr_dims:
    _, hv, dk, dv = state.shape
    return gdr_dims(h_qk=hv, h_v=hv, d_k=dk, d_v=dv, chunk=64, in_dtype=GDR_F32,
                    out_dtype=GDR_F32, scale=1.0)


def gdr_state_snapshot(state, snapshot, *, stream=None) -> None:
    dims = _state_dims(state)
    st = lib().gdr_state_snapshot(ctypes.byref(dims), state.shape[0], _ptr(state), _ptr(snapshot),
                                  _stream_handle(stream, state.device))
    _check(st, "gdr_state_snapshot")


def gdr_state_restore(snapshot, state, *, stream=None) -> None:
    dims = _state_dims(state)
    st = lib().gdr_state_restore(ctypes.byref(dims), state.shape[0], _ptr(snapshot), _ptr(state),
                                 _stream_handle(stream, state.device))
    _check(st, "gdr_state_restore")


def gdr_device_error(*, stream=None, device=None) -> int:
    """Synchronise the stream and return (and clear) the device error word."""
    code = ctypes.c_int32(0)
    _check(lib().gdr_device_error(_stream_handle(stream, device), ctypes.byref(code)), "gdr_device_error")
    return int(code.value)


def gdr_selftest_wait_timeout(limit_cycles: int, *, stream=None, device=None) -> None:
    """Launch the self-test block whose bounded wait on a barrier nothing arrives
    on gives up after limit_cycles SM clocks and records GDR_ERR_DEVICE_TIMEOUT."""
    _check(lib().gdr_selftest_wait_timeout(int(limit_cycles), _stream_handle(stream, device)),
           "gdr_selftest_wait_timeout")


# --- softmax attention beside the rule ------------------------------------------
# A decode step's kernels take a few microseconds, so its call must not cost the
# host more: every attribute of a tensor is read once.

# dtype -> code, int32, fp32, the raw current stream of a device index, the current device (None: there is only one,
# and nothing to ask, which would take half a microsecond)
_attn_types = None


def _attn_init():
    global _attn_types
    torch = _torch()
    _attn_types = ({torch.bfloat16: GDR_BF16, torch.float16: GDR_F16, torch.float32: GDR_F32}, torch.int32,
                   torch.float32, getattr(torch._C, "_cuda_getCurrentRawStream", None),
                   torch.cuda.current_device if torch.cuda.device_count() > 1 else None)
    return _attn_types


# Read only; making one takes 0.4 us.  They are kept by value: a scale enters as a float, since a tensor's own key would
# be its identity, whatever it holds by now.
_attn_struct = functools.lru_cache(maxsize=256)(gdr_attn_dims)
_rule_struct = functools.lru_cache(maxsize=256)(gdr_dims)


def _attn_dims(h_q: int, h_kv: int, d: int, dtype, scale) -> gdr_attn_dims:
    code = (_attn_types or _attn_init())[0].get(dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {dtype}")
    return _attn_struct(h_q, h_kv, d, code, d ** -0.5 if scale is None else float(scale))


def _attn_stream(stream, dev: int):
    if dev < 0:
        raise ValueError("tensors must be on a CUDA device")
    if _attn_types[4] is not None and _attn_types[4]() != dev:
        # kernels, streams' default handle and the error word are the current device's
        raise ValueError(f"tensors are on device {dev}, but device {_attn_types[4]()} is current")
    if stream is None:
        raw = _attn_types[3]
        return raw(dev) if raw is not None else _torch().cuda.current_stream(dev).cuda_stream
    return stream if isinstance(stream, int) else stream.cuda_stream


def _rows(t, shape, dtype, dev: int, name: str) -> gdr_rows:
    """Strided rows of t, checked to be of this shape [tokens, heads, d], dtype and device."""
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {shape}, not {tuple(t.shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must have dtype {dtype}")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, not on device {dev}")
    ts, hs, es = t.stride()
    if es != 1:
        raise ValueError(f"{name}'s last dimension must be contiguous")
    # the stride of a dimension of one entry is never used, and may be anything
    return gdr_rows(t.data_ptr(), ts if shape[0] > 1 else 0, hs if shape[1] > 1 else 0)


def _plain(t, shape, dtype, dev: int, name: str) -> int:
    """Address of a contiguous tensor of this shape, dtype and device."""
    if t.dtype != dtype:
        raise TypeError(f"{name} must have dtype {dtype}")
    if t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous tensor of shape {shape}")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, not on device {dev}")
    return t.data_ptr()


def _cache(k_cache, v_cache, page_table, n_seqs: int, heads: int, d: int, dtype, dev: int) -> gdr_kv_cache:
    shape, strides = k_cache.shape, k_cache.stride()
    if len(shape) != 4 or shape[2] != heads or shape[3] != d:
        raise ValueError(f"the caches must have shape (n_pages, page_size, {heads}, {d}), not {tuple(shape)}")
    if v_cache.shape != shape or v_cache.stride() != strides:
        raise ValueError("k_cache and v_cache must have the same shape and strides")
    return _cache_of(shape, strides, k_cache, v_cache, page_table, n_seqs, dtype, dev)


def _cache_of(shape, strides, k_cache, v_cache, page_table, n_seqs: int, dtype, dev: int) -> gdr_kv_cache:
    """A layer's cache of this shape and strides, at the start of k_cache and v_cache."""
    if k_cache.dtype != dtype or v_cache.dtype != dtype:
        raise TypeError(f"the caches must have dtype {dtype}")
    if strides[3] != 1:
        raise ValueError("the caches' last dimension must be contiguous")
    if page_table.dtype != _attn_types[1]:
        raise TypeError("page_table must be int32")
    table = page_table.shape
    if len(table) != 2 or table[0] != n_seqs:
        raise ValueError(f"page_table must have shape ({n_seqs}, max_pages)")
    n, width = table
    rs, cs = page_table.stride()
    if cs != 1 and width > 1:
        raise ValueError("page_table's rows must be contiguous")
    if k_cache.get_device() != dev or v_cache.get_device() != dev or page_table.get_device() != dev:
        raise ValueError(f"the caches and page_table must be on device {dev}")
    n_pages, page = shape[0], shape[1]
    return gdr_kv_cache(k_cache.data_ptr(), v_cache.data_ptr(), strides[0] if n_pages > 1 else 0,
                        strides[1] if page > 1 else 0, strides[2] if shape[2] > 1 else 0, page_table.data_ptr(),
                        rs if n > 1 else 0, n_pages, page, width)


def gdr_attn_append(q, k, v, q_out, k_out, k_cache, v_cache, page_table, kv_lens, inv_freq, cu_seqlens=None, *,
                    interleaved: bool = False, stream=None) -> None:
    """Rotate new queries and keys by their positions and append keys and values to
    the paged cache (see gdr_attn_append in include/gdr.h).

    q, q_out [T, H_q, d] (both may be None); k, v [T, H_kv, d]; k_out like k, k itself
    or None; k_cache, v_cache [n_pages, page_size, H_kv, d] with any strides (a
    head-major cache is passed as cache.transpose(1, 2)); page_table int32 [n, max_pages];
    kv_lens int32 [n], each sequence's tokens including the new ones; inv_freq fp32
    [rot_dim / 2] (None: no rotation); cu_seqlens int32 [n + 1], or None when every
    sequence has T / n new tokens."""
    _append(q, k, v, q_out, k_out, k_cache, v_cache, page_table, kv_lens, inv_freq, cu_seqlens, None, interleaved,
            stream)


def _append(q, k, v, q_out, k_out, k_cache, v_cache, page_table, kv_lens, inv_freq, cu_seqlens, parents, interleaved,
            stream) -> None:
    kv = k.shape
    if len(kv) != 3:
        raise ValueError("k must be [T, H_kv, d]")
    T, h_kv, d = kv
    n, dtype, dev = kv_lens.shape[0], k.dtype, k.get_device()
    qr = qo = ko = None
    h_q = h_kv
    if q is not None and q_out is not None:
        h_q = q.shape[1]
        qs = (T, h_q, d)
        dims = _attn_dims(h_q, h_kv, d, dtype, 1.0)
        qr, qo = _rows(q, qs, dtype, dev, "q"), _rows(q_out, qs, dtype, dev, "q_out")
    elif q is q_out:
        dims = _attn_dims(h_kv, h_kv, d, dtype, 1.0)
    else:
        raise ValueError("q and q_out come together")
    kr, vr = _rows(k, kv, dtype, dev, "k"), _rows(v, kv, dtype, dev, "v")
    if k_out is not None:
        ko = _rows(k_out, kv, dtype, dev, "k_out")
    i32, f32 = _attn_types[1], _attn_types[2]
    half = 0 if inv_freq is None else inv_freq.shape[0]
    if parents is not None:
        n_tok = _tree_rows(parents, n, T)
        tree = _plain(parents, (n, n_tok), i32, dev, "parents")
    elif cu_seqlens is not None:
        cu_seqlens = _plain(cu_seqlens, (n + 1,), i32, dev, "cu_seqlens")
    rest = (qr, kr, vr, qo, ko, _cache(k_cache, v_cache, page_table, n, h_kv, d, dtype, dev),
            _plain(kv_lens, (n,), i32, dev, "kv_lens"),
            _plain(inv_freq, (half,), f32, dev, "inv_freq") if half else None, 2 * half, 1 if interleaved else 0,
            _attn_stream(stream, dev))
    if parents is not None:
        st = (_lib or lib()).gdr_attn_append_tree(dims, n, n_tok, tree, *rest)
    else:
        st = (_lib or lib()).gdr_attn_append(dims, n, cu_seqlens, T, *rest)
    if st != GDR_OK:
        raise GdrError(st, "gdr_attn_append" if parents is None else "gdr_attn_append_tree")


def gdr_attn_prefill(q, k, v, o, cu_seqlens, *, scale: Optional[float] = None, lse=None, stream=None) -> None:
    """Causal attention over whole packed prompts (see gdr_attn_prefill in
    include/gdr.h): q, o [T, H_q, d]; k, v [T, H_kv, d], strided rows; cu_seqlens int32
    [n + 1] on the device; scale defaults to 1 / sqrt(d); lse fp32 [T, H_q] or None."""
    qs, kv = q.shape, k.shape
    if len(qs) != 3 or len(kv) != 3 or qs[0] != kv[0] or qs[2] != kv[2]:
        raise ValueError("q must be [T, H_q, d] and k [T, H_kv, d]")
    T, h_q, d = qs
    dtype, dev = q.dtype, q.get_device()
    dims = _attn_dims(h_q, kv[1], d, dtype, scale)
    n = cu_seqlens.shape[0] - 1
    st = (_lib or lib()).gdr_attn_prefill(
        dims, n, _plain(cu_seqlens, (n + 1,), _attn_types[1], dev, "cu_seqlens"), T, _rows(q, qs, dtype, dev, "q"),
        _rows(k, kv, dtype, dev, "k"), _rows(v, kv, dtype, dev, "v"), _rows(o, qs, dtype, dev, "o"),
        None if lse is None else _plain(lse, (T, h_q), _attn_types[2], dev, "lse"), _attn_stream(stream, dev))
    if st != GDR_OK:
        raise GdrError(st, "gdr_attn_prefill")


def gdr_attn_decode_workspace_bytes(q, k_cache, n_seqs: int, n_tok: int = 1) -> int:
    """Device scratch bytes gdr_attn_decode needs."""
    dims = _attn_dims(q.shape[1], k_cache.shape[2], k_cache.shape[3], q.dtype, None)
    return int(lib().gdr_attn_decode_workspace_bytes(dims, int(n_seqs), int(n_tok)))


def gdr_attn_decode(q, k_cache, v_cache, page_table, kv_lens, o, n_tok: int = 1, *, scale: Optional[float] = None,
                    lse=None, workspace=None, stream=None) -> None:
    """Attention of every sequence's last n_tok (1 .. 16) tokens over its paged cache
    (see gdr_attn_decode in include/gdr.h): q, o [n * n_tok, H_q, d]; caches, page_table
    and kv_lens as for gdr_attn_append; lse fp32 [n * n_tok, H_q] or None.  Without
    ``workspace`` (a device tensor of gdr_attn_decode_workspace_bytes bytes) one is taken
    from torch's allocator on the call's stream."""
    _decode(q, k_cache, v_cache, page_table, kv_lens, o, n_tok, None, scale, lse, workspace, stream)


def _decode(q, k_cache, v_cache, page_table, kv_lens, o, n_tok, parents, scale, lse, workspace, stream) -> None:
    qs = q.shape
    if len(qs) != 3 or k_cache.dim() != 4:
        raise ValueError("q must be [n * n_tok, H_q, d] and the caches [n_pages, page_size, H_kv, d]")
    n, h_q, d = kv_lens.shape[0], qs[1], qs[2]
    if qs[0] != n * n_tok:
        raise ValueError(f"q must have n * n_tok = {n * n_tok} rows, not {qs[0]}")
    h_kv = k_cache.shape[2]
    dtype, dev = q.dtype, q.get_device()
    dims = _attn_dims(h_q, h_kv, d, dtype, scale)
    L = _lib or lib()
    if parents is not None:
        tree = _plain(parents, (n, n_tok), _attn_types[1], dev, "parents")
    if workspace is None:
        torch = _torch()
        size = L.gdr_attn_decode_workspace_bytes if parents is None else L.gdr_attn_decode_tree_workspace_bytes
        need = int(size(dims, n, n_tok))
        if need > 0:
            s = stream if stream is not None else torch.cuda.current_stream(q.device)
            if isinstance(s, int):
                s = torch.cuda.ExternalStream(s, device=q.device)
            with torch.cuda.stream(s):
                workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    elif workspace.get_device() != dev:
        raise ValueError(f"workspace is not on device {dev}")
    rest = (_rows(q, qs, dtype, dev, "q"), _cache(k_cache, v_cache, page_table, n, h_kv, d, dtype, dev),
            _plain(kv_lens, (n,), _attn_types[1], dev, "kv_lens"), _rows(o, qs, dtype, dev, "o"),
            None if lse is None else _plain(lse, (qs[0], h_q), _attn_types[2], dev, "lse"), _ptr(workspace),
            0 if workspace is None else workspace.nbytes, _attn_stream(stream, dev))
    if parents is None:
        st = L.gdr_attn_decode(dims, n, n_tok, *rest)
    else:
        st = L.gdr_attn_decode_tree(dims, n, n_tok, tree, *rest)
    if st != GDR_OK:
        raise GdrError(st, "gdr_attn_decode" if parents is None else "gdr_attn_decode_tree")


# --- trees of drafted tokens ------------------------------------------------------

def _tree_rows(parents, n: int, rows: Optional[int]) -> int:
    """Rows of each of n trees; ``rows`` is what the tensors have, if any."""
    shape = parents.shape
    if len(shape) != 2 or shape[0] != n:
        raise ValueError(f"parents must have shape ({n}, n_tok)")
    n_tok = shape[1]
    if rows is not None and rows != n * n_tok:
        raise ValueError(f"the tensors must have n * n_tok = {n * n_tok} rows, not {rows}")
    return n_tok


def gdr_attn_append_tree(q, k, v, q_out, k_out, k_cache, v_cache, page_table, kv_lens, inv_freq, parents, *,
                         interleaved: bool = False, stream=None) -> None:
    """gdr_attn_append for trees of drafted tokens (see gdr_attn_append_tree in
    include/gdr.h): parents int32 [n, n_tok], tensors of n * n_tok rows; a node's
    position is its path's, its slot its row's; rows that are no nodes are written nowhere."""
    if parents is None:
        raise ValueError("parents must be an int32 tensor [n, n_tok]")
    _append(q, k, v, q_out, k_out, k_cache, v_cache, page_table, kv_lens, inv_freq, None, parents, interleaved, stream)


def gdr_attn_decode_tree_workspace_bytes(q, k_cache, parents) -> int:
    """Device scratch bytes gdr_attn_decode_tree needs for these shapes (see include/gdr.h): fewer tokens may need
    more, so a buffer kept for trees of several sizes has the largest of their bytes."""
    dims = _attn_dims(q.shape[1], k_cache.shape[2], k_cache.shape[3], q.dtype, None)
    return int(lib().gdr_attn_decode_tree_workspace_bytes(dims, *parents.shape))


def gdr_attn_decode_tree(q, k_cache, v_cache, page_table, kv_lens, o, parents, *, scale: Optional[float] = None,
                         lse=None, workspace=None, stream=None) -> None:
    """Attention of every sequence's tree of up to 64 drafted tokens over its paged cache
    (see gdr_attn_decode_tree in include/gdr.h): parents int32 [n, n_tok]; everything else as
    for gdr_attn_decode, the workspace of gdr_attn_decode_tree_workspace_bytes bytes."""
    n_tok = _tree_rows(parents, kv_lens.shape[0], q.shape[0])
    _decode(q, k_cache, v_cache, page_table, kv_lens, o, n_tok, parents, scale, lse, workspace, stream)


def gdr_attn_commit_tree(k_cache, v_cache, page_table, kv_lens, parents, last, lens_out=None, *, stream=None) -> None:
    """Move every tree's accepted path, which ends in node ``last`` (int32 [n], -1: none), to
    the front of the tree's slots (see gdr_attn_commit_tree in include/gdr.h).  k_cache,
    v_cache [n_pages, page_size, H_kv, d], or [layers, n_pages, page_size, H_kv, d] for all
    layers at once; lens_out int32 [n] (not kv_lens or last itself) receives the new lengths."""
    shape, strides = k_cache.shape, k_cache.stride()
    if len(shape) == 4:
        layers, stride = 1, 0
    elif len(shape) == 5:
        layers, stride = shape[0], strides[0] if shape[0] > 1 else 0
        if layers == 0:
            if lens_out is not None:
                raise ValueError("without layers there is nothing that gives lens_out")
            return
        shape, strides = shape[1:], strides[1:]
    else:
        raise ValueError("the caches must be [n_pages, page_size, H_kv, d] or [layers, n_pages, page_size, H_kv, d]")
    if v_cache.shape != k_cache.shape or v_cache.stride() != k_cache.stride():
        raise ValueError("k_cache and v_cache must have the same shape and strides")
    h_kv, d = shape[2], shape[3]
    dtype, dev = k_cache.dtype, k_cache.get_device()
    dims = _attn_dims(h_kv, h_kv, d, dtype, 1.0)
    i32, n = _attn_types[1], kv_lens.shape[0]
    n_tok = _tree_rows(parents, n, None)
    st = (_lib or lib()).gdr_attn_commit_tree(
        dims, n, n_tok, _plain(parents, (n, n_tok), i32, dev, "parents"), _plain(last, (n,), i32, dev, "last"), layers,
        stride, _cache_of(shape, strides, k_cache, v_cache, page_table, n, dtype, dev),
        _plain(kv_lens, (n,), i32, dev, "kv_lens"),
        None if lens_out is None else _plain(lens_out, (n,), i32, dev, "lens_out"), _attn_stream(stream, dev))
    if st != GDR_OK:
        raise GdrError(st, "gdr_attn_commit_tree")


def _tree_dims(h_qk: int, h_v: int, d_k: int, d_v: int, dtype, out_dtype, scale, flags: int) -> gdr_dims:
    codes = (_attn_types or _attn_init())[0]
    io, out = codes.get(dtype), codes.get(out_dtype)
    if io in (None, GDR_F16) or out in (None, GDR_F16):
        raise TypeError(f"unsupported dtypes {dtype} and {out_dtype}")
    return _rule_struct(h_qk, h_v, d_k, d_v, 64, io, out, float(scale), flags)


def gdr_verify_tree(q, k, v, g, beta, state, o, parents, *, deltas=None, scale: float = 1.0, qk_l2norm: bool = False,
                    beta_logits: bool = False, stream=None) -> None:
    """The rule along every path of each sequence's tree of up to 64 drafted tokens, from its
    state, which stays as it is (see gdr_verify_tree in include/gdr.h).  parents int32
    [n, n_tok]; q, k [n * n_tok, H_qk, d]; v, o [n * n_tok, H_v, d]; g, beta [n * n_tok, H_v]
    fp32; state [n, H_v, d, d] fp32; ``deltas`` (fp32, shaped like v) receives the corrections
    that gdr_verify_tree_commit takes."""
    qs, vs, ss = q.shape, v.shape, state.shape
    if len(qs) != 3 or len(vs) != 3 or len(ss) != 4:
        raise ValueError("q must be [T, H_qk, d], v [T, H_v, d] and state [n, H_v, d, d]")
    (T, h_qk, d), hv, n = qs, vs[1], ss[0]
    dims = _tree_dims(h_qk, hv, d, vs[2], q.dtype, o.dtype, scale, flags_of(qk_l2norm, beta_logits))
    dev = q.get_device()
    types = _attn_types
    n_tok = _tree_rows(parents, n, T)
    f32 = types[2]
    st = (_lib or lib()).gdr_verify_tree(
        dims, n, n_tok, _plain(parents, (n, n_tok), types[1], dev, "parents"), _plain(q, qs, q.dtype, dev, "q"),
        _plain(k, qs, q.dtype, dev, "k"), _plain(v, (T, hv, d), q.dtype, dev, "v"), _plain(g, (T, hv), f32, dev, "g"),
        _plain(beta, (T, hv), f32, dev, "beta"), _plain(state, (n, hv, d, d), f32, dev, "state"),
        _plain(o, (T, hv, d), o.dtype, dev, "o"),
        None if deltas is None else _plain(deltas, (T, hv, d), f32, dev, "deltas"), _attn_stream(stream, dev))
    if st != GDR_OK:
        raise GdrError(st, "gdr_verify_tree")


def gdr_verify_tree_commit(k, g, deltas, state, parents, last, *, qk_l2norm: bool = False, stream=None) -> None:
    """Move every state to its tree's last accepted node, in place (see
    gdr_verify_tree_commit in include/gdr.h): ``last`` int32 [n], -1 for none; k, g and deltas
    as gdr_verify_tree took and wrote them."""
    if k.dim() != 3 or state.dim() != 4:
        raise ValueError("k must be [T, H_qk, d] and state [n, H_v, d, d]")
    n, hv, d, _ = state.shape
    T, h_qk, _ = ks = k.shape
    dims = _tree_dims(h_qk, hv, d, d, k.dtype, state.dtype, 1.0, flags_of(qk_l2norm))
    dev = state.get_device()
    n_tok = _tree_rows(parents, n, T)
    i32, f32 = _attn_types[1], _attn_types[2]
    if ks[2] != d:
        raise ValueError(f"k must have shape {(T, h_qk, d)}")
    st = (_lib or lib()).gdr_verify_tree_commit(
        dims, n, n_tok, _plain(parents, (n, n_tok), i32, dev, "parents"), _plain(last, (n,), i32, dev, "last"),
        _plain(k, ks, k.dtype, dev, "k"), _plain(g, (T, hv), f32, dev, "g"),
        _plain(deltas, (T, hv, d), f32, dev, "deltas"), _plain(state, (n, hv, d, d), f32, dev, "state"),
        _attn_stream(stream, dev))
    if st != GDR_OK:
        raise GdrError(st, "gdr_verify_tree_commit")
