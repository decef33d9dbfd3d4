"""Thin ctypes binding of libibp_kv (include/ibp_kv.h), same names as the C
ABI: an 8-bit KV page cache, the attention that reads it, and eviction of its
pages by accumulated attention weight.

Argument marshalling only; every step runs in the HIP kernels of
libibp_kv.so.  If the library has not been built this module raises on first
use; there is no fallback.
"""
from __future__ import annotations

import ctypes
import math
import os

import torch

from .ibp import (IBP_ERR_HIP, IBP_ERR_INVALID_ARGUMENT, IBP_ERR_LAYOUT,  # noqa: F401
                  IBP_ERR_UNSUPPORTED, IBP_OK)

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libibp_kv.so")

IBP_KV_BF16 = 0
IBP_KV_FP16 = 1
_DTYPES = {torch.bfloat16: IBP_KV_BF16, torch.float16: IBP_KV_FP16}


class IBPKVError(RuntimeError):
    def __init__(self, fn: str, status: int):
        msg = f"{fn}: {status_string(status)} ({status})"
        if status == IBP_ERR_HIP:
            msg += f", hipError {lib().ibp_kv_last_hip_error()}"
        super().__init__(msg)
        self.status = status


class ibp_kv_table(ctypes.Structure):
    """Which pages hold which head of which sequence (see include/ibp_kv.h)."""
    _fields_ = [("n_seqs", ctypes.c_uint64),
                ("kv_heads", ctypes.c_uint64),
                ("max_pages", ctypes.c_uint64),
                ("pages", ctypes.c_void_p),
                ("lengths", ctypes.c_void_p)]


class ibp_kv_tensor(ctypes.Structure):
    """A strided 16-bit tensor [n_seqs][n_new][heads][head_dim]."""
    _fields_ = [("data", ctypes.c_void_p),
                ("seq_stride", ctypes.c_int64),
                ("token_stride", ctypes.c_int64),
                ("head_stride", ctypes.c_int64)]


class ibp_kv_cache(ctypes.Structure):
    """The pool of pages: k_codes and v_codes are uint8 GPU tensors of
    n_pages rows of page_tokens * head_dim bytes, k_scales and v_scales
    float32 [n_pages].  Holds on to the tensors."""
    _fields_ = [("n_pages", ctypes.c_uint64),
                ("page_tokens", ctypes.c_uint32),
                ("head_dim", ctypes.c_uint32),
                ("k_codes", ctypes.c_void_p),
                ("k_scales", ctypes.c_void_p),
                ("v_codes", ctypes.c_void_p),
                ("v_scales", ctypes.c_void_p)]

    def __init__(self, k_codes: torch.Tensor, k_scales: torch.Tensor, v_codes: torch.Tensor,
                 v_scales: torch.Tensor, page_tokens: int, head_dim: int):
        _need(k_codes, torch.uint8, "k_codes")
        _need(k_scales, torch.float32, "k_scales")
        _need(v_codes, torch.uint8, "v_codes")
        _need(v_scales, torch.float32, "v_scales")
        n = k_scales.numel()
        if not k_codes.numel() == v_codes.numel() == n * page_tokens * head_dim or v_scales.numel() != n:
            raise ValueError(f"{n} pages of {page_tokens} x {head_dim} codes and as many scales expected, "
                             "for keys and for values")
        super().__init__(n, page_tokens, head_dim, k_codes.data_ptr(), k_scales.data_ptr(),
                         v_codes.data_ptr(), v_scales.data_ptr())
        self.tensors = (k_codes, k_scales, v_codes, v_scales)


_lib = None


def lib() -> ctypes.CDLL:
    """Load libibp_kv.so (built in-tree by lossless_bit_level_amd.build)."""
    global _lib
    if _lib is None:
        if not os.path.exists(_LIB_PATH):
            raise RuntimeError(f"{_LIB_PATH} is missing: build it with "
                               "`python -m lossless_bit_level_amd.build`")
        L = ctypes.CDLL(_LIB_PATH)
        vp, u64, u32, i32 = ctypes.c_void_p, ctypes.c_uint64, ctypes.c_uint32, ctypes.c_int
        cache, table = ctypes.POINTER(ibp_kv_cache), ctypes.POINTER(ibp_kv_table)
        tensor = ctypes.POINTER(ibp_kv_tensor)
        L.ibp_kv_append.argtypes = [cache, table, u32, u64, tensor, tensor, vp, vp]
        L.ibp_kv_attention_workspace_bytes.argtypes = [cache, table, u64, u64, i32]
        L.ibp_kv_attention_workspace_bytes.restype = u64
        L.ibp_kv_attention.argtypes = [cache, table, u32, u64, u64, tensor, tensor, vp,
                                       ctypes.c_float, vp, vp, vp, u64, vp]
        L.ibp_kv_evict.argtypes = [table, u32, u64, u64, u64, vp, vp, vp, vp, vp]
        L.ibp_kv_status_string.argtypes = [i32]
        L.ibp_kv_status_string.restype = ctypes.c_char_p
        L.ibp_kv_last_hip_error.argtypes = []
        for f in ("ibp_kv_append", "ibp_kv_attention", "ibp_kv_evict", "ibp_kv_last_hip_error"):
            getattr(L, f).restype = i32
        _lib = L
    return _lib


def status_string(status: int) -> str:
    return lib().ibp_kv_status_string(status).decode()


def _check(fn: str, status: int):
    if status != IBP_OK:
        raise IBPKVError(fn, status)


def _stream(t: torch.Tensor) -> int:
    """The current stream of t's device."""
    return torch._C._cuda_getCurrentRawStream(t.device.index)


def _need(t: torch.Tensor, dtype: torch.dtype, name: str, shape=None):
    """Contiguous GPU tensors only: the kernels take their addresses as they
    are (a CPU pointer there would fault the GPU)."""
    if not t.is_cuda or t.dtype is not dtype or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} GPU tensor")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must have the shape {tuple(shape)}")


def _table(pages: torch.Tensor, lengths: torch.Tensor) -> ibp_kv_table:
    if pages.dim() != 3:
        raise ValueError("pages must be [n_seqs, kv_heads, max_pages]")
    _need(pages, torch.int32, "pages")
    _need(lengths, torch.int32, "lengths", pages.shape[:2])
    n_seqs, heads, max_pages = pages.shape
    return ibp_kv_table(n_seqs, heads, max_pages, pages.data_ptr(), lengths.data_ptr())


def _tensor(t: torch.Tensor, name: str, dtype, shape) -> ibp_kv_tensor:
    """Strides of the leading axes are free, the head axis is contiguous."""
    if not t.is_cuda or t.dtype is not dtype or t.shape != shape:
        raise ValueError(f"{name} must be a {dtype} GPU tensor of shape {tuple(shape)}")
    s = t.stride()
    if s[3] != 1:
        raise ValueError(f"the last axis of {name} must be contiguous")
    return ibp_kv_tensor(t.data_ptr(), s[0], s[1], s[2])


def _new_dtype(t: torch.Tensor, name: str) -> int:
    dtype = _DTYPES.get(t.dtype)
    if dtype is None or t.dim() != 4:
        raise ValueError(f"{name} must be a bfloat16 or float16 tensor "
                         "[n_seqs, n_new, heads, head_dim]")
    return dtype


def _counts(counts, n_seqs: int):
    if counts is None:
        return None
    _need(counts, torch.int32, "counts", (n_seqs,))
    return counts.data_ptr()


def ibp_kv_append(cache: ibp_kv_cache, pages: torch.Tensor, lengths: torch.Tensor,
                  k: torch.Tensor, v: torch.Tensor, counts: torch.Tensor | None = None,
                  stream=None):
    """Append the tokens of k and v ([n_seqs, n_new, kv_heads, head_dim],
    bfloat16 or float16, any strides of the leading axes) to the pages of
    their rows.  pages: int32 [n_seqs, kv_heads, max_pages]; lengths: int32
    [n_seqs, kv_heads], the new tokens counted in; counts: int32 [n_seqs], how
    many of the n_new tokens each sequence brings (default: all).
    Asynchronous on the current stream, or on stream=."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return ibp_kv_append(cache, pages, lengths, k, v, counts)
    dtype = _new_dtype(k, "k")
    table = _table(pages, lengths)
    shape = (table.n_seqs, k.shape[1], table.kv_heads, cache.head_dim)
    kt, vt = _tensor(k, "k", k.dtype, shape), _tensor(v, "v", k.dtype, shape)
    _check("ibp_kv_append",
           lib().ibp_kv_append(cache, table, dtype, k.shape[1], kt, vt,
                               _counts(counts, table.n_seqs), _stream(pages)))


def ibp_kv_attention_workspace_bytes(cache: ibp_kv_cache, pages: torch.Tensor,
                                     lengths: torch.Tensor, q_heads: int, n_new: int,
                                     with_weights: bool) -> int:
    return int(lib().ibp_kv_attention_workspace_bytes(cache, _table(pages, lengths), q_heads,
                                                      n_new, int(with_weights)))


def ibp_kv_attention(cache: ibp_kv_cache, pages: torch.Tensor, lengths: torch.Tensor,
                     q: torch.Tensor, scale: float | None = None,
                     weights: torch.Tensor | None = None,
                     weights_out: torch.Tensor | None = None,
                     counts: torch.Tensor | None = None, out: torch.Tensor | None = None,
                     workspace: torch.Tensor | None = None, stream=None):
    """Attention of the new tokens' queries q ([n_seqs, n_new, q_heads,
    head_dim], bfloat16 or float16) over the rows' pages, causal among the new
    tokens; scale defaults to head_dim ** -0.5.  With weights (float32
    [n_seqs, kv_heads, max_pages]) weights_out = weights + the attention
    weight each page received; it may be weights itself and defaults to a new
    tensor.  workspace: a uint8 GPU tensor of at least
    ibp_kv_attention_workspace_bytes (default: allocated).  Returns
    (out, weights_out), the second None without weights.  Asynchronous on the
    current stream, or on stream=."""
    if stream is not None:  # what the call allocates is the stream's too
        with torch.cuda.stream(stream):
            return ibp_kv_attention(cache, pages, lengths, q, scale, weights, weights_out, counts,
                                    out, workspace)
    dtype = _new_dtype(q, "q")
    table = _table(pages, lengths)
    n_new, q_heads = q.shape[1], q.shape[2]
    if table.kv_heads and (q_heads == 0 or q_heads % table.kv_heads):
        raise ValueError("q_heads must be a multiple of kv_heads")
    shape = (table.n_seqs, n_new, q_heads, cache.head_dim)
    qt = _tensor(q, "q", q.dtype, shape)
    if out is None:
        out = torch.empty_like(q, memory_format=torch.contiguous_format)
        ot = ibp_kv_tensor(out.data_ptr(), *out.stride()[:3])
    else:
        ot = _tensor(out, "out", q.dtype, shape)
    w = wo = None
    if weights is not None:
        _need(weights, torch.float32, "weights", pages.shape)
        if weights_out is None:
            weights_out = torch.empty_like(weights)
        else:
            _need(weights_out, torch.float32, "weights_out", pages.shape)
        w, wo = weights.data_ptr(), weights_out.data_ptr()
    elif weights_out is not None:
        raise ValueError("weights_out without weights")
    L = lib()
    if workspace is None:
        n = L.ibp_kv_attention_workspace_bytes(cache, table, q_heads, n_new, w is not None)
        if n:
            workspace = torch.empty(n, dtype=torch.uint8, device=q.device)
    else:
        _need(workspace, torch.uint8, "workspace")
    ws, ws_bytes = (None, 0) if workspace is None else (workspace.data_ptr(), workspace.numel())
    _check("ibp_kv_attention",
           L.ibp_kv_attention(cache, table, dtype, q_heads, n_new, qt, ot,
                              _counts(counts, table.n_seqs),
                              1.0 / math.sqrt(cache.head_dim) if scale is None else scale,
                              w, wo, ws, ws_bytes, _stream(q)))
    return out, weights_out


def ibp_kv_evict(pages: torch.Tensor, weights: torch.Tensor, lengths: torch.Tensor,
                 page_tokens: int, keep_pages: int, sink_pages: int = 1, recent_pages: int = 1,
                 pages_out: torch.Tensor | None = None, weights_out: torch.Tensor | None = None,
                 lengths_out: torch.Tensor | None = None, stream=None):
    """Cut every row to keep_pages pages: the first sink_pages, the last
    recent_pages and the heaviest between.  Returns (pages, weights, lengths)
    with the kept pages first, the evicted ones after them (weight 0) and the
    row's other entries as they were.  The outputs must not overlap the
    inputs.  Asynchronous on the current stream, or on stream=."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return ibp_kv_evict(pages, weights, lengths, page_tokens, keep_pages, sink_pages,
                                recent_pages, pages_out, weights_out, lengths_out)
    table = _table(pages, lengths)
    _need(weights, torch.float32, "weights", pages.shape)
    if pages_out is None:
        pages_out = torch.empty_like(pages)
    else:
        _need(pages_out, torch.int32, "pages_out", pages.shape)
    if weights_out is None:
        weights_out = torch.empty_like(weights)
    else:
        _need(weights_out, torch.float32, "weights_out", pages.shape)
    if lengths_out is None:
        lengths_out = torch.empty_like(lengths)
    else:
        _need(lengths_out, torch.int32, "lengths_out", lengths.shape)
    _check("ibp_kv_evict",
           lib().ibp_kv_evict(table, page_tokens, keep_pages, sink_pages, recent_pages,
                              weights.data_ptr(), pages_out.data_ptr(), weights_out.data_ptr(),
                              lengths_out.data_ptr(), _stream(pages)))
    return pages_out, weights_out, lengths_out
