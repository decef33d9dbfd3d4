"""Thin binding of libibp_kv (include/ibp_kv.h), same names as the C ABI: an
8-bit KV page cache, the attention that reads it, and eviction of its pages by
accumulated attention weight.

Argument marshalling only; every step runs in the HIP kernels of
libibp_kv.so.  The structures and lib() are ctypes; the calls take torch
tensors through a small extension module (csrc/ibp_kv_torch.cpp), since a
decoding step makes many short ones: it checks the arguments, allocates
results and calls the C ABI.  If either has not been built this module raises
on first use; there is no fallback.

No call has a gradient.  Codes and scales carry none; going backward through a
result of inputs that require one raises, and a given output with such inputs
is refused.
"""
from __future__ import annotations

import ctypes
import os

import torch

from .ibp import (IBP_ERR_HIP, IBP_ERR_INVALID_ARGUMENT, IBP_ERR_LAYOUT,  # noqa: F401
                  IBP_ERR_UNSUPPORTED, IBP_OK)

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libibp_kv.so")

IBP_KV_BF16 = 0
IBP_KV_FP16 = 1


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
        _ext().set_cache(self, k_codes, k_scales, v_codes, v_scales, page_tokens, head_dim)
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


_module = None


def _ext():
    """The extension module (built in-tree by lossless_bit_level_amd.build)."""
    global _module
    if _module is None:
        lib()
        try:
            from . import _ibp_kv
        except ImportError as e:
            raise RuntimeError("_ibp_kv.so is missing or does not load: build it with "
                               f"`python -m lossless_bit_level_amd.build` ({e})") from e
        _module = _ibp_kv
    return _module


def status_string(status: int) -> str:
    return lib().ibp_kv_status_string(status).decode()


def _check(fn: str, status: int):
    if status != IBP_OK:
        raise IBPKVError(fn, status)


def _stream(t: torch.Tensor) -> int:
    """The current stream of t's device (a CPU tensor is refused later on)."""
    return torch._C._cuda_getCurrentRawStream(t.get_device()) if t.is_cuda else 0


def _on(stream, t: torch.Tensor):
    """stream= as the current stream, for a call on t's GPU."""
    if t.is_cuda and stream.device != t.device:
        raise ValueError(f"stream of another GPU: {stream.device}, tensors on {t.device}")
    return torch.cuda.stream(stream)


def ibp_kv_append(cache: ibp_kv_cache, pages: torch.Tensor, lengths: torch.Tensor,
                  k: torch.Tensor, v: torch.Tensor, counts: torch.Tensor | None = None,
                  stream=None):
    """Append the tokens of k and v ([n_seqs, n_new, kv_heads, head_dim],
    bfloat16 or float16, any strides of the leading axes) to the pages of
    their rows.  pages: int32 [n_seqs, kv_heads, max_pages]; lengths: int32
    [n_seqs, kv_heads], the new tokens counted in; counts: int32 [n_seqs], how
    many of the n_new tokens each sequence brings (default: all).
    Asynchronous on the current stream of the tensors' GPU, or on stream=."""
    if stream is not None:
        with _on(stream, pages):
            return ibp_kv_append(cache, pages, lengths, k, v, counts)
    _check("ibp_kv_append",
           _ext().append(cache, pages, lengths, k, v, counts, _stream(pages)))


def ibp_kv_attention_workspace_bytes(cache: ibp_kv_cache, pages: torch.Tensor,
                                     lengths: torch.Tensor, q_heads: int, n_new: int,
                                     with_weights: bool) -> int:
    table = ibp_kv_table(*pages.shape, pages.data_ptr(), lengths.data_ptr())
    with torch.cuda.device_of(pages):
        return int(lib().ibp_kv_attention_workspace_bytes(cache, table, q_heads, n_new,
                                                          int(with_weights)))


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
    current stream of the tensors' GPU, or on stream=."""
    if stream is not None:  # what the call allocates is the stream's too
        with _on(stream, pages):
            return ibp_kv_attention(cache, pages, lengths, q, scale, weights, weights_out, counts,
                                    out, workspace)
    status, out, weights_out = _ext().attention(cache, pages, lengths, q, scale, weights,
                                                weights_out, counts, out, workspace, _stream(q))
    _check("ibp_kv_attention", status)
    return out, weights_out


def ibp_kv_evict(pages: torch.Tensor, weights: torch.Tensor, lengths: torch.Tensor,
                 page_tokens: int, keep_pages: int, sink_pages: int = 1, recent_pages: int = 1,
                 pages_out: torch.Tensor | None = None, weights_out: torch.Tensor | None = None,
                 lengths_out: torch.Tensor | None = None, stream=None):
    """Cut every row to keep_pages pages: the first sink_pages, the last
    recent_pages and the heaviest between.  Returns (pages, weights, lengths)
    with the kept pages first, the evicted ones after them (weight 0) and the
    row's other entries as they were.  The outputs must not overlap the
    inputs.  Asynchronous on the current stream of the tensors' GPU, or on
    stream=."""
    if stream is not None:
        with _on(stream, pages):
            return ibp_kv_evict(pages, weights, lengths, page_tokens, keep_pages, sink_pages,
                                recent_pages, pages_out, weights_out, lengths_out)
    status, *out = _ext().evict(pages, weights, lengths, page_tokens, keep_pages, sink_pages,
                                recent_pages, pages_out, weights_out, lengths_out, _stream(pages))
    _check("ibp_kv_evict", status)
    return tuple(out)
