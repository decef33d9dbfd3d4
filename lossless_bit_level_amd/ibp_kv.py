"""Thin binding of libibp_kv and libibp_kv_long (include/ibp_kv.h,
include/ibp_kv_long.h), same names as the C ABI: an 8-bit KV page cache, the
attention that reads it, and eviction of its pages by accumulated attention
weight; for long and shared contexts appends with rotated positions, outlines
and selection of pages, and attention over a shared prefix.

Argument marshalling only; every step runs in the HIP kernels of
libibp_kv.so and libibp_kv_long.so.  The structures, lib() and long_lib() are
ctypes; the calls take torch tensors through a small extension module
(csrc/ibp_kv_torch.cpp), since a decoding step makes many short ones: it checks
the arguments, allocates results and calls the C ABI.  If one of them has not
been built its calls raise (all do without libibp_kv.so or the module); there is
no fallback.

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
_LONG_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libibp_kv_long.so")

IBP_KV_BF16 = 0
IBP_KV_FP16 = 1


class IBPKVError(RuntimeError):
    def __init__(self, fn: str, status: int):
        msg = f"{fn}: {status_string(status)} ({status})"
        if status == IBP_ERR_HIP:
            last = long_lib().ibp_kv_long_last_hip_error if fn in _LONG else lib().ibp_kv_last_hip_error
            msg += f", hipError {last()}"
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


class ibp_kv_rotation(ctypes.Structure):
    """Tables of a rotation (see include/ibp_kv_long.h)."""
    _fields_ = [("n_positions", ctypes.c_uint64),
                ("rotary_dim", ctypes.c_uint32),
                ("interleaved", ctypes.c_uint32),
                ("cos", ctypes.c_void_p),
                ("sin", ctypes.c_void_p),
                ("positions", ctypes.c_void_p)]


class ibp_kv_outlines(ctypes.Structure):
    """What bounds the keys of each page (see include/ibp_kv_long.h)."""
    _fields_ = [("codes", ctypes.c_void_p),
                ("scales", ctypes.c_void_p)]


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


_long_lib = None
_LONG = ("ibp_kv_append_rotated", "ibp_kv_outline", "ibp_kv_select", "ibp_kv_attention_shared")


def long_lib() -> ctypes.CDLL:
    """Load libibp_kv_long.so (built in-tree by lossless_bit_level_amd.build)."""
    global _long_lib
    if _long_lib is None:
        if not os.path.exists(_LONG_LIB_PATH):
            raise RuntimeError(f"{_LONG_LIB_PATH} is missing: build it with "
                               "`python -m lossless_bit_level_amd.build`")
        L = ctypes.CDLL(_LONG_LIB_PATH)
        vp, u64, u32, i32 = ctypes.c_void_p, ctypes.c_uint64, ctypes.c_uint32, ctypes.c_int
        cache, table = ctypes.POINTER(ibp_kv_cache), ctypes.POINTER(ibp_kv_table)
        tensor, outlines = ctypes.POINTER(ibp_kv_tensor), ctypes.POINTER(ibp_kv_outlines)
        L.ibp_kv_append_rotated.argtypes = [cache, table, u32, u64, tensor, tensor, vp,
                                            ctypes.POINTER(ibp_kv_rotation), u64, tensor, tensor,
                                            outlines, vp]
        L.ibp_kv_outline.argtypes = [cache, outlines, table, u64, vp, vp]
        L.ibp_kv_select_workspace_bytes.argtypes = [cache, table]
        L.ibp_kv_select.argtypes = [cache, outlines, table, u32, u64, u64, tensor, vp, u64, u64, u64,
                                    vp, vp, vp, vp, u64, vp]
        L.ibp_kv_attention_shared_workspace_bytes.argtypes = [cache, table, table, u64, u64]
        L.ibp_kv_attention_shared.argtypes = [cache, table, table, u32, u64, u64, tensor, tensor, vp,
                                              ctypes.c_float, vp, u64, vp]
        L.ibp_kv_long_last_hip_error.argtypes = []
        for f in (*_LONG, "ibp_kv_long_last_hip_error"):
            getattr(L, f).restype = i32
        for f in ("ibp_kv_select_workspace_bytes", "ibp_kv_attention_shared_workspace_bytes"):
            getattr(L, f).restype = u64
        _long_lib = L
    return _long_lib


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
        if os.path.exists(_LONG_LIB_PATH):  # without it its calls raise, and the others work
            _ibp_kv.load_long(_LONG_LIB_PATH)
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


def ibp_kv_append_rotated(cache: ibp_kv_cache, pages: torch.Tensor, lengths: torch.Tensor,
                          k: torch.Tensor, v: torch.Tensor, cos: torch.Tensor, sin: torch.Tensor,
                          positions: torch.Tensor | None = None, q: torch.Tensor | None = None,
                          q_out: torch.Tensor | None = None, counts: torch.Tensor | None = None,
                          interleaved: bool = False,
                          outlines: tuple[torch.Tensor, torch.Tensor] | None = None, stream=None):
    """ibp_kv_append of keys whose positions are rotated on the way.  cos, sin:
    float32 [n_positions, rotary_dim / 2]; pairs are dims i and i +
    rotary_dim / 2 or, interleaved, 2 i and 2 i + 1.  positions: int32
    [n_seqs, n_new] (default: the tokens' places in their rows, which count
    no prefix that other tables hold).  With q
    ([n_seqs, n_new, q_heads, head_dim], the type of k) the queries are rotated
    too, into q_out (default: a new tensor; q itself is allowed), which is
    returned.  outlines: (int8 [n_pages, 2, head_dim], float32 [n_pages]),
    brought up to date for the pages that receive tokens.  Asynchronous on the
    current stream of the tensors' GPU, or on stream=."""
    if stream is not None:
        with _on(stream, pages):
            return ibp_kv_append_rotated(cache, pages, lengths, k, v, cos, sin, positions, q, q_out,
                                         counts, interleaved, outlines)
    codes, scales = outlines if outlines is not None else (None, None)
    status, out = _ext().append_rotated(cache, pages, lengths, k, v, cos, sin, positions, q, q_out,
                                        counts, interleaved, codes, scales, _stream(pages))
    _check("ibp_kv_append_rotated", status)
    return out


def ibp_kv_outline(cache: ibp_kv_cache, outlines: tuple[torch.Tensor, torch.Tensor],
                   pages: torch.Tensor, lengths: torch.Tensor, n_new: int | None = None,
                   counts: torch.Tensor | None = None, stream=None):
    """Outlines (int8 [n_pages, 2, head_dim], float32 [n_pages]) of the pages
    that hold the rows' last tokens: n_new of them or, with counts (int32
    [n_seqs]), each sequence's own number up to n_new; by default of all pages
    that hold tokens.  Rows that name the same page must hold the same number
    of its tokens.  Asynchronous on the current stream of the tensors' GPU,
    or on stream=."""
    if stream is not None:
        with _on(stream, pages):
            return ibp_kv_outline(cache, outlines, pages, lengths, n_new, counts)
    _check("ibp_kv_outline",
           _ext().outline(cache, *outlines, pages, lengths, n_new, counts, _stream(pages)))


def ibp_kv_select_workspace_bytes(cache: ibp_kv_cache, pages: torch.Tensor,
                                  lengths: torch.Tensor) -> int:
    table = ibp_kv_table(*pages.shape, pages.data_ptr(), lengths.data_ptr())
    return int(long_lib().ibp_kv_select_workspace_bytes(cache, table))


def ibp_kv_select(cache: ibp_kv_cache, outlines: tuple[torch.Tensor, torch.Tensor],
                  pages: torch.Tensor, lengths: torch.Tensor, q: torch.Tensor, keep_pages: int,
                  sink_pages: int = 1, recent_pages: int = 1, counts: torch.Tensor | None = None,
                  pages_out: torch.Tensor | None = None, lengths_out: torch.Tensor | None = None,
                  places_out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                  stream=None):
    """For each row the pages that its new tokens' queries q ([n_seqs, n_new,
    q_heads, head_dim]) are to attend over: the first sink_pages, the last
    recent_pages (which must cover the new tokens) and, of those between, the
    ones whose outlines promise the largest scores, keep_pages at most.  Returns
    (pages, lengths, places): int32 [n_seqs, kv_heads, keep_pages] ids in table
    order, -1 past the kept ones; the tokens of the kept pages; and the pages'
    places in the row's table.  The first two are a table for
    ibp_kv_attention.  workspace: a uint8 GPU tensor of at least
    ibp_kv_select_workspace_bytes (default: allocated).  Asynchronous on the
    current stream of the tensors' GPU, or on stream=."""
    if stream is not None:
        with _on(stream, pages):
            return ibp_kv_select(cache, outlines, pages, lengths, q, keep_pages, sink_pages,
                                 recent_pages, counts, pages_out, lengths_out, places_out, workspace)
    status, *out = _ext().select(cache, *outlines, pages, lengths, q, keep_pages, sink_pages,
                                 recent_pages, counts, pages_out, lengths_out, places_out, workspace,
                                 _stream(pages))
    _check("ibp_kv_select", status)
    return tuple(out)


def ibp_kv_attention_shared_workspace_bytes(cache: ibp_kv_cache, prefix_pages: torch.Tensor,
                                            prefix_lengths: torch.Tensor, pages: torch.Tensor,
                                            lengths: torch.Tensor, q_heads: int, n_new: int) -> int:
    prefix = ibp_kv_table(1, *prefix_pages.shape, prefix_pages.data_ptr(), prefix_lengths.data_ptr())
    table = ibp_kv_table(*pages.shape, pages.data_ptr(), lengths.data_ptr())
    with torch.cuda.device_of(pages):
        return int(long_lib().ibp_kv_attention_shared_workspace_bytes(cache, prefix, table, q_heads, n_new))


def ibp_kv_attention_shared(cache: ibp_kv_cache, prefix_pages: torch.Tensor,
                            prefix_lengths: torch.Tensor, pages: torch.Tensor,
                            lengths: torch.Tensor, q: torch.Tensor, scale: float | None = None,
                            counts: torch.Tensor | None = None, out: torch.Tensor | None = None,
                            workspace: torch.Tensor | None = None, stream=None):
    """ibp_kv_attention of sequences that begin with the same tokens, those of
    prefix_pages (int32 [kv_heads, max_prefix_pages]) and prefix_lengths (int32
    [kv_heads]), which are read once for all of them; pages and lengths are the
    sequences' own, without these.  workspace: a uint8 GPU tensor of at least
    ibp_kv_attention_shared_workspace_bytes (default: allocated).  Returns out.
    Asynchronous on the current stream of the tensors' GPU, or on stream=."""
    if stream is not None:  # what the call allocates is the stream's too
        with _on(stream, pages):
            return ibp_kv_attention_shared(cache, prefix_pages, prefix_lengths, pages, lengths, q,
                                           scale, counts, out, workspace)
    status, out = _ext().attention_shared(cache, prefix_pages, prefix_lengths, pages, lengths, q,
                                          scale, counts, out, workspace, _stream(q))
    _check("ibp_kv_attention_shared", status)
    return out
