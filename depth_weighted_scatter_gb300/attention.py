"""Thin ctypes binding of libbevpool's token operators (include/bevpool.h):
head norms with rotary positions, the plan of a batch's pages, the append to a
paged key/value cache, and attention of new tokens over that cache.

The functions named like the C entry points only marshal arguments.  The
tensor-level helpers (``qk_norm_rope``, ``qk_norm_rope_backward``,
``plan_pages``, ``kv_append``, ``paged_attention`` and the last two's forms for a
cache with page scales, ``..._scaled``) go through the native module
``_token_ops``, which checks shapes and types, allocates outputs and workspaces
with PyTorch and names the stream.  Every step of the computation runs in the
library's CUDA kernels; there is no CPU fallback.  Importing this module raises
if the library or ``_token_ops`` has not been built.

Head tensors are [tokens, heads, head_dim], fp16 or bf16, with any token and
head strides that are multiples of 8 elements (a slice of a fused projection
is taken as it is).  A cache is [n_pages, n_k_heads, page_size, head_dim] (or
a permuted view of [n_pages, page_size, n_k_heads, head_dim] memory), of the
heads' type, or E4M3 codes (torch.float8_e4m3fn or uint8); its strides are
multiples of 16 bytes, so E4M3 rows start 16 elements apart or a multiple of it.
"""
from __future__ import annotations

import contextlib
import ctypes
from typing import NamedTuple, Optional

import torch

from .bevpool import BEVPOOL_OK, BevpoolError, _lib
from . import _token_ops as _ops

BEVPOOL_BF16 = 3

_i32, _i64, _sz, _vp, _f32 = ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t, ctypes.c_void_p, ctypes.c_float
_dt = ctypes.c_int
_rows = [_vp, _i64, _i64]
_rotary = [_vp, _i32, _vp, _i32, _vp, _i32]                 # positions, n_axes, sections, rotary_dim, inv_freq, interleaved
_pages = [_i64, _i64, _i64, _i32, _i32, _vp, _i32, _vp, _vp, _i32]
_scaled_pages = _pages[:3] + [_vp, _vp] + _pages[3:]        # with k_scales, v_scales

_lib.bevpool_qk_norm_rope.argtypes = ([_dt] + _rows * 2 + [_i32] * 4 + [_vp, _vp, _f32] + _rotary + _rows * 2 + [_vp])
_lib.bevpool_qk_norm_rope.restype = ctypes.c_int
_lib.bevpool_qk_norm_rope_backward_workspace_size.argtypes = [_i32] * 4
_lib.bevpool_qk_norm_rope_backward_workspace_size.restype = _sz
_lib.bevpool_qk_norm_rope_backward.argtypes = ([_dt] + _rows * 4 + [_i32] * 4 + [_vp, _vp, _f32] + _rotary + _rows * 2
                                               + [_vp, _vp, _vp, _sz, _vp])
_lib.bevpool_qk_norm_rope_backward.restype = ctypes.c_int
_lib.bevpool_kv_append.argtypes = ([_dt, _dt] + _rows * 3 + [_i32] * 4 + [_vp, _vp, _f32] + _rotary + _rows
                                   + [_vp, _vp] + _pages + [_f32, _f32, _vp])
_lib.bevpool_kv_append.restype = ctypes.c_int
_lib.bevpool_kv_append_scaled.argtypes = ([_dt] + _rows * 3 + [_i32] * 4 + [_vp, _vp, _f32] + _rotary + _rows + [_vp, _vp]
                                          + _scaled_pages + [_vp])
_lib.bevpool_kv_append_scaled.restype = ctypes.c_int
_lib.bevpool_paged_attention_workspace_size.argtypes = [_i32] * 8
_lib.bevpool_paged_attention_workspace_size.restype = _sz
_lib.bevpool_paged_attention.argtypes = ([_dt, _dt] + _rows + [_vp, _vp] + _pages + [_i32] * 6
                                         + [_f32, _i32, _i32, _f32, _f32] + _rows + [_vp, _vp, _sz, _vp])
_lib.bevpool_paged_attention.restype = ctypes.c_int
_lib.bevpool_paged_attention_scaled_workspace_size.argtypes = [_i32] * 8
_lib.bevpool_paged_attention_scaled_workspace_size.restype = _sz
_lib.bevpool_paged_attention_scaled.argtypes = ([_dt] + _rows + [_vp, _vp] + _scaled_pages + [_i32] * 6 + [_f32, _i32, _i32]
                                                + _rows + [_vp, _vp, _sz, _vp])
_lib.bevpool_paged_attention_scaled.restype = ctypes.c_int
_lib.bevpool_plan_pages.argtypes = [_vp] * 7 + [_i32] * 5 + [_vp] * 10
_lib.bevpool_plan_pages.restype = ctypes.c_int
_lib.bevpool_attention_timeouts.argtypes = [_vp]
_lib.bevpool_attention_timeouts.restype = ctypes.c_int


# ---------------------------------------------------------------- raw C entry points (arguments as in the header)

def bevpool_qk_norm_rope(*args) -> int:
    return _lib.bevpool_qk_norm_rope(*args)


def bevpool_qk_norm_rope_backward_workspace_size(n_tokens: int, n_q_heads: int, n_k_heads: int, head_dim: int) -> int:
    return _lib.bevpool_qk_norm_rope_backward_workspace_size(n_tokens, n_q_heads, n_k_heads, head_dim)


def bevpool_qk_norm_rope_backward(*args) -> int:
    return _lib.bevpool_qk_norm_rope_backward(*args)


def bevpool_kv_append(*args) -> int:
    return _lib.bevpool_kv_append(*args)


def bevpool_kv_append_scaled(*args) -> int:
    return _lib.bevpool_kv_append_scaled(*args)


def bevpool_paged_attention_workspace_size(n_seqs: int, n_tokens: int, n_q_heads: int, n_k_heads: int, head_dim: int,
                                           max_q_len: int, max_kv_len: int, window: int) -> int:
    return _lib.bevpool_paged_attention_workspace_size(n_seqs, n_tokens, n_q_heads, n_k_heads, head_dim, max_q_len,
                                                       max_kv_len, window)


def bevpool_paged_attention(*args) -> int:
    return _lib.bevpool_paged_attention(*args)


def bevpool_paged_attention_scaled_workspace_size(n_seqs: int, n_tokens: int, n_q_heads: int, n_k_heads: int, head_dim: int,
                                                  max_q_len: int, max_kv_len: int, window: int) -> int:
    return _lib.bevpool_paged_attention_scaled_workspace_size(n_seqs, n_tokens, n_q_heads, n_k_heads, head_dim, max_q_len,
                                                              max_kv_len, window)


def bevpool_paged_attention_scaled(*args) -> int:
    return _lib.bevpool_paged_attention_scaled(*args)


def bevpool_plan_pages(*args) -> int:
    return _lib.bevpool_plan_pages(*args)


def bevpool_attention_timeouts() -> int:
    """Bounded waits of the attention kernels that ran out so far (0 unless the device misbehaves); synchronises."""
    n = _i64(0)
    st = _lib.bevpool_attention_timeouts(ctypes.byref(n))
    if st != BEVPOOL_OK:
        raise BevpoolError(st, "bevpool_attention_timeouts")
    return n.value


# ---------------------------------------------------------------- tensor helpers (checks, allocations: _token_ops)

_ops.set_error(BevpoolError)


def _stream_of(stream):
    return torch.cuda.stream(stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(int(stream)))


# Each helper takes `stream` (a torch stream or a cudaStream_t; None: torch's
# current one).  Another stream is made torch's current stream for the call, so
# that what the helper allocates belongs to the stream that uses it.  A
# `workspace` is a contiguous tensor on the current device, 256-byte aligned, of
# the bytes that the C entry point's ..._workspace_size names, or more.
#
# The helpers do not take part in autograd: a tensor that requires gradients (with
# grad mode on) or carries a forward-mode tangent is refused.  Training calls
# qk_norm_rope_backward.

def qk_norm_rope(q, k, positions, inv_freq, *, sections=None, q_weight=None, k_weight=None, eps: float = 1e-6,
                 interleaved: bool = False, q_out=None, k_out=None, stream=None):
    """bevpool_qk_norm_rope: norms of q and k for each head (where the weight is
    given) and their rotary positions.  positions int32 [tokens] or [tokens,
    axes]; inv_freq float32 [rotary_dim / 2]; sections: pairs of each axis.
    Returns (q_out, k_out); q_out=q, k_out=k works in place."""
    if stream is not None:
        with _stream_of(stream):
            return _ops.qk_norm_rope(q, k, q_weight, k_weight, q_out, k_out, eps, positions, inv_freq, sections, interleaved)
    return _ops.qk_norm_rope(q, k, q_weight, k_weight, q_out, k_out, eps, positions, inv_freq, sections, interleaved)


def qk_norm_rope_backward(dq_out, dk_out, q, k, positions, inv_freq, *, sections=None, q_weight=None, k_weight=None,
                          eps: float = 1e-6, interleaved: bool = False, dq=None, dk=None, workspace=None, stream=None):
    """bevpool_qk_norm_rope_backward: gradients of qk_norm_rope's inputs and
    weights from those of its outputs.  Returns (dq, dk, dq_weight, dk_weight);
    a weight that is None has the gradient None."""
    with contextlib.nullcontext() if stream is None else _stream_of(stream):
        return _ops.qk_norm_rope_backward(dq_out, dk_out, q, k, q_weight, k_weight, dq, dk, workspace, eps, positions, inv_freq,
                                          sections, interleaved)


def kv_append(k, v, k_cache, v_cache, block_table, kv_len, cu_q, positions, inv_freq, *, sections=None, k_weight=None,
              eps: float = 1e-6, interleaved: bool = False, k_scale: float = 1.0, v_scale: float = 1.0, q=None,
              q_weight=None, q_out=None, stream=None):
    """bevpool_kv_append: the keys (normed where k_weight is given, and turned)
    and values of new tokens into the paged cache; with q, its norm and rotation
    too.  kv_len counts the new tokens.  Returns q_out (None without q)."""
    if stream is not None:
        with _stream_of(stream):
            return _ops.kv_append(k, v, q, k_weight, q_weight, q_out, k_scale, v_scale, k_cache, v_cache, block_table, kv_len,
                                  cu_q, eps, positions, inv_freq, sections, interleaved)
    return _ops.kv_append(k, v, q, k_weight, q_weight, q_out, k_scale, v_scale, k_cache, v_cache, block_table, kv_len, cu_q,
                          eps, positions, inv_freq, sections, interleaved)


def kv_append_scaled(k, v, k_cache, v_cache, k_scales, v_scales, block_table, kv_len, cu_q, positions, inv_freq, *,
                     sections=None, k_weight=None, eps: float = 1e-6, interleaved: bool = False, q=None, q_weight=None,
                     q_out=None, stream=None):
    """bevpool_kv_append_scaled: kv_append to a cache of E4M3 codes with a scale
    for each page and key head (k_scales, v_scales: float32 [n_pages,
    n_k_heads]), worked out from what a page gets.  Returns q_out (None without
    q)."""
    if stream is not None:
        with _stream_of(stream):
            return _ops.kv_append_scaled(k, v, q, k_weight, q_weight, q_out, k_scales, v_scales, k_cache, v_cache, block_table,
                                         kv_len, cu_q, eps, positions, inv_freq, sections, interleaved)
    return _ops.kv_append_scaled(k, v, q, k_weight, q_weight, q_out, k_scales, v_scales, k_cache, v_cache, block_table, kv_len,
                                 cu_q, eps, positions, inv_freq, sections, interleaved)


def paged_attention(q, k_cache, v_cache, block_table, kv_len, cu_q, *, max_q_len: int, max_kv_len: int,
                    scale: Optional[float] = None, causal: bool = True, window: int = 0, k_scale: float = 1.0,
                    v_scale: float = 1.0, out=None, return_lse: bool = False, workspace=None, stream=None):
    """bevpool_paged_attention: new tokens (rows cu_q[b] .. cu_q[b+1]-1 of q are
    request b's) over the paged cache.  scale defaults to head_dim ** -0.5;
    max_q_len and max_kv_len are host bounds of the requests' lengths.  Returns
    out, or (out, lse) with return_lse.  Rows of q outside every request keep
    what `out` held."""
    if stream is not None:
        with _stream_of(stream):
            return _ops.paged_attention(q, workspace, k_cache, v_cache, block_table, kv_len, cu_q, max_q_len, max_kv_len, scale,
                                        causal, window, k_scale, v_scale, out, return_lse)
    return _ops.paged_attention(q, workspace, k_cache, v_cache, block_table, kv_len, cu_q, max_q_len, max_kv_len, scale, causal,
                                window, k_scale, v_scale, out, return_lse)


def paged_attention_scaled(q, k_cache, v_cache, k_scales, v_scales, block_table, kv_len, cu_q, *, max_q_len: int, max_kv_len: int,
                           scale: Optional[float] = None, causal: bool = True, window: int = 0, out=None,
                           return_lse: bool = False, workspace=None, stream=None):
    """bevpool_paged_attention_scaled: paged_attention over a cache of E4M3 codes
    with a scale for each page and key head (k_scales, v_scales: float32 [n_pages,
    n_k_heads]), as kv_append_scaled makes it."""
    if stream is not None:
        with _stream_of(stream):
            return _ops.paged_attention_scaled(q, workspace, k_scales, v_scales, k_cache, v_cache, block_table, kv_len, cu_q,
                                               max_q_len, max_kv_len, scale, causal, window, out, return_lse)
    return _ops.paged_attention_scaled(q, workspace, k_scales, v_scales, k_cache, v_cache, block_table, kv_len, cu_q, max_q_len,
                                       max_kv_len, scale, causal, window, out, return_lse)


class PagePlan(NamedTuple):
    """What plan_pages returns; kv_len, first, block_table, free_pages and n_free are the next call's state."""

    cu_q: torch.Tensor          # int32 [n_seqs + 1]
    positions: torch.Tensor     # int32 [n_tokens]
    slots: torch.Tensor         # int64 [n_tokens]
    kv_len: torch.Tensor        # int32 [n_seqs]
    first: torch.Tensor         # int32 [n_seqs]
    block_table: torch.Tensor   # int32 [n_seqs, pages]
    free_pages: torch.Tensor    # int32 [n_pool]
    n_free: torch.Tensor        # int32 [1]
    missing: torch.Tensor       # int32 [1]: 0 unless the batch does not fit


def plan_pages(q_len, kv_len, first, block_table, free_pages, n_free, *, page_size: int, n_tokens: int, drop=None,
               out: Optional[PagePlan] = None, stream=None) -> PagePlan:
    """bevpool_plan_pages: pages given back and handed out for q_len new tokens a
    request, on the device: cu_q, kv_len and block_table as kv_append and
    paged_attention take them, each new token's position and slot.  All tensors
    int32 (slots int64); n_tokens is a host bound of the new tokens; drop: oldest
    pages that a request gives back first, negative: it ends.  Pages that requests
    share are not for planning: each request would give them back.  With missing !=
    0 nothing has changed and cu_q is 0 throughout: an append with it puts nothing
    into the cache, an attention computes no rows, so a program looks at it before
    it uses them.  `out`: an earlier plan's tensors to write to, none of which this
    call reads."""
    if stream is not None:
        with _stream_of(stream):
            return PagePlan._make(_ops.plan_pages(q_len, kv_len, first, drop, block_table, free_pages, n_free, page_size, n_tokens, out))
    return PagePlan._make(_ops.plan_pages(q_len, kv_len, first, drop, block_table, free_pages, n_free, page_size, n_tokens, out))
