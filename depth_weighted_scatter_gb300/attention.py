"""Thin ctypes binding of libbevpool's token operators (include/bevpool.h):
head norms with rotary positions, the append to a paged key/value cache, and
attention of new tokens over that cache.

The functions named like the C entry points only marshal arguments; the
tensor-level helpers (``qk_norm_rope``, ``qk_norm_rope_backward``,
``kv_append``, ``paged_attention``) check shapes and types, allocate outputs
and workspaces with PyTorch and name the stream.  Every step of the
computation runs in the library's CUDA kernels; there is no CPU fallback.

Head tensors are [tokens, heads, head_dim], fp16 or bf16, with any token and
head strides that are multiples of 8 elements (a slice of a fused projection
is taken as it is).  A cache is [n_pages, n_k_heads, page_size, head_dim] (or
a permuted view of [n_pages, page_size, n_k_heads, head_dim] memory), of the
heads' type, or E4M3 codes (torch.float8_e4m3fn or uint8).
"""
from __future__ import annotations

import ctypes
import functools
from typing import Optional, Sequence

import torch

from .bevpool import (BEVPOOL_E4M3, BEVPOOL_ERR_INVALID_ARG, BEVPOOL_ERR_UNSUPPORTED, BEVPOOL_F16, BEVPOOL_OK,
                      BevpoolError, _lib)

BEVPOOL_BF16 = 3
MAX_AXES = 4

_i32, _i64, _sz, _vp, _f32 = ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t, ctypes.c_void_p, ctypes.c_float
_dt = ctypes.c_int
_rows = [_vp, _i64, _i64]
_rotary = [_vp, _i32, _vp, _i32, _vp, _i32]                 # positions, n_axes, sections, rotary_dim, inv_freq, interleaved
_pages = [_i64, _i64, _i64, _i32, _i32, _vp, _i32, _vp, _vp, _i32]

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
_lib.bevpool_paged_attention_workspace_size.argtypes = [_i32] * 8
_lib.bevpool_paged_attention_workspace_size.restype = _sz
_lib.bevpool_paged_attention.argtypes = ([_dt, _dt] + _rows + [_vp, _vp] + _pages + [_i32] * 6
                                         + [_f32, _i32, _i32, _f32, _f32] + _rows + [_vp, _vp, _sz, _vp])
_lib.bevpool_paged_attention.restype = ctypes.c_int
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


def bevpool_paged_attention_workspace_size(n_seqs: int, n_tokens: int, n_q_heads: int, n_k_heads: int, head_dim: int,
                                           max_q_len: int, max_kv_len: int, window: int) -> int:
    return _lib.bevpool_paged_attention_workspace_size(n_seqs, n_tokens, n_q_heads, n_k_heads, head_dim, max_q_len,
                                                       max_kv_len, window)


def bevpool_paged_attention(*args) -> int:
    return _lib.bevpool_paged_attention(*args)


def bevpool_attention_timeouts() -> int:
    """Bounded waits of the attention kernels that ran out so far (0 unless the device misbehaves); synchronises."""
    n = _i64(0)
    st = _lib.bevpool_attention_timeouts(ctypes.byref(n))
    if st != BEVPOOL_OK:
        raise BevpoolError(st, "bevpool_attention_timeouts")
    return n.value


# ---------------------------------------------------------------- tensor helpers

_DTYPES = {torch.float16: BEVPOOL_F16, torch.bfloat16: BEVPOOL_BF16}
_CACHE_DTYPES = {torch.float16: BEVPOOL_F16, torch.bfloat16: BEVPOOL_BF16, torch.float8_e4m3fn: BEVPOOL_E4M3,
                 torch.uint8: BEVPOOL_E4M3}
_F32, _I32 = torch.float32, torch.int32

# A decoding step calls these helpers for every layer, so they keep to a few
# cheap tensor attributes each: device indexes instead of device objects, the
# raw stream instead of a Stream object, one message built only on refusal.


def _refuse(what: str, status: int = BEVPOOL_ERR_INVALID_ARG):
    raise BevpoolError(status, what)


def _heads(name: str, t, shape, dtype, dev: int) -> tuple:
    """(pointer, token stride, head stride) of a [tokens, heads, head_dim] tensor of this shape, type and device."""
    if t.shape != shape or t.dtype != dtype or t.get_device() != dev:
        _refuse(f"{name}: a {dtype} tensor of shape {tuple(shape)} on CUDA device {dev} is wanted, got {t.dtype} "
                f"{tuple(t.shape)} on {t.device}")
    ts, hs, es = t.stride()
    if es != 1:
        _refuse(f"{name}: the last axis must be contiguous")
    # the stride of an axis of one entry is never used
    return t.data_ptr(), ts if shape[0] > 1 else 0, hs if shape[1] > 1 else 0


def _check_first(name: str, t) -> tuple:
    """(shape, type, library type, device index) of the tensor that the others are checked against."""
    if t.dim() != 3:
        _refuse(f"{name}: a [tokens, heads, head_dim] tensor is wanted")
    dtype, dev = t.dtype, t.get_device()
    code = _DTYPES.get(dtype)
    if code is None:
        _refuse(f"{name}: fp16 or bf16 is wanted, got {dtype}", BEVPOOL_ERR_UNSUPPORTED)
    if dev < 0 or dev != torch._C._cuda_getDevice():
        _refuse(f"{name}: tensors must be on the current CUDA device")
    return t.shape, dtype, code, dev


def _vector(name: str, t, n: int, dtype, dev: int):
    if t is None:
        return None
    if t.dtype != dtype or t.get_device() != dev or t.numel() != n or not t.is_contiguous():
        _refuse(f"{name}: a contiguous {dtype} tensor of {n} entries on CUDA device {dev} is wanted")
    return t.data_ptr()


@functools.lru_cache(maxsize=64)
def _sections(sections: tuple):
    return (_i32 * len(sections))(*sections)


def _position_args(T: int, dev: int, positions, inv_freq, sections: Optional[Sequence[int]], interleaved: bool) -> tuple:
    shape = positions.shape
    n_axes = shape[1] if len(shape) == 2 else 1
    if not 1 <= len(shape) <= 2 or shape[0] != T or not 1 <= n_axes <= MAX_AXES:
        _refuse(f"positions: int32 [tokens] or [tokens, axes <= {MAX_AXES}] is wanted")
    n = inv_freq.numel()
    sec = (n,) if sections is None else tuple(sections)
    if len(sec) != n_axes:
        _refuse("sections: one entry an axis is wanted")
    return (_vector("positions", positions, T * n_axes, _I32, dev), n_axes, _sections(sec), 2 * n,
            _vector("inv_freq", inv_freq, n, _F32, dev), 1 if interleaved else 0)


def _cache_args(k_cache, v_cache, block_table, kv_len, cu_q, dev: int, n_k_heads: Optional[int], D: int) -> tuple:
    """(cache type, pointers, page arguments); n_k_heads None: whatever the cache has."""
    shape, dtype, strides = k_cache.shape, k_cache.dtype, k_cache.stride()
    if len(shape) != 4 or v_cache.shape != shape or v_cache.dtype != dtype or v_cache.stride() != strides:
        _refuse("caches: two [n_pages, n_k_heads, page_size, head_dim] tensors of one type and layout are wanted")
    code = _CACHE_DTYPES.get(dtype)
    if code is None:
        _refuse(f"caches: {dtype}", BEVPOOL_ERR_UNSUPPORTED)
    n_pages, heads, page_size, d = shape
    if (n_k_heads is not None and heads != n_k_heads) or d != D or k_cache.get_device() != dev or v_cache.get_device() != dev:
        _refuse("caches: heads, head_dim or device does not match")
    sp, sh, ss, se = strides
    if se != 1:
        _refuse("caches: the last axis must be contiguous")
    tshape = block_table.shape
    if len(tshape) != 2:
        _refuse("block_table: [n_seqs, pages] is wanted")
    n_seqs, table_pages = tshape
    return (code, (k_cache.data_ptr(), v_cache.data_ptr()),
            (sp if n_pages > 1 else 0, ss, sh if heads > 1 else 0, n_pages, page_size,
             _vector("block_table", block_table, n_seqs * table_pages, _I32, dev), table_pages,
             _vector("kv_len", kv_len, n_seqs, _I32, dev), _vector("cu_q", cu_q, n_seqs + 1, _I32, dev), n_seqs))


def _stream_of(stream):
    return stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(int(stream))


# Each helper takes `stream` (a torch stream or a cudaStream_t; None: torch's
# current one).  Another stream is made torch's current stream for the call, so
# that what the helper allocates belongs to the stream that uses it.

def qk_norm_rope(q, k, positions, inv_freq, *, sections=None, q_weight=None, k_weight=None, eps: float = 1e-6,
                 interleaved: bool = False, q_out=None, k_out=None, stream=None):
    """bevpool_qk_norm_rope: norms of q and k for each head (where the weight is
    given) and their rotary positions.  positions int32 [tokens] or [tokens,
    axes]; inv_freq float32 [rotary_dim / 2]; sections: pairs of each axis.
    Returns (q_out, k_out); q_out=q, k_out=k works in place."""
    if stream is not None:
        with torch.cuda.stream(_stream_of(stream)):
            return qk_norm_rope(q, k, positions, inv_freq, sections=sections, q_weight=q_weight, k_weight=k_weight, eps=eps,
                                interleaved=interleaved, q_out=q_out, k_out=k_out)
    qs, dtype, code, dev = _check_first("q", q)
    T, Hq, D = qs
    ks = (T, k.shape[1] if k.dim() == 3 else -1, D)
    pos = _position_args(T, dev, positions, inv_freq, sections, interleaved)
    qw, kw = _vector("q_weight", q_weight, D, _F32, dev), _vector("k_weight", k_weight, D, _F32, dev)
    qa, ka = _heads("q", q, qs, dtype, dev), _heads("k", k, ks, dtype, dev)
    if q_out is None:
        q_out = torch.empty(qs, dtype=dtype, device=q.device)
    if k_out is None:
        k_out = torch.empty(ks, dtype=dtype, device=q.device)
    st = _lib.bevpool_qk_norm_rope(code, *qa, *ka, T, Hq, ks[1], D, qw, kw, eps, *pos,
                                   *_heads("q_out", q_out, qs, dtype, dev), *_heads("k_out", k_out, ks, dtype, dev),
                                   torch._C._cuda_getCurrentRawStream(dev))
    if st != BEVPOOL_OK:
        raise BevpoolError(st, "bevpool_qk_norm_rope")
    return q_out, k_out


def qk_norm_rope_backward(dq_out, dk_out, q, k, positions, inv_freq, *, sections=None, q_weight=None, k_weight=None,
                          eps: float = 1e-6, interleaved: bool = False, dq=None, dk=None, workspace=None, stream=None):
    """bevpool_qk_norm_rope_backward: gradients of qk_norm_rope's inputs and
    weights from those of its outputs.  Returns (dq, dk, dq_weight, dk_weight);
    a weight that is None has the gradient None."""
    if stream is not None:
        with torch.cuda.stream(_stream_of(stream)):
            return qk_norm_rope_backward(dq_out, dk_out, q, k, positions, inv_freq, sections=sections, q_weight=q_weight,
                                         k_weight=k_weight, eps=eps, interleaved=interleaved, dq=dq, dk=dk,
                                         workspace=workspace)
    qs, dtype, code, dev = _check_first("q", q)
    T, Hq, D = qs
    ks = (T, k.shape[1] if k.dim() == 3 else -1, D)
    pos = _position_args(T, dev, positions, inv_freq, sections, interleaved)
    qw, kw = _vector("q_weight", q_weight, D, _F32, dev), _vector("k_weight", k_weight, D, _F32, dev)
    ga, ha = _heads("dq_out", dq_out, qs, dtype, dev), _heads("dk_out", dk_out, ks, dtype, dev)
    qa, ka = _heads("q", q, qs, dtype, dev), _heads("k", k, ks, dtype, dev)
    if dq is None:
        dq = torch.empty(qs, dtype=dtype, device=q.device)
    if dk is None:
        dk = torch.empty(ks, dtype=dtype, device=q.device)
    dqw = None if qw is None else torch.empty_like(q_weight)
    dkw = None if kw is None else torch.empty_like(k_weight)
    if workspace is None and not (qw is None and kw is None):
        workspace = torch.empty(max(_lib.bevpool_qk_norm_rope_backward_workspace_size(T, Hq, ks[1], D), 1),
                                dtype=torch.uint8, device=q.device)
    st = _lib.bevpool_qk_norm_rope_backward(
        code, *ga, *ha, *qa, *ka, T, Hq, ks[1], D, qw, kw, eps, *pos, *_heads("dq", dq, qs, dtype, dev),
        *_heads("dk", dk, ks, dtype, dev), None if dqw is None else dqw.data_ptr(), None if dkw is None else dkw.data_ptr(),
        None if workspace is None else workspace.data_ptr(), 0 if workspace is None else workspace.nbytes,
        torch._C._cuda_getCurrentRawStream(dev))
    if st != BEVPOOL_OK:
        raise BevpoolError(st, "bevpool_qk_norm_rope_backward")
    return dq, dk, dqw, dkw


def kv_append(k, v, k_cache, v_cache, block_table, kv_len, cu_q, positions, inv_freq, *, sections=None, k_weight=None,
              eps: float = 1e-6, interleaved: bool = False, k_scale: float = 1.0, v_scale: float = 1.0, q=None,
              q_weight=None, q_out=None, stream=None):
    """bevpool_kv_append: the keys (normed where k_weight is given, and turned)
    and values of new tokens into the paged cache; with q, its norm and rotation
    too.  kv_len counts the new tokens.  Returns q_out (None without q)."""
    if stream is not None:
        with torch.cuda.stream(_stream_of(stream)):
            return kv_append(k, v, k_cache, v_cache, block_table, kv_len, cu_q, positions, inv_freq, sections=sections,
                             k_weight=k_weight, eps=eps, interleaved=interleaved, k_scale=k_scale, v_scale=v_scale, q=q,
                             q_weight=q_weight, q_out=q_out)
    ks, dtype, code, dev = _check_first("k", k)
    T, Hk, D = ks
    pos = _position_args(T, dev, positions, inv_freq, sections, interleaved)
    cache_code, ptrs, pages = _cache_args(k_cache, v_cache, block_table, kv_len, cu_q, dev, Hk, D)
    qw, kw = _vector("q_weight", q_weight, D, _F32, dev), _vector("k_weight", k_weight, D, _F32, dev)
    Hq, qa, oa = 0, (None, 0, 0), (None, 0, 0)
    if q is not None:
        Hq = q.shape[1] if q.dim() == 3 else -1
        qs = (T, Hq, D)
        qa = _heads("q", q, qs, dtype, dev)
        if q_out is None:
            q_out = torch.empty(qs, dtype=dtype, device=q.device)
        oa = _heads("q_out", q_out, qs, dtype, dev)
    elif q_out is not None:
        _refuse("q_out without q")
    st = _lib.bevpool_kv_append(code, cache_code, *_heads("k", k, ks, dtype, dev), *_heads("v", v, ks, dtype, dev), *qa, T, Hq,
                                Hk, D, qw, kw, eps, *pos, *oa, *ptrs, *pages, k_scale, v_scale,
                                torch._C._cuda_getCurrentRawStream(dev))
    if st != BEVPOOL_OK:
        raise BevpoolError(st, "bevpool_kv_append")
    return q_out


def paged_attention(q, k_cache, v_cache, block_table, kv_len, cu_q, *, max_q_len: int, max_kv_len: int,
                    scale: Optional[float] = None, causal: bool = True, window: int = 0, k_scale: float = 1.0,
                    v_scale: float = 1.0, out=None, return_lse: bool = False, workspace=None, stream=None):
    """bevpool_paged_attention: new tokens (rows cu_q[b] .. cu_q[b+1]-1 of q are
    request b's) over the paged cache.  scale defaults to head_dim ** -0.5;
    max_q_len and max_kv_len are host bounds of the requests' lengths.  Returns
    out, or (out, lse) with return_lse.  Rows of q outside every request keep
    what `out` held."""
    if stream is not None:
        with torch.cuda.stream(_stream_of(stream)):
            return paged_attention(q, k_cache, v_cache, block_table, kv_len, cu_q, max_q_len=max_q_len,
                                   max_kv_len=max_kv_len, scale=scale, causal=causal, window=window, k_scale=k_scale,
                                   v_scale=v_scale, out=out, return_lse=return_lse, workspace=workspace)
    qs, dtype, code, dev = _check_first("q", q)
    T, Hq, D = qs
    cache_code, ptrs, pages = _cache_args(k_cache, v_cache, block_table, kv_len, cu_q, dev, None, D)
    Hk = k_cache.shape[1]
    if out is None:
        out = torch.empty(qs, dtype=dtype, device=q.device)
    lse = torch.empty((T, Hq), dtype=_F32, device=q.device) if return_lse else None
    if workspace is None:
        n = _lib.bevpool_paged_attention_workspace_size(pages[9], T, Hq, Hk, D, max_q_len, max_kv_len, window)
        if n:
            workspace = torch.empty(n, dtype=torch.uint8, device=q.device)
    st = _lib.bevpool_paged_attention(
        code, cache_code, *_heads("q", q, qs, dtype, dev), *ptrs, *pages, T, Hq, Hk, D, max_q_len, max_kv_len,
        D ** -0.5 if scale is None else scale, 1 if causal else 0, window, k_scale, v_scale,
        *_heads("out", out, qs, dtype, dev), None if lse is None else lse.data_ptr(),
        None if workspace is None else workspace.data_ptr(), 0 if workspace is None else workspace.nbytes,
        torch._C._cuda_getCurrentRawStream(dev))
    if st != BEVPOOL_OK:
        raise BevpoolError(st, "bevpool_paged_attention")
    return (out, lse) if return_lse else out
