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

import contextlib
import ctypes
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


def _refuse(what: str, status: int = BEVPOOL_ERR_INVALID_ARG):
    raise BevpoolError(status, what)


def _heads(name: str, t, like=None):
    """Checks a [tokens, heads, head_dim] tensor; returns (pointer, token stride, head stride)."""
    if t.dim() != 3 or not t.is_cuda:
        _refuse(f"{name}: a [tokens, heads, head_dim] CUDA tensor is wanted")
    if t.dtype not in _DTYPES:
        _refuse(f"{name}: fp16 or bf16 is wanted, got {t.dtype}", BEVPOOL_ERR_UNSUPPORTED)
    ts, hs, es = t.stride()
    if es != 1 and t.shape[2] != 1:
        _refuse(f"{name}: the last axis must be contiguous")
    if like is not None and (t.dtype != like.dtype or t.device != like.device or t.shape[0] != like.shape[0]
                             or t.shape[2] != like.shape[2]):
        _refuse(f"{name}: type, device, tokens and head_dim must match")
    # the stride of an axis of one entry is never used
    return t.data_ptr(), (ts if t.shape[0] > 1 else 0), (hs if t.shape[1] > 1 else 0)


def _out(name: str, t, like, heads: int):
    if t is None:
        return torch.empty((like.shape[0], heads, like.shape[2]), dtype=like.dtype, device=like.device)
    if t.shape != (like.shape[0], heads, like.shape[2]) or t.dtype != like.dtype or t.device != like.device:
        _refuse(f"{name}: shape, type or device does not match")
    return t


def _vector(name: str, t, n: int, dtype, device):
    if t is None:
        return None
    if t.dtype != dtype or t.device != device or t.numel() != n or not t.is_contiguous():
        _refuse(f"{name}: a contiguous {dtype} tensor of {n} entries on {device} is wanted")
    return t.data_ptr()


def _position_args(like, positions, inv_freq, sections: Optional[Sequence[int]], interleaved: bool) -> tuple:
    T = like.shape[0]
    n_axes = positions.shape[1] if positions.dim() == 2 else 1
    if positions.dim() not in (1, 2) or positions.shape[0] != T or not 1 <= n_axes <= MAX_AXES:
        _refuse(f"positions: int32 [tokens] or [tokens, axes <= {MAX_AXES}] is wanted")
    n = inv_freq.numel()
    sec = [n] if sections is None else list(sections)
    if len(sec) != n_axes:
        _refuse("sections: one entry an axis is wanted")
    return (_vector("positions", positions, T * n_axes, torch.int32, like.device), n_axes, (_i32 * n_axes)(*sec), 2 * n,
            _vector("inv_freq", inv_freq, n, torch.float32, like.device), int(interleaved))


def _cache_args(k_cache, v_cache, block_table, kv_len, cu_q, like, n_k_heads: int) -> tuple:
    """(cache dtype, (k pointer, v pointer), page arguments)."""
    if k_cache.dim() != 4 or k_cache.shape != v_cache.shape or k_cache.dtype != v_cache.dtype:
        _refuse("caches: two [n_pages, n_k_heads, page_size, head_dim] tensors of one type are wanted")
    if k_cache.dtype not in _CACHE_DTYPES:
        _refuse(f"caches: {k_cache.dtype}", BEVPOOL_ERR_UNSUPPORTED)
    n_pages, heads, page_size, D = k_cache.shape
    if heads != n_k_heads or D != like.shape[2] or k_cache.device != like.device or v_cache.device != like.device:
        _refuse("caches: heads, head_dim or device does not match")
    if k_cache.stride() != v_cache.stride() or k_cache.stride(3) != 1:
        _refuse("caches: equal strides and a contiguous last axis are wanted")
    if block_table.dim() != 2 or cu_q.numel() != block_table.shape[0] + 1:
        _refuse("block_table [n_seqs, pages] and cu_q [n_seqs + 1] are wanted")
    n_seqs, table_pages = block_table.shape
    sp, sh, ss, _ = k_cache.stride()
    dev = like.device
    return (_CACHE_DTYPES[k_cache.dtype], (k_cache.data_ptr(), v_cache.data_ptr()),
            (sp if n_pages > 1 else 0, ss, sh if heads > 1 else 0, n_pages, page_size,
             _vector("block_table", block_table, n_seqs * table_pages, torch.int32, dev), table_pages,
             _vector("kv_len", kv_len, n_seqs, torch.int32, dev), _vector("cu_q", cu_q, n_seqs + 1, torch.int32, dev),
             n_seqs))


@contextlib.contextmanager
def _torch_stream(stream):
    with torch.cuda.stream(stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(int(stream))):
        yield


def _on_stream(fn):
    """Runs a helper with `stream` (a torch stream or a cudaStream_t; None: the
    current one) as torch's current stream, so that what it allocates belongs
    to the stream that uses it."""
    def run(*args, stream=None, **kw):
        if stream is None:
            return fn(*args, stream=torch.cuda.current_stream().cuda_stream, **kw)
        with _torch_stream(stream):
            return fn(*args, stream=torch.cuda.current_stream().cuda_stream, **kw)

    run.__name__, run.__doc__ = fn.__name__, fn.__doc__
    run.__wrapped__ = fn
    return run


def _check_device(t):
    if t.device.index != torch.cuda.current_device():
        _refuse("tensors must be on the current CUDA device")


@_on_stream
def qk_norm_rope(q, k, positions, inv_freq, *, sections=None, q_weight=None, k_weight=None, eps: float = 1e-6,
                 interleaved: bool = False, q_out=None, k_out=None, stream=None):
    """bevpool_qk_norm_rope: norms of q and k for each head (where the weight is
    given) and their rotary positions.  positions int32 [tokens] or [tokens,
    axes]; inv_freq float32 [rotary_dim / 2]; sections: pairs of each axis.
    Returns (q_out, k_out); q_out=q, k_out=k works in place."""
    qa, ka = _heads("q", q), _heads("k", k, q)
    _check_device(q)
    D = q.shape[2]
    pos = _position_args(q, positions, inv_freq, sections, interleaved)
    w = (_vector("q_weight", q_weight, D, torch.float32, q.device), _vector("k_weight", k_weight, D, torch.float32, q.device))
    q_out, k_out = _out("q_out", q_out, q, q.shape[1]), _out("k_out", k_out, k, k.shape[1])
    st = bevpool_qk_norm_rope(_DTYPES[q.dtype], *qa, *ka, q.shape[0], q.shape[1], k.shape[1], D, *w, eps, *pos,
                              *_heads("q_out", q_out), *_heads("k_out", k_out), stream)
    if st != BEVPOOL_OK:
        raise BevpoolError(st, "bevpool_qk_norm_rope")
    return q_out, k_out


@_on_stream
def qk_norm_rope_backward(dq_out, dk_out, q, k, positions, inv_freq, *, sections=None, q_weight=None, k_weight=None,
                          eps: float = 1e-6, interleaved: bool = False, dq=None, dk=None, workspace=None, stream=None):
    """bevpool_qk_norm_rope_backward: gradients of qk_norm_rope's inputs and
    weights from those of its outputs.  Returns (dq, dk, dq_weight, dk_weight);
    a weight that is None has the gradient None."""
    ga, ha, qa, ka = _heads("dq_out", dq_out, q), _heads("dk_out", dk_out, q), _heads("q", q), _heads("k", k, q)
    _check_device(q)
    T, Hq, D = q.shape
    Hk = k.shape[1]
    if dq_out.shape[1] != Hq or dk_out.shape[1] != Hk:
        _refuse("dq_out, dk_out: heads must match q and k")
    pos = _position_args(q, positions, inv_freq, sections, interleaved)
    w = (_vector("q_weight", q_weight, D, torch.float32, q.device), _vector("k_weight", k_weight, D, torch.float32, q.device))
    dq, dk = _out("dq", dq, q, Hq), _out("dk", dk, k, Hk)
    dqw, dkw = (None if x is None else torch.empty(D, dtype=torch.float32, device=q.device) for x in (q_weight, k_weight))
    if workspace is None and (q_weight is not None or k_weight is not None):
        n = bevpool_qk_norm_rope_backward_workspace_size(T, Hq, Hk, D)
        workspace = torch.empty(max(n, 1), dtype=torch.uint8, device=q.device)
    st = bevpool_qk_norm_rope_backward(
        _DTYPES[q.dtype], *ga, *ha, *qa, *ka, T, Hq, Hk, D, *w, eps, *pos, *_heads("dq", dq), *_heads("dk", dk),
        None if dqw is None else dqw.data_ptr(), None if dkw is None else dkw.data_ptr(),
        None if workspace is None else workspace.data_ptr(),
        0 if workspace is None else workspace.numel() * workspace.element_size(), stream)
    if st != BEVPOOL_OK:
        raise BevpoolError(st, "bevpool_qk_norm_rope_backward")
    return dq, dk, dqw, dkw


@_on_stream
def kv_append(k, v, k_cache, v_cache, block_table, kv_len, cu_q, positions, inv_freq, *, sections=None, k_weight=None,
              eps: float = 1e-6, interleaved: bool = False, k_scale: float = 1.0, v_scale: float = 1.0, q=None,
              q_weight=None, q_out=None, stream=None):
    """bevpool_kv_append: the keys (normed where k_weight is given, and turned)
    and values of new tokens into the paged cache; with q, its norm and rotation
    too.  kv_len counts the new tokens.  Returns q_out (None without q)."""
    ka, va = _heads("k", k), _heads("v", v, k)
    _check_device(k)
    T, Hk, D = k.shape
    if v.shape[1] != Hk:
        _refuse("v: heads must match k")
    pos = _position_args(k, positions, inv_freq, sections, interleaved)
    cache_dtype, ptrs, pages = _cache_args(k_cache, v_cache, block_table, kv_len, cu_q, k, Hk)
    w = (_vector("q_weight", q_weight, D, torch.float32, k.device), _vector("k_weight", k_weight, D, torch.float32, k.device))
    if q is None:
        if q_out is not None:
            _refuse("q_out without q")
        Hq, qa, oa = 0, (None, 0, 0), (None, 0, 0)
    else:
        Hq, qa = q.shape[1], _heads("q", q, k)
        q_out = _out("q_out", q_out, q, Hq)
        oa = _heads("q_out", q_out)
    st = bevpool_kv_append(_DTYPES[k.dtype], cache_dtype, *ka, *va, *qa, T, Hq, Hk, D, *w, eps, *pos, *oa, *ptrs, *pages,
                           k_scale, v_scale, stream)
    if st != BEVPOOL_OK:
        raise BevpoolError(st, "bevpool_kv_append")
    return q_out


@_on_stream
def paged_attention(q, k_cache, v_cache, block_table, kv_len, cu_q, *, max_q_len: int, max_kv_len: int,
                    scale: Optional[float] = None, causal: bool = True, window: int = 0, k_scale: float = 1.0,
                    v_scale: float = 1.0, out=None, return_lse: bool = False, workspace=None, stream=None):
    """bevpool_paged_attention: new tokens (rows cu_q[b] .. cu_q[b+1]-1 of q are
    request b's) over the paged cache.  scale defaults to head_dim ** -0.5;
    max_q_len and max_kv_len are host bounds of the requests' lengths.  Returns
    out, or (out, lse) with return_lse.  Rows of q outside every request keep
    what `out` held."""
    qa = _heads("q", q)
    _check_device(q)
    T, Hq, D = q.shape
    Hk = k_cache.shape[1] if k_cache.dim() == 4 else 0
    cache_dtype, ptrs, pages = _cache_args(k_cache, v_cache, block_table, kv_len, cu_q, q, Hk)
    out = _out("out", out, q, Hq)
    lse = torch.empty((T, Hq), dtype=torch.float32, device=q.device) if return_lse else None
    if workspace is None:
        n = bevpool_paged_attention_workspace_size(pages[-1], T, Hq, Hk, D, max_q_len, max_kv_len, window)
        workspace = torch.empty(n, dtype=torch.uint8, device=q.device) if n else None
    st = bevpool_paged_attention(
        _DTYPES[q.dtype], cache_dtype, *qa, *ptrs, *pages, T, Hq, Hk, D, max_q_len, max_kv_len,
        D ** -0.5 if scale is None else scale, int(causal), window, k_scale, v_scale, *_heads("out", out),
        None if lse is None else lse.data_ptr(), None if workspace is None else workspace.data_ptr(),
        0 if workspace is None else workspace.numel() * workspace.element_size(), stream)
    if st != BEVPOOL_OK:
        raise BevpoolError(st, "bevpool_paged_attention")
    return (out, lse) if return_lse else out
