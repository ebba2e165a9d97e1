"""The token operators from their definitions, in FP64 on the CPU, and the
error bounds of their kernels.

Bounds, derived from the arithmetic the header promises (u: half a unit in
the last place of the 16-bit type, 2^-11 for fp16 and 2^-8 for bf16; FP32
operations err by 2^-24 of their result):
  * a normed and turned element is r * (a x + b x') with r from a sum of at
    most 256 squares, cos and sin good to a few 2^-24: about twenty roundings,
    so 2^-18 * r * (|w x| + |w' x'|) covers them with room; then one rounding u.
  * a gradient dx = r (g w - xh mean(g w xh)): the same with the mean's sum,
    2^-16 of the sum of the terms' magnitudes; then one rounding u.
  * a weight's gradient is a sum over rows whose longest FP32 chain is below
    2^7 terms here: 2^-16 of the sum of magnitudes.
  * a score is a dot product of D exact products accumulated in FP32, possibly
    with truncation: off by at most (D + 8) * 2^-23 * scale * sum|q k| = d.  A
    weight is then off by 2 d + 2^-18 relatively (score, exponential, sum) and
    by u once more for its 16-bit rounding, or, where an fp16 weight is
    subnormal, by 2^-24 of the largest; the output is rounded once, u.
  * an E4M3 code: half a step, at most 2^-4 of the value or 2^-10, and what
    the FP32 arithmetic before it may add.
"""
import numpy as np
import torch

U = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}


def tiny(dtype):
    return 2.0 ** -25 if dtype == torch.float16 else 0.0


def cos_sin(positions, inv_freq, sections):
    """[T, R/2] in FP64."""
    pos = positions.cpu().double()
    pos = pos[:, None] if pos.dim() == 1 else pos
    axis = np.repeat(np.arange(len(sections)), sections)
    ang = pos[:, torch.from_numpy(axis)] * inv_freq.cpu().double()[None]
    return torch.cos(ang), torch.sin(ang)


def turn(y, cos, sin, interleaved, back=False):
    """Rotation of [T, H, D] by the first R elements; back: by the negative angle."""
    half = cos.shape[1]
    c, s = cos[:, None], (-sin if back else sin)[:, None]
    out = y.clone()
    a, b = (y[..., 0:2 * half:2], y[..., 1:2 * half:2]) if interleaved else (y[..., :half], y[..., half:2 * half])
    p, q = a * c - b * s, a * s + b * c
    if interleaved:
        out[..., 0:2 * half:2], out[..., 1:2 * half:2] = p, q
    else:
        out[..., :half], out[..., half:2 * half] = p, q
    return out


def partner_abs(y, half, interleaved):
    """|y| plus the magnitude of each turned element's partner."""
    y = y.abs()
    out = y.clone()
    if interleaved:
        out[..., 0:2 * half:2] += y[..., 1:2 * half:2]
        out[..., 1:2 * half:2] += y[..., 0:2 * half:2]
    else:
        out[..., :half] += y[..., half:2 * half]
        out[..., half:2 * half] += y[..., :half]
    return out


def norm_rope(x, w, cos, sin, interleaved, eps):
    """(value, magnitude of its terms) of one tensor; w None: no norm."""
    x = x.cpu().double()
    if w is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * w.cpu().double()
    return turn(x, cos, sin, interleaved), partner_abs(x, cos.shape[1], interleaved)


def norm_rope_back(dy, x, w, cos, sin, interleaved, eps):
    """(dx, its terms' magnitude, dw, its terms' magnitude)."""
    dy, x = dy.cpu().double(), x.cpu().double()
    g, ga = turn(dy, cos, sin, interleaved, back=True), partner_abs(dy, cos.shape[1], interleaved)
    if w is None:
        return g, ga, None, None
    w = w.cpu().double()
    r = 1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    xh = x * r
    dx = r * (g * w - xh * (g * w * xh).mean(-1, keepdim=True))
    mag = r * (ga * w.abs() + xh.abs() * (ga * w.abs() * xh.abs()).mean(-1, keepdim=True))
    return dx, mag, (g * xh).sum((0, 1)), (ga * xh.abs()).sum((0, 1))


def place_of(cu_q, kv_len, block_table, page_size, n_pages, t):
    """(page, slot) of token t, or None where nothing is written."""
    for b in range(len(kv_len)):
        if cu_q[b] <= t < cu_q[b + 1]:
            place = kv_len[b] - cu_q[b + 1] + t
            if place < 0 or place // page_size >= block_table.shape[1]:
                return None
            page = int(block_table[b, place // page_size])
            return (page, place % page_size) if 0 <= page < n_pages else None
    return None


def attention(q, k_cache, v_cache, block_table, kv_len, cu_q, *, max_q_len, max_kv_len, scale, causal, window,
              k_scale=1.0, v_scale=1.0):
    """(out, lse, bound of out, bound of lse, computed rows) in FP64; caches [pages, heads, page, D] in their type."""
    T, Hq, D = q.shape
    n_pages, Hk, page, _ = k_cache.shape
    dtype, u = q.dtype, U[q.dtype]
    q = q.cpu().double()
    table, kv_len, cu = block_table.cpu().numpy(), kv_len.cpu().numpy(), cu_q.cpu().numpy()
    kc, vc = k_cache.float().cpu(), v_cache.float().cpu()      # exact; 8-bit tensors take no indexing
    out, lse = torch.zeros(T, Hq, D, dtype=torch.float64), torch.full((T, Hq), -np.inf, dtype=torch.float64)
    tol, lse_tol = torch.zeros_like(out), torch.zeros_like(lse)
    done = torch.zeros(T, dtype=torch.bool)
    for b in range(len(kv_len)):
        n_q, n_kv = int(cu[b + 1] - cu[b]), int(kv_len[b])
        last = max(min(n_kv, max_kv_len, table.shape[1] * page), 0)
        j = np.arange(last)
        pages = table[b][j // page] if last else np.zeros(0, np.int64)
        live = (pages >= 0) & (pages < n_pages)
        for i in range(min(n_q, max_q_len)):
            t, pos = int(cu[b]) + i, n_kv - n_q + i
            done[t] = True
            see = live.copy()
            if causal:
                see &= j <= pos
            if window:
                see &= j > pos - window
            idx = j[see]
            if not len(idx):
                continue
            at = torch.from_numpy(pages[see].astype(np.int64)), torch.from_numpy((idx % page).astype(np.int64))
            for h in range(Hk):
                k = kc[at[0], h, at[1]].double() * k_scale
                v = vc[at[0], h, at[1]].double() * v_scale
                qs = q[t, h * (Hq // Hk):(h + 1) * (Hq // Hk)]
                s = qs @ k.T * scale
                d = (D + 8) * 2.0 ** -23 * scale * (qs.abs() @ k.abs().T).max(-1).values
                m = s.max(-1, keepdim=True).values
                p = torch.exp(s - m)
                l = p.sum(-1, keepdim=True)
                o = (p / l) @ v
                rows = slice(h * (Hq // Hk), (h + 1) * (Hq // Hk))
                out[t, rows], lse[t, rows] = o, (m + torch.log(l))[:, 0]
                mag = (p / l) @ v.abs()
                sub = 2.0 ** -24 * v.abs().sum(0)[None] / l if dtype == torch.float16 else 0.0
                tol[t, rows] = (u + 2 * d[:, None] + 2.0 ** -18) * mag + sub + u * o.abs() + tiny(dtype)
                lse_tol[t, rows] = d + 2.0 ** -18 + 2.0 ** -22 * lse[t, rows].abs()
    return out, lse, tol, lse_tol, done
