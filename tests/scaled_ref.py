"""The operators of a cache with page scales from their definitions, in FP64 on
the CPU, and the error bounds of their kernels.

Bounds (u, and what an element of a normed and turned key may be off, e =
2^-18 of its terms' magnitude: token_ref):
  * a fresh page's scale is top / 448 rounded once: off by 2^-24 of it and
    e / 448.  One that grows does so by a power of two, the least that holds
    top; where top is within e (and 2^-22 of itself, for two roundings of the
    quotient) of a power's border either is right.
  * a code is within half a step of value / scale: 2^-4 of it or 2^-10, and
    what the value is off.  Values that are exact (no norm, no rotation) have
    the codes of the quotient rounded once.
  * attention: a key's weight in the product is w = 2^(t - M), t = s + log2 of
    the value's scale, s the score in base 2.  Besides the score's own error d
    (token_ref) three FP32 roundings of numbers up to max|s| + max|log2 scale|
    each way: at most 2^-22 of the sum of both, relatively, in w and again in
    the sum.  fp16 weights below 2^-14 are subnormal and off by 2^-25: of 2^14
    times the largest w over few rows (whatever the heads' type), which is 2^-39
    of it, of 2^7 times it or 1 elsewhere (fp16 heads); 2^-38 and 2^-24 of max w
    sum|code| / l cover these.
"""
import numpy as np
import torch

import token_ref as ref

LO, HI = 2.0 ** -48, 2.0 ** 48


def e4m3_of(x):
    """Codes' values of FP64 numbers: nearest, even where halfway, saturating; from the format's definition."""
    a = x.abs().clamp(max=448.0)
    step = torch.exp2(torch.floor(torch.log2(a.clamp(min=2.0 ** -6))) - 3)              # of the code's binade
    return torch.copysign(torch.round(a / step) * step, x)                              # torch.round: halves to even


def page_runs(cu_q, kv_len, table, page, n_pages):
    """(first token, past the last, page, slot of the first) of every run of new tokens of a request on one page."""
    res = []
    for b in range(len(kv_len)):
        t, start = int(cu_q[b]), int(kv_len[b]) - int(cu_q[b + 1] - cu_q[b])
        while t < cu_q[b + 1]:
            place = start + t - int(cu_q[b])
            end = min(int(cu_q[b + 1]), t + page - place % page)
            i = place // page
            p = int(table[b][i]) if 0 <= i < len(table[b]) else -1
            if 0 <= p < n_pages:
                res.append((t, end, p, place % page))
            t = end
    return res


def check_append(runs, value, err, before, scales_before, after, scales_after, exact, what):
    """One cache.  value, err [T, Hk, D] in FP64; codes' values [pages, Hk, page, D] before and after."""
    page = after.shape[2]
    codes, scales = before.clone(), scales_before.clone()
    for t0, t1, p, slot in runs:
        x, e = value[t0:t1].transpose(0, 1), err[t0:t1].transpose(0, 1)                 # [Hk, n, D]
        fin = x.isfinite()
        top = torch.where(fin, x.abs(), torch.zeros_like(x)).amax((1, 2))
        top_e = torch.where(fin, e, torch.zeros_like(x)).amax((1, 2))
        now = scales_after[p].double()
        if slot == 0:
            want = (top / 448).clamp(LO, HI)
            assert ((now - want).abs() <= 2.0 ** -24 * want + top_e / 448).all(), (what, p, now, want)
        else:
            was = scales_before[p].double().clamp(LO, HI)
            n = torch.log2(now / was)
            assert (n == n.round()).all() and (n >= 0).all(), (what, p, n)
            slack = top_e + 2.0 ** -22 * top
            assert ((448 * now >= top - slack) | (now == HI)).all(), (what, p)            # it holds the largest
            assert ((n == 0) | (448 * now / 2 < top + slack)).all(), (what, p)            # and half of it would not
            codes[p, :, :slot] = e4m3_of(before[p, :, :slot] * (was / now)[:, None, None])
        scales[p] = now.float()
        q = x / now[:, None, None]
        got = after[p, :, slot:slot + t1 - t0]
        if exact:
            q = (x.float() / now.float()[:, None, None]).double()
            want = torch.where(q.isnan(), q, e4m3_of(q))
            assert torch.equal(got.nan_to_num(nan=1e9), want.nan_to_num(nan=1e9)), (what, p)
        else:
            tol = torch.maximum(q.abs().clamp(max=448) * 2.0 ** -4, torch.tensor(2.0 ** -10, dtype=torch.float64)) + 1.0625 * e / now[:, None, None]
            assert ((got - q.clamp(-448, 448)).abs() <= tol).all(), (what, p)
        codes[p, :, slot:slot + t1 - t0] = got
    same = (after == codes) | (after.isnan() & codes.isnan())
    assert same.all(), (what, "other slots", (~same).nonzero()[0])
    assert torch.equal(scales.nan_to_num(nan=-1), scales_after.nan_to_num(nan=-1)), (what, "other scales")


def attention(q, k_cache, v_cache, k_scales, v_scales, block_table, kv_len, cu_q, *, max_q_len, max_kv_len, scale, causal=True,
              window=0):
    """(out, lse, bound of out, bound of lse, computed rows) in FP64."""
    T, Hq, D = q.shape
    n_pages, Hk, page, _ = k_cache.shape
    G, dtype, u = Hq // Hk, q.dtype, ref.U[q.dtype]
    q = q.cpu().double()
    table, kv_len, cu = block_table.cpu().numpy(), kv_len.cpu().numpy(), cu_q.cpu().numpy()
    kc, vc = k_cache.float().cpu(), v_cache.float().cpu()
    ks, vs = (x.cpu().double().nan_to_num(nan=LO).clamp(LO, HI) for x in (k_scales, v_scales))
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
            pg, sl = torch.from_numpy(pages[see].astype(np.int64)), torch.from_numpy((idx % page).astype(np.int64))
            for h in range(Hk):
                code = vc[pg, h, sl].double()
                k, f = kc[pg, h, sl].double() * ks[pg, h][:, None], vs[pg, h]
                rows = slice(h * G, (h + 1) * G)
                qs = q[t, rows]
                s = qs @ k.T * scale
                d = (D + 8) * 2.0 ** -23 * scale * (qs.abs() @ k.abs().T).max(-1).values
                d = d + 2.0 ** -22 * 1.4427 * s.abs().max(-1).values + 2.0 ** -22 * f.log2().abs().max()
                m = s.max(-1, keepdim=True).values
                p = torch.exp(s - m)
                l = p.sum(-1, keepdim=True)
                o, mag = (p * f / l) @ code, (p * f / l) @ code.abs()
                out[t, rows], lse[t, rows] = o, (m + torch.log(l))[:, 0]
                sub = 2.0 ** (-24 if dtype == torch.float16 else -38) * (p * f).max(-1, keepdim=True).values * code.abs().sum(0)[None] / l
                tol[t, rows] = (u + 2 * d[:, None] + 2.0 ** -18) * mag + sub + u * o.abs() + ref.tiny(dtype)
                lse_tol[t, rows] = d + 2.0 ** -18 + 2.0 ** -22 * lse[t, rows].abs()
    return out, lse, tol, lse_tol, done
