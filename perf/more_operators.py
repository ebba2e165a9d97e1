"""Measured cases of the operators around an 8-bit paged cache with a scale for
each page and key head: pages handed to requests from their lengths, the append
that works the scales out, and the attention that reads such a cache.

With ``own`` false, ``run`` computes the operators from elementary torch
operations in 32 bits (64 for counts), rounded once at the end; with ``own``
true it calls the library's entry points (depth_weighted_scatter_gb300.attention).

  plan     lengths, tables and free pages -> cu_q, positions, slots and the new lengths, tables and free pages
  append   k, v (and q) of new tokens -> codes and scales of the paged cache (and q)
  attend   q of new tokens over the paged cache -> out, lse
"""
import math

import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
EPS = 1e-6
THETA = 10000.0
LARGEST = 448.0                       # of an E4M3 code
SCALE_LO, SCALE_HI = 2.0 ** -48, 2.0 ** 48


# ------------------------------------------------------------------ cases

def listed():
    return [
        # A decoding step of 64 requests: launch latency is what counts.
        dict(name="plan_step", op="plan", B=64, q_max=1, kv_max=8192, page=16, drop=0, ended=0.0),
        # A new frame of four samples' 128 x 128 BEV grids; each gives its oldest frame's 256 pages back.
        dict(name="plan_frames", op="plan", B=4, q_max=16384, kv_max=65536, page=64, drop=256, ended=0.0),
        # Many short requests with a few drafted tokens each, one in eight of them ended.
        dict(name="plan_many", op="plan", B=4000, q_max=7, kv_max=2000, page=16, drop=0, ended=0.125),
        # A decoding step of 64 requests: one token each into a page that is partly filled, q on the way.
        dict(name="append_step", op="append", B=64, q_max=1, kv_max=2000, Hq=32, Hk=8, D=128, R=128, axes=1,
             interleaved=False, dtype="bf16", page=16),
        # Ragged chunks of prompts that begin inside a page.
        dict(name="append_chunks", op="append", B=6, q_max=1501, kv_max=12000, Hq=32, Hk=8, D=128, R=96, axes=1,
             interleaved=False, dtype="bf16", page=64),
        # Four cameras' or samples' BEV grids at once, positions (time, y, x).
        dict(name="append_frames", op="append", B=4, q_max=16384, kv_max=16384, Hq=8, Hk=8, D=64, R=64, axes=3,
             interleaved=True, dtype="f16", page=64),
        # One request's single token over a short context: the smallest call.
        dict(name="attend_step_one", op="attend", B=1, q_max=1, kv_max=777, Hq=8, Hk=8, D=64, causal=True, window=0,
             dtype="f16", page=16),
        # A decoding step of 64 requests with ragged contexts.
        dict(name="attend_step_batch", op="attend", B=64, q_max=1, kv_max=8192, Hq=32, Hk=8, D=128, causal=True,
             window=0, dtype="bf16", page=16),
        # Two long contexts: few rows, a long axis.
        dict(name="attend_step_long", op="attend", B=2, q_max=1, kv_max=131072, Hq=32, Hk=8, D=128, causal=True,
             window=0, dtype="bf16", page=64),
        # Ragged chunks of prompts over what is cached of each request.
        dict(name="attend_chunks", op="attend", B=6, q_max=500, kv_max=12000, Hq=32, Hk=8, D=128, causal=True,
             window=0, dtype="bf16", page=16),
        # The 50 x 50 BEV grid of a new frame over itself and four earlier frames, every cell seeing every cell.
        dict(name="attend_frames", op="attend", B=2, q_max=2500, kv_max=12500, Hq=8, Hk=8, D=64, causal=False,
             window=0, dtype="f16", page=64),
        # A whole prompt at once.
        dict(name="attend_prompt", op="attend", B=1, q_max=8192, kv_max=8192, Hq=32, Hk=8, D=128, causal=True,
             window=0, dtype="bf16", page=128),
    ]


def _size(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm; odd ones as likely as even ones."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["plan", "append", "append", "attend", "attend", "attend"])
    page = rng.choice([16, 32, 64, 128, 256])
    if op == "plan":
        B = _size(rng, 1, 4000)
        q_max = _size(rng, 1, max(1, min(16384, 65536 // B)))
        kv_max = _size(rng, 1, min(65536, (1 << 23) // B))
        return dict(op=op, B=B, q_max=q_max, kv_max=kv_max, page=page,
                    drop=rng.choice([0, 0, 1, max(1, kv_max // page // 3)]), ended=rng.choice([0.0, 0.0, 0.125, 0.5]))
    dtype = rng.choice(["f16", "bf16"])
    Hk = rng.choice([1, 2, 4, 8])
    Hq = Hk * rng.choice([1, 2, 4, 7] if Hk < 8 else [1, 2, 4])
    D = rng.choice([64, 128])
    if op == "append":
        B = _size(rng, 1, 64)
        q_max = _size(rng, 1, max(1, min(16384, 65536 * 24 * 64 // (B * D * (Hq + 2 * Hk)))))
        kv_max = _size(rng, q_max, max(q_max, min(q_max + 4000, 65536 // B)))
        return dict(op=op, B=B, q_max=q_max, kv_max=kv_max, Hq=Hq, Hk=Hk, D=D, R=rng.choice([D, D, D // 2]),
                    axes=rng.choice([1, 3]), interleaved=rng.random() < 0.5, dtype=dtype, page=page)
    causal = rng.random() < 0.75
    window = _size(rng, 64, 4096) if causal and rng.random() < 0.3 else 0
    if rng.random() < 0.5:
        # few new tokens over a cache of up to about 0.5 GB
        B, q_max = _size(rng, 1, 64), rng.choice([1, 1, 1, 2, 4])
        kv_max = _size(rng, 64, max(64, min(131072, (1 << 28) // (B * Hk * D))))
    else:
        # chunks: rows x keys bounded by the whole prompt's
        B, q_max = _size(rng, 1, 8), _size(rng, 16, 4000)
        most = 32 * 8192 * 8192 // (2 * Hq * B * q_max)
        kv_max = _size(rng, q_max, max(q_max, min(32768, most, (1 << 28) // (B * Hk * D))))
        B = max(1, min(B, most * B // kv_max))
    return dict(op=op, B=B, q_max=q_max, kv_max=kv_max, Hq=Hq, Hk=Hk, D=D, causal=causal, window=window, dtype=dtype,
                page=page)


def _lengths(case):
    """New tokens and cached tokens (the new ones included) of each request: ragged, the first one the longest."""
    B, q_max, kv_max = case["B"], case["q_max"], case["kv_max"]
    q_len = [max(1, q_max - int(q_max * 0.6 * ((b * 0.6180339887) % 1.0))) for b in range(B)]
    kv_len = [max(q, kv_max - int(kv_max * 0.6 * ((b * 0.7548776662) % 1.0))) for b, q in enumerate(q_len)]
    return q_len, kv_len


def _sections(case):
    P = case["R"] // 2
    if case["axes"] == 1:
        return [P]
    first = P // 4
    return [first, (P - first) // 2, P - first - (P - first) // 2]


# ------------------------------------------------------------------ inputs

def _randn(g, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _positions(case, starts, lens):
    """int32 [T, axes]: the index in the request, or (time, y, x) on a BEV grid of 128 columns."""
    at = torch.cat([torch.arange(s, s + n, device="cuda") for s, n in zip(starts, lens)])
    if case["axes"] == 1:
        return at.to(torch.int32)[:, None].contiguous()
    return torch.stack([at // 16384, at % 16384 // 128, at % 128], dim=1).to(torch.int32).contiguous()


def _rotary(case, g):
    D, p = case["D"], torch.arange(case["R"] // 2, dtype=torch.float64)
    return dict(inv_freq=torch.pow(THETA, -2.0 * p / case["R"]).to(torch.float32).cuda(), sections=_sections(case),
                q_weight=1.0 + 0.1 * _randn(g, D), k_weight=1.0 + 0.1 * _randn(g, D))


def _table(order, n_pages, width):
    """[B, width] page numbers out of `order`, -1 past each request's pages; the pages taken."""
    n = torch.tensor(n_pages, device="cuda")
    first = n.cumsum(0) - n
    col = torch.arange(width, device="cuda")[None, :]
    at = (first[:, None] + col).clamp(max=order.numel() - 1)
    return torch.where(col < n[:, None], order[at], torch.full_like(order[:1], -1)).contiguous()


def _prepare_plan(case, s, g):
    q_len, kv_len = _lengths(case)
    B, page = case["B"], case["page"]
    n_pages = [-(-n // page) for n in kv_len]
    width = -(-(case["kv_max"] + case["q_max"]) // page) + 1
    total = sum(-(-(n + q) // page) for n, q in zip(kv_len, q_len)) + 64       # pages enough whatever is dropped
    order = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    used = sum(n_pages)
    free = torch.full((total,), -1, dtype=torch.int32, device="cuda")
    free[:total - used] = order[used:]
    ends = torch.rand(B, generator=g, device="cuda") < case["ended"]
    some = torch.randint(0, case["drop"] + 1, (B,), generator=g, device="cuda")          # pages given back, ragged
    s.update(q_len=_i32(q_len), kv_len=_i32(kv_len), page=page, n_tokens=sum(q_len),
             first=torch.randint(0, 1000, (B,), generator=g, device="cuda").to(torch.int32),
             block_table=_table(order, n_pages, width), free_pages=free, n_free=_i32([total - used]), drop=None)
    if case["drop"] or case["ended"]:
        some = torch.full_like(some, case["drop"]) if case["ended"] == 0.0 else some     # frames leave whole
        s["drop"] = torch.where(ends, torch.full_like(some, -1), some).to(torch.int32)
    return s


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    s = dict(case=case)
    if case["op"] == "plan":
        return _prepare_plan(case, s, g)
    D, Hq, Hk, dtype = case["D"], case["Hq"], case["Hk"], DTYPES[case["dtype"]]
    q_len, kv_len = _lengths(case)
    page, T = case["page"], sum(q_len)
    n_pages = [-(-n // page) for n in kv_len]
    total = sum(n_pages)
    order = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    s.update(block_table=_table(order, n_pages, max(n_pages)), kv_len=_i32(kv_len),
             cu_q=torch.tensor([0] + q_len).cumsum(0).to(torch.int32).cuda(), max_q_len=max(q_len),
             max_kv_len=max(kv_len))

    def pool():
        # codes whose largest are near 448, as the append makes them, and pages of different magnitudes
        x = (_randn(g, total, Hk, page, D, dtype=torch.float16) * 112.0).clamp(-LARGEST, LARGEST)
        return x.to(torch.float8_e4m3fn), (torch.exp(0.5 * _randn(g, total, Hk)) / 112.0).contiguous()

    s["k_cache"], s["k_scales"] = pool()
    s["v_cache"], s["v_scales"] = pool()
    if case["op"] == "append":
        s.update(_rotary(case, g))
        qkv = _randn(g, T, Hq + 2 * Hk, D, dtype=dtype)        # the fused projection's output
        s.update(q=qkv[:, :Hq], k=qkv[:, Hq:Hq + Hk], v=qkv[:, Hq + Hk:])
        s["positions"] = _positions(case, [n - q for n, q in zip(kv_len, q_len)], q_len)
    else:
        s["q"] = _randn(g, T, Hq, D, dtype=dtype)
    return s


# ------------------------------------------------------------------ plain forms

def _plain_plan(s):
    page, T = s["page"], s["n_tokens"]
    table, free, n_free = s["block_table"].long(), s["free_pages"].long(), s["n_free"].long()
    B, width = table.shape
    dev, cap = table.device, free.numel()
    q, old = s["q_len"].long().clamp(min=0), s["kv_len"].long().clamp(min=0)
    pages = (old + page - 1) // page
    drop = torch.zeros_like(q) if s["drop"] is None else s["drop"].long()
    d = torch.where(drop < 0, pages, torch.minimum(drop, pages))
    kept = (old - d * page).clamp(min=0)
    first = torch.where(drop < 0, torch.zeros_like(old), s["first"].long() + old - kept)
    had, has = pages - d, (kept + q + page - 1) // page
    want = has - had
    cu, wants, drops = (torch.cat([x.new_zeros(1), x.cumsum(0)]) for x in (q, want, d))
    given, top = drops[-1], n_free + drops[-1]
    fits = (has <= width).all() & (pages <= width).all() & (cu[-1] <= T) & (top <= cap)
    ok = fits & (wants[-1] <= top)
    # the free pages with those given back on top, in the requests' order
    v = torch.arange(cap, device=dev)
    b = (torch.searchsorted(drops, v - n_free, right=True) - 1).clamp(0, B - 1)
    back = table[b, (v - n_free - drops[b]).clamp(0, width - 1)]
    stack = torch.where(v < n_free, free, back)
    left = torch.where(ok, top - wants[-1], n_free)
    col = torch.arange(width, device=dev)[None, :]
    moved = table.gather(1, (col + d[:, None]).clamp(max=width - 1))
    taken = stack[(top - 1 - (wants[:-1, None] + col - had[:, None])).clamp(0, cap - 1)]
    none = torch.full_like(moved, -1)
    after = torch.where(col < had[:, None], moved, torch.where(col < has[:, None], taken, none))
    after = torch.where(ok, after, table)
    t = torch.arange(T, device=dev)
    r = (torch.searchsorted(cu, t, right=True) - 1).clamp(0, B - 1)
    place = kept[r] + t - cu[r]
    live = ok & (t < cu[-1])
    slots = after[r, (place // page).clamp(0, width - 1)] * page + place % page
    lack = torch.where(fits, (wants[-1] - top).clamp(min=0), torch.full_like(given, -1))
    i32 = torch.int32
    return dict(cu_q=torch.where(ok, cu, torch.zeros_like(cu)).to(i32),
                positions=torch.where(live, first[r] + place, torch.zeros_like(place)).to(i32),
                slots=torch.where(live, slots, torch.full_like(slots, -1)),
                kv_len=torch.where(ok, kept + q, old).to(i32), first=torch.where(ok, first, s["first"].long()).to(i32),
                block_table=after.to(i32),
                free_pages=torch.where(v < left, torch.where(ok, stack, free), torch.full_like(v, -1)).to(i32),
                n_free=left.to(i32), missing=lack.reshape(1).to(i32))


def _cos_sin(s):
    """cos and sin [T, 1, R/2] of position * inv_freq.  The frequency and the position are split so that the large
    products are exact in 32 bits; the angles then add by the angle-sum formula."""
    f = s["inv_freq"]
    axis = torch.repeat_interleave(torch.arange(len(s["sections"]), device=f.device),
                                   torch.tensor(s["sections"], device=f.device), output_size=f.numel())
    pos = s["positions"][:, axis]
    f_hi = (f.view(torch.int32) & -4096).view(torch.float32)
    a = (pos & -4096).float() * f_hi
    b = (pos & 4095).float() * f_hi
    c = pos.float() * (f - f_hi)
    ca, sa, cb, sb, cc, sc = a.cos(), a.sin(), b.cos(), b.sin(), c.cos(), c.sin()
    cab, sab = ca * cb - sa * sb, sa * cb + ca * sb
    return (cab * cc - sab * sc)[:, None], (sab * cc + cab * sc)[:, None]


def _turned(x, w, cos, sin, R, interleaved):
    x = x.float()
    x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w
    a, b = (x[..., 0:R:2], x[..., 1:R:2]) if interleaved else (x[..., :R // 2], x[..., R // 2:R])
    y0, y1 = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([y0, y1], dim=-1).flatten(-2) if interleaved else torch.cat([y0, y1], dim=-1)
    return torch.cat([turned, x[..., R:]], dim=-1)


def _codes(x):
    return x.clamp(-LARGEST, LARGEST).to(torch.float8_e4m3fn)


def _put(s, cache, scales, x):
    """Rows x [T, Hk, D] into a cache, its pages' scales with them."""
    page, cu, kv_len, table = s["case"]["page"], s["cu_q"].long(), s["kv_len"].long(), s["block_table"].long()
    t = torch.arange(x.shape[0], device=x.device)
    b = torch.searchsorted(cu[1:], t, right=True)
    place = kv_len[b] - cu[b + 1] + t
    pages = table[b, place // page]
    # the largest magnitude that each page gets
    top = torch.zeros_like(scales).index_reduce_(0, pages, x.abs().amax(-1), "amax")
    fresh = (top / LARGEST).clamp(min=SCALE_LO, max=SCALE_HI)
    # a request's first page may hold earlier tokens: its scale only grows, by powers of two
    start = kv_len - (cu[1:] - cu[:-1])
    held = start % page
    head = table.gather(1, (start // page).clamp(max=table.shape[1] - 1)[:, None])[:, 0]
    some = (held > 0) & (cu[1:] > cu[:-1])
    was = scales[head].clamp(min=SCALE_LO, max=SCALE_HI)
    m, e = torch.frexp(top[head] / (LARGEST * was))
    grow = torch.where(m == 0.5, e - 1, e).clamp(min=0)
    now = torch.ldexp(was, grow).clamp(max=SCALE_HI)
    now = torch.where(some[:, None], now, fresh[head])
    slot = torch.arange(page, device=x.device)
    bytes_ = cache.view(torch.uint8)                       # float8 tensors take no indexed writes
    old = bytes_[head]                                     # [B, Hk, page, D]
    moved = _codes(old.view(torch.float8_e4m3fn).float() * (was / now)[..., None, None]).view(torch.uint8)
    keep = (slot < held[:, None])[:, None, :, None] & some[:, None, None, None]
    bytes_[head] = torch.where(keep, moved, old)
    fresh[head] = now
    scales[pages] = fresh[pages]
    bytes_[pages, :, place % page] = _codes(x / fresh[pages][..., None]).view(torch.uint8)


def _plain_append(s):
    case = s["case"]
    cos, sin = _cos_sin(s)
    turn = (cos, sin, case["R"], case["interleaved"])
    _put(s, s["k_cache"], s["k_scales"], _turned(s["k"], s["k_weight"], *turn))
    _put(s, s["v_cache"], s["v_scales"], s["v"].float())
    return dict(q=_turned(s["q"], s["q_weight"], *turn).to(DTYPES[case["dtype"]]), k_cache=s["k_cache"],
                v_cache=s["v_cache"], k_scales=s["k_scales"], v_scales=s["v_scales"])


def _plain_attend(s):
    case = s["case"]
    B, Hq, Hk, D = case["B"], case["Hq"], case["Hk"], case["D"]
    G, qm = Hq // Hk, s["max_q_len"]
    cu, kv_len, dev = s["cu_q"].long(), s["kv_len"].long(), s["q"].device
    table = s["block_table"].long().clamp(min=0)

    def rows(cache, scales):       # [B, Hk, L, D]
        x = cache.view(torch.uint8)[table].view(cache.dtype).float() * scales[table][..., None, None]
        return x.permute(0, 2, 1, 3, 4).reshape(B, Hk, -1, D)

    q_len = cu[1:] - cu[:-1]
    i = torch.arange(qm, device=dev)
    take = (cu[:-1, None] + i).clamp(max=s["q"].shape[0] - 1)
    q = s["q"][take].float().view(B, qm, Hk, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hk, G * qm, D)
    sc = (q * (1.0 / math.sqrt(D))) @ rows(s["k_cache"], s["k_scales"]).transpose(-1, -2)
    j = torch.arange(sc.shape[-1], device=dev)
    pos = (kv_len - q_len)[:, None] + i                                    # [B, qm]
    last = pos if case["causal"] else (kv_len - 1)[:, None].expand(B, qm)
    seen = (j <= last[..., None]) & (j < kv_len[:, None, None])
    if case["window"]:
        seen &= j > (pos - case["window"])[..., None]
    sc.view(B, Hk, G, qm, -1).masked_fill_(~seen[:, None, None], float("-inf"))
    m = sc.amax(-1, keepdim=True)
    e = sc.sub_(m).exp_()
    l = e.sum(-1, keepdim=True)
    o = (e @ rows(s["v_cache"], s["v_scales"])) / l
    o = o.view(B, Hk, G, qm, D).permute(0, 3, 1, 2, 4).reshape(B, qm, Hq, D)
    lse = (m + l.log()).view(B, Hk, G, qm).permute(0, 3, 1, 2).reshape(B, qm, Hq)
    t = torch.arange(s["q"].shape[0], device=dev)
    b = torch.searchsorted(cu[1:], t, right=True)
    return dict(out=o[b, t - cu[b]].to(s["q"].dtype), lse=lse[b, t - cu[b]].contiguous())


# ------------------------------------------------------------------ one pass

def _own(s):
    from depth_weighted_scatter_gb300 import attention

    case = s["case"]
    if case["op"] == "plan":
        plan = attention.plan_pages(s["q_len"], s["kv_len"], s["first"], s["block_table"], s["free_pages"], s["n_free"],
                                    page_size=s["page"], n_tokens=s["n_tokens"], drop=s["drop"])
        return plan._asdict()
    pages = (s["block_table"], s["kv_len"], s["cu_q"])
    if case["op"] == "attend":
        out, lse = attention.paged_attention_scaled(
            s["q"], s["k_cache"], s["v_cache"], s["k_scales"], s["v_scales"], *pages, max_q_len=s["max_q_len"],
            max_kv_len=s["max_kv_len"], causal=case["causal"], window=case["window"], return_lse=True)
        return dict(out=out, lse=lse)
    q = attention.kv_append_scaled(
        s["k"], s["v"], s["k_cache"], s["v_cache"], s["k_scales"], s["v_scales"], *pages, s["positions"], s["inv_freq"],
        sections=s["sections"], k_weight=s["k_weight"], eps=EPS, interleaved=case["interleaved"], q=s["q"],
        q_weight=s["q_weight"])
    return dict(q=q, k_cache=s["k_cache"], v_cache=s["v_cache"], k_scales=s["k_scales"], v_scales=s["v_scales"])


def run(state):
    if own:
        return _own(state)
    return {"plan": _plain_plan, "append": _plain_append, "attend": _plain_attend}[state["case"]["op"]](state)


# ------------------------------------------------------------------ what a pass cannot do without

def _seen(case, q_len, kv_len):
    """Keys seen by all new tokens of one request, and the keys that any of them sees."""
    if not case["causal"]:
        return q_len * kv_len, kv_len
    w = case["window"] or kv_len
    n = sum(min(w, kv_len - q_len + i + 1) for i in range(q_len))
    return n, min(kv_len, w + q_len - 1)


def work(case):
    q_len, kv_len = _lengths(case)
    T, page, B = sum(q_len), case["page"], case["B"]
    if case["op"] == "plan":
        width = -(-(case["kv_max"] + case["q_max"]) // page) + 1
        pool = sum(-(-(n + q) // page) for n, q in zip(kv_len, q_len)) + 64
        used = sum(-(-n // page) for n in kv_len)
        state = B * 4 * (3 + 2 + 1 + (1 if case["drop"] or case["ended"] else 0))
        return dict(bytes=state + used * 4 + B * width * 4 + (pool - used) * 4 + pool * 4 + T * 12,
                    flops=T * 8 + B * 16)
    D, Hq, Hk = case["D"], case["Hq"], case["Hk"]
    if case["op"] == "append":
        moved = T * D * ((2 * Hq + 2 * Hk) * 2 + 2 * Hk)
        touched = sum((n - 1) // page - (n - q) // page + 1 for n, q in zip(kv_len, q_len))
        return dict(bytes=moved + T * case["axes"] * 4 + case["R"] * 2 + 2 * D * 4 + touched * (Hk * 8 + 4) + B * 8,
                    flops=T * (Hq + Hk) * D * 7 + T * Hk * D * 4)
    pairs = [_seen(case, q, n) for q, n in zip(q_len, kv_len)]
    keys = sum(p[1] for p in pairs)
    return dict(bytes=T * Hq * (2 * D * 2 + 4) + keys * Hk * D * 2 + keys // page * (Hk * 8 + 4),
                flops=sum(p[0] for p in pairs) * Hq * D * 4)


# ------------------------------------------------------------------ in 64 bits

def _exact_turn(s, x, w):
    case = s["case"]
    x, T, R, il = x.double(), x.shape[0], case["R"], case["interleaved"]
    ang = torch.empty(T, R // 2, dtype=torch.float64, device=x.device)
    p = 0
    for a, n in enumerate(s["sections"]):
        ang[:, p:p + n] = s["positions"][:, a:a + 1].double() * s["inv_freq"][p:p + n].double()
        p += n
    y = x * (x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + EPS).pow(-0.5) * w.double()
    z = torch.complex(y[..., 0:R:2], y[..., 1:R:2]) if il else torch.complex(y[..., :R // 2], y[..., R // 2:R])
    z = z * torch.polar(torch.ones_like(ang), ang)[:, None]                # rotation as a complex product
    if il:
        y[..., 0:R:2], y[..., 1:R:2] = z.real, z.imag
    else:
        y[..., :R // 2], y[..., R // 2:R] = z.real, z.imag
    return y


def _exact_append(s, q_len, kv_len):
    """Codes before their rounding, scales and q."""
    page = s["case"]["page"]
    res = dict(q=_exact_turn(s, s["q"], s["q_weight"]))
    for name, x in (("k", _exact_turn(s, s["k"], s["k_weight"])), ("v", s["v"].double())):
        codes, scales = s[name + "_cache"].double(), s[name + "_scales"].double()
        t = 0
        for b, (n, m) in enumerate(zip(q_len, kv_len)):
            row = s["block_table"][b].tolist()
            at = m - n
            while at < m:                                                  # one page after the other
                end = min(m, (at // page + 1) * page)
                new, pg, slot = x[t:t + end - at], row[at // page], at % page
                top = new.abs().amax((0, 2))
                if slot:
                    was = scales[pg].clone()
                    n2 = torch.ceil(torch.log2(top / (LARGEST * was))).clamp(min=0)
                    scales[pg] = was * 2.0 ** n2
                    codes[pg, :, :slot] *= (was / scales[pg])[:, None, None]
                else:
                    scales[pg] = (top / LARGEST).clamp(min=SCALE_LO)
                codes[pg, :, slot:slot + end - at] = (new / scales[pg][:, None]).transpose(0, 1)
                t += end - at
                at = end
        res[name + "_cache"], res[name + "_scales"] = codes, scales
    return res


def exact(case, seed):
    if case["op"] == "plan":
        return None                                                        # whole numbers
    s = prepare(case, seed)
    q_len, kv_len = _lengths(case)
    page = case["page"]
    if case["op"] == "append":
        if sum(q // page + 2 for q in q_len) > 40000:
            return None
        return _exact_append(s, q_len, kv_len)
    Hq, G = case["Hq"], case["Hq"] // case["Hk"]
    if sum(q * n for q, n in zip(q_len, kv_len)) * Hq * case["D"] > 40e10:
        return None                                                        # over about 20 s in 64 bits
    out = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.empty(s["q"].shape[:2], dtype=torch.float64, device="cuda")
    t = 0
    for b, (n, m) in enumerate(zip(q_len, kv_len)):
        pg = s["block_table"][b][:-(-m // page)].long()
        for h in range(case["Hk"]):
            kk, vv = ((c[:, h].view(torch.uint8)[pg].view(c.dtype).double() * f[pg, h].double()[:, None, None])
                      .reshape(-1, case["D"])[:m]
                      for c, f in ((s["k_cache"], s["k_scales"]), (s["v_cache"], s["v_scales"])))
            for g in range(G):
                for r in range(0, n, 2048):                        # rows of queries at a time
                    q = s["q"][t + r:t + min(n, r + 2048), h * G + g].double()
                    z = q @ kk.T / math.sqrt(case["D"])
                    i = torch.arange(m - n + r, m - n + r + q.shape[0], device="cuda")[:, None]
                    j = torch.arange(m, device="cuda")[None, :]
                    if case["causal"]:
                        z[j > i] = -math.inf
                        if case["window"]:
                            z[j <= i - case["window"]] = -math.inf
                    u = torch.logsumexp(z, -1)
                    lse[t + r:t + r + q.shape[0], h * G + g] = u
                    out[t + r:t + r + q.shape[0], h * G + g] = torch.exp(z - u[:, None]) @ vv
        t += n
    return dict(out=out, lse=lse)
