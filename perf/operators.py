"""Measured cases of the token operators: head norms with rotary positions
(forward and backward), the append to a paged key/value cache, and attention of
new tokens over that cache.

With ``own`` false, ``run`` computes the operators from elementary torch
operations in 32 bits, rounded once at the end; with ``own`` true it calls the
library's entry points (depth_weighted_scatter_gb300.attention).

  norm_rope   q, k -> normed and rotated q, k ("train": the gradients too)
  append      k, v (and q) of new tokens -> rows of the paged cache (and q)
  attend      q of new tokens over the paged cache -> out, lse
"""
import math

import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
EPS = 1e-6
THETA = 10000.0
LEFT_OUT = 3 * 1024      # no length or row width of this size


# ------------------------------------------------------------------ cases

def listed():
    return [
        # One decoding step of four requests: launch latency is what counts.
        dict(name="rope_step", op="norm_rope", train=False, T=4, Hq=32, Hk=8, D=128, R=128, axes=1,
             interleaved=False, dtype="bf16"),
        # A prompt batch of odd length, grouped heads, read out of the fused qkv projection.
        dict(name="rope_prompt", op="norm_rope", train=False, T=20001, Hq=32, Hk=8, D=128, R=128, axes=1,
             interleaved=False, dtype="bf16"),
        # A training step over one 128 x 128 BEV grid: (time, y, x) positions, all heads with keys of their own.
        dict(name="rope_train_bev", op="norm_rope", train=True, T=16384, Hq=8, Hk=8, D=64, R=64, axes=3,
             interleaved=True, dtype="f16"),
        # A training step over packed documents, with a quarter of each head left unrotated.
        dict(name="rope_train_packed", op="norm_rope", train=True, T=32768, Hq=16, Hk=2, D=128, R=96, axes=1,
             interleaved=False, dtype="bf16"),
        # A decoding step of 64 requests: one token each into its own page, q normed and rotated on the way.
        dict(name="append_step", op="append", B=64, q_max=1, kv_max=2000, Hq=32, Hk=8, D=128, R=128, axes=1,
             interleaved=False, dtype="bf16", cache="bf16", page=16),
        # Four cameras' or samples' BEV grids at once into an E4M3 cache.
        dict(name="append_frames", op="append", B=4, q_max=16384, kv_max=16384, Hq=8, Hk=8, D=64, R=64, axes=3,
             interleaved=True, dtype="f16", cache="e4m3", page=64),
        # One request's single token over a short context: the smallest call.
        dict(name="attend_step_one", op="attend", B=1, q_max=1, kv_max=777, Hq=8, Hk=8, D=64, causal=True, window=0,
             dtype="f16", cache="f16", page=16),
        # A decoding step of 64 requests with ragged contexts.
        dict(name="attend_step_batch", op="attend", B=64, q_max=1, kv_max=8192, Hq=32, Hk=8, D=128, causal=True,
             window=0, dtype="bf16", cache="bf16", page=16),
        # Two long contexts in an E4M3 cache: few rows, a long axis.
        dict(name="attend_step_long", op="attend", B=2, q_max=1, kv_max=131072, Hq=32, Hk=8, D=128, causal=True,
             window=0, dtype="bf16", cache="e4m3", page=64),
        # Ragged chunks of prompts over what is cached of each request.
        dict(name="attend_chunks", op="attend", B=6, q_max=500, kv_max=12000, Hq=32, Hk=8, D=128, causal=True,
             window=0, dtype="bf16", cache="bf16", page=16),
        # The 50 x 50 BEV grid of a new frame over itself and four earlier frames, every cell seeing every cell.
        dict(name="attend_frames", op="attend", B=2, q_max=2500, kv_max=12500, Hq=8, Hk=8, D=64, causal=False,
             window=0, dtype="f16", cache="e4m3", page=64),
        # A whole prompt at once.
        dict(name="attend_prompt", op="attend", B=1, q_max=8192, kv_max=8192, Hq=32, Hk=8, D=128, causal=True,
             window=0, dtype="bf16", cache="bf16", page=128),
    ]


def _between(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm; odd ones as likely as even ones."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def _size(rng, lo, hi):
    n = _between(rng, lo, hi)
    return n + 1 if n == LEFT_OUT else n


def draw(rng):
    while True:
        c = _draw(rng)
        if LEFT_OUT not in [n * c["D"] for n in (c["Hq"], c["Hq"] + c["Hk"], c["Hq"] + 2 * c["Hk"])]:
            return c


def _draw(rng):
    op = rng.choice(["norm_rope", "append", "attend", "attend"])
    dtype = rng.choice(["f16", "bf16"])
    Hk = rng.choice([1, 2, 4, 8])
    Hq = Hk * rng.choice([1, 2, 4, 7] if Hk < 8 else [1, 2, 4])
    axes = rng.choice([1, 3])
    if op == "norm_rope":
        D = rng.choice([64, 80, 96, 128, 256])
        R = D if rng.random() < 0.6 else D // 32 * 16
        train = rng.random() < 0.5
        most = 32768 * 18 * 128 // (D * (Hq + Hk)) if train else 20001 * 40 * 128 // (D * (Hq + Hk))
        return dict(op=op, train=train, T=_size(rng, 1, min(50000, most)), Hq=Hq, Hk=Hk, D=D, R=R, axes=axes,
                    interleaved=rng.random() < 0.5, dtype=dtype)
    page = rng.choice([16, 32, 64, 128])
    cache = rng.choice([dtype, dtype, "e4m3"])
    if op == "append":
        D = rng.choice([64, 80, 128])
        B = _size(rng, 1, 64)
        q_max = _size(rng, 1, max(1, min(16384, 65536 * 24 * 64 // (B * D * (Hq + 2 * Hk)))))
        kv_max = _size(rng, q_max, max(q_max, min(q_max + 4000, 65536 // B)))
        return dict(op=op, B=B, q_max=q_max, kv_max=kv_max, Hq=Hq, Hk=Hk, D=D, R=D if D != 80 else 64, axes=axes,
                    interleaved=rng.random() < 0.5, dtype=dtype, cache=cache, page=page)
    D = rng.choice([64, 128])
    causal = rng.random() < 0.75
    window = _size(rng, 64, 4096) if causal and rng.random() < 0.3 else 0
    if rng.random() < 0.5:
        # few new tokens over a cache of up to about 1 GB in 16 bits
        B, q_max = _size(rng, 1, 64), rng.choice([1, 1, 1, 2, 4])
        kv_max = _size(rng, 64, max(64, min(131072, (1 << 28) // (B * Hk * D))))
    else:
        # chunks: rows x keys bounded by the whole prompt's
        B, q_max = _size(rng, 1, 8), _size(rng, 16, 4000)
        most = 32 * 8192 * 8192 // (2 * Hq * B * q_max)
        kv_max = _size(rng, q_max, max(q_max, min(32768, most, (1 << 28) // (B * Hk * D))))
        B = max(1, min(B, 32 * 8192 * 8192 // (Hq * q_max * kv_max)))
    return dict(op=op, B=B, q_max=q_max, kv_max=kv_max, Hq=Hq, Hk=Hk, D=D, causal=causal, window=window, dtype=dtype,
                cache=cache, page=page)


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


def _positions(case, starts, lens):
    """int32 [T, axes]: the index in the request, or (time, y, x) on a BEV grid of 128 columns."""
    at = torch.cat([torch.arange(s, s + n, device="cuda") for s, n in zip(starts, lens)])
    if case["axes"] == 1:
        return at.to(torch.int32)[:, None].contiguous()
    return torch.stack([at // 16384, at % 16384 // 128, at % 128], dim=1).to(torch.int32).contiguous()


def _inv_freq(case):
    p = torch.arange(case["R"] // 2, dtype=torch.float64)
    return torch.pow(THETA, -2.0 * p / case["R"]).to(torch.float32).cuda()


def _rotary(case, g):
    D = case["D"]
    return dict(inv_freq=_inv_freq(case), sections=_sections(case),
                q_weight=1.0 + 0.1 * _randn(g, D), k_weight=1.0 + 0.1 * _randn(g, D))


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    s = dict(case=case)
    D, Hq, Hk, dtype = case["D"], case["Hq"], case["Hk"], DTYPES[case["dtype"]]
    if case["op"] == "norm_rope":
        T = case["T"]
        s.update(_rotary(case, g))
        qkv = _randn(g, T, Hq + 2 * Hk, D, dtype=dtype)        # the fused projection's output
        s.update(q=qkv[:, :Hq], k=qkv[:, Hq:Hq + Hk])
        doc = 4000                                             # packed documents restart their positions
        lens = [min(doc, T - t) for t in range(0, T, doc)] if case["axes"] == 1 else [T]
        s["positions"] = _positions(case, [0] * len(lens), lens)
        if case["train"]:
            s.update(dq_out=_randn(g, T, Hq, D, dtype=dtype), dk_out=_randn(g, T, Hk, D, dtype=dtype))
        return s
    q_len, kv_len = _lengths(case)
    B, page = case["B"], case["page"]
    T = sum(q_len)
    n_pages = [-(-n // page) for n in kv_len]
    total = sum(n_pages)
    order = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    first = torch.tensor([0] + n_pages[:-1]).cumsum(0).cuda()
    col = torch.arange(max(n_pages), device="cuda")[None, :]
    used = col < torch.tensor(n_pages, device="cuda")[:, None]
    table = torch.where(used, order[(first[:, None] + col).clamp(max=total - 1)], torch.full_like(order[:1], -1))
    s.update(block_table=table.contiguous(), kv_len=torch.tensor(kv_len, dtype=torch.int32, device="cuda"),
             cu_q=torch.tensor([0] + q_len).cumsum(0).to(torch.int32).cuda(), max_q_len=max(q_len),
             max_kv_len=max(kv_len), k_scale=1.0, v_scale=1.0)
    if case["cache"] == "e4m3":
        s.update(k_scale=1.0 / 64.0, v_scale=1.0 / 64.0)

    def pool():
        x = _randn(g, total, Hk, page, D, dtype=torch.float16)
        if case["cache"] == "e4m3":
            return (x * 64.0).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
        return x.to(DTYPES[case["cache"]])

    s.update(k_cache=pool(), v_cache=pool())
    if case["op"] == "append":
        s.update(_rotary(case, g))
        qkv = _randn(g, T, Hq + 2 * Hk, D, dtype=dtype)
        s.update(q=qkv[:, :Hq], k=qkv[:, Hq:Hq + Hk], v=qkv[:, Hq + Hk:])
        s["positions"] = _positions(case, [n - q for n, q in zip(kv_len, q_len)], q_len)
    else:
        s["q"] = _randn(g, T, Hq, D, dtype=dtype)
    return s


# ------------------------------------------------------------------ plain forms

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


def _rotate(x, cos, sin, R, interleaved):
    a, b = (x[..., 0:R:2], x[..., 1:R:2]) if interleaved else (x[..., :R // 2], x[..., R // 2:R])
    y0, y1 = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([y0, y1], dim=-1).flatten(-2) if interleaved else torch.cat([y0, y1], dim=-1)
    return torch.cat([turned, x[..., R:]], dim=-1)


def _normed(x, w):
    x = x.float()
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w


def _norm_back(g, x, w):
    """Gradients of _normed for x and w."""
    x = x.float()
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    xh = x * r
    gw = g * w
    return r * (gw - xh * (gw * xh).mean(-1, keepdim=True)), (g * xh).sum((0, 1))


def _plain_norm_rope(s):
    case = s["case"]
    dtype, R, il = DTYPES[case["dtype"]], case["R"], case["interleaved"]
    cos, sin = _cos_sin(s)
    res = dict(q=_rotate(_normed(s["q"], s["q_weight"]), cos, sin, R, il).to(dtype),
               k=_rotate(_normed(s["k"], s["k_weight"]), cos, sin, R, il).to(dtype))
    if case["train"]:
        gq = _rotate(s["dq_out"].float(), cos, -sin, R, il)
        gk = _rotate(s["dk_out"].float(), cos, -sin, R, il)
        dq, res["dq_weight"] = _norm_back(gq, s["q"], s["q_weight"])
        dk, res["dk_weight"] = _norm_back(gk, s["k"], s["k_weight"])
        res["dq"], res["dk"] = dq.to(dtype), dk.to(dtype)
    return res


def _plain_append(s):
    case = s["case"]
    dtype, R, il, page = DTYPES[case["dtype"]], case["R"], case["interleaved"], case["page"]
    cos, sin = _cos_sin(s)
    q = _rotate(_normed(s["q"], s["q_weight"]), cos, sin, R, il).to(dtype)
    k = _rotate(_normed(s["k"], s["k_weight"]), cos, sin, R, il)
    v = s["v"].float()
    cu = s["cu_q"].long()
    t = torch.arange(k.shape[0], device=k.device)
    b = torch.searchsorted(cu[1:], t, right=True)
    at = s["kv_len"].long()[b] - cu[b + 1] + t
    pages = s["block_table"].long()[b, at // page]
    for_cache = [(s["k_cache"], k / s["k_scale"]), (s["v_cache"], v / s["v_scale"])]
    if case["cache"] == "e4m3":
        # float8 tensors take no indexed writes: the codes are written through their bytes
        put = [(c.view(torch.uint8), x.clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8))
               for c, x in for_cache]
    else:
        put = [(c, x.to(c.dtype)) for c, x in for_cache]
    put[0][0][pages, :, at % page] = put[0][1]
    put[1][0][pages, :, at % page] = put[1][1]
    return dict(q=q, k_cache=s["k_cache"], v_cache=s["v_cache"])


def _plain_attend(s):
    case = s["case"]
    B, Hq, Hk, D, page = case["B"], case["Hq"], case["Hk"], case["D"], case["page"]
    G, qm = Hq // Hk, s["max_q_len"]
    cu, kv_len, dev = s["cu_q"].long(), s["kv_len"].long(), s["q"].device
    table = s["block_table"].long().clamp(min=0)

    def rows(cache, scale):        # [B, Hk, L, D]
        # gathered as bytes where the codes are 8 bits wide
        x = cache.view(torch.uint8)[table].view(cache.dtype) if cache.dtype == torch.float8_e4m3fn else cache[table]
        return x.permute(0, 2, 1, 3, 4).reshape(B, Hk, -1, D).float() * scale

    q_len = cu[1:] - cu[:-1]
    i = torch.arange(qm, device=dev)
    take = (cu[:-1, None] + i).clamp(max=s["q"].shape[0] - 1)
    q = s["q"][take].float().view(B, qm, Hk, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hk, G * qm, D)
    sc = (q * (1.0 / math.sqrt(D))) @ rows(s["k_cache"], s["k_scale"]).transpose(-1, -2)
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
    o = (e @ rows(s["v_cache"], s["v_scale"])) / l
    o = o.view(B, Hk, G, qm, D).permute(0, 3, 1, 2, 4).reshape(B, qm, Hq, D)
    lse = (m + l.log()).view(B, Hk, G, qm).permute(0, 3, 1, 2).reshape(B, qm, Hq)
    t = torch.arange(s["q"].shape[0], device=dev)
    b = torch.searchsorted(cu[1:], t, right=True)
    return dict(out=o[b, t - cu[b]].to(s["q"].dtype), lse=lse[b, t - cu[b]].contiguous())


# ------------------------------------------------------------------ one pass

def _own(s):
    from depth_weighted_scatter_gb300 import attention

    case = s["case"]
    if case["op"] == "attend":
        out, lse = attention.paged_attention(
            s["q"], s["k_cache"], s["v_cache"], s["block_table"], s["kv_len"], s["cu_q"], max_q_len=s["max_q_len"],
            max_kv_len=s["max_kv_len"], causal=case["causal"], window=case["window"], k_scale=s["k_scale"],
            v_scale=s["v_scale"], return_lse=True)
        return dict(out=out, lse=lse)
    rot = dict(sections=s["sections"], q_weight=s["q_weight"], k_weight=s["k_weight"], eps=EPS,
               interleaved=case["interleaved"])
    if case["op"] == "append":
        q = attention.kv_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["block_table"], s["kv_len"], s["cu_q"],
                                s["positions"], s["inv_freq"], q=s["q"], k_scale=s["k_scale"], v_scale=s["v_scale"],
                                **rot)
        return dict(q=q, k_cache=s["k_cache"], v_cache=s["v_cache"])
    q, k = attention.qk_norm_rope(s["q"], s["k"], s["positions"], s["inv_freq"], **rot)
    res = dict(q=q, k=k)
    if case["train"]:
        res["dq"], res["dk"], res["dq_weight"], res["dk_weight"] = attention.qk_norm_rope_backward(
            s["dq_out"], s["dk_out"], s["q"], s["k"], s["positions"], s["inv_freq"], **rot)
    return res


def run(state):
    if own:
        return _own(state)
    return {"norm_rope": _plain_norm_rope, "append": _plain_append, "attend": _plain_attend}[state["case"]["op"]](state)


# ------------------------------------------------------------------ what a pass cannot do without

def _seen(case, q_len, kv_len):
    """Keys seen by all new tokens of one request, and the keys that any of them sees."""
    if not case["causal"]:
        return q_len * kv_len, kv_len
    w = case["window"] or kv_len
    n = sum(min(w, kv_len - q_len + i + 1) for i in range(q_len))
    return n, min(kv_len, w + q_len - 1)


def work(case):
    D, Hq, Hk = case["D"], case["Hq"], case["Hk"]
    if case["op"] == "norm_rope":
        T = case["T"]
        x = T * (Hq + Hk) * D * 2
        small = T * case["axes"] * 4 + case["R"] * 2 + 2 * D * 4
        if not case["train"]:
            return dict(bytes=2 * x + small, flops=T * (Hq + Hk) * D * 7)
        return dict(bytes=4 * x + small + 2 * D * 4, flops=T * (Hq + Hk) * D * 25)
    q_len, kv_len = _lengths(case)
    T = sum(q_len)
    cb = 1 if case["cache"] == "e4m3" else 2
    if case["op"] == "append":
        moved = T * D * ((2 * Hq + 2 * Hk) * 2 + 2 * Hk * cb)
        return dict(bytes=moved + T * (case["axes"] * 4 + 4) + case["R"] * 2 + 2 * D * 4,
                    flops=T * (Hq + Hk) * D * 7)
    pairs = [_seen(case, q, n) for q, n in zip(q_len, kv_len)]
    keys = sum(p[1] for p in pairs)
    return dict(bytes=T * Hq * (2 * D * 2 + 4) + keys * Hk * D * 2 * cb + keys // case["page"] * 4,
                flops=sum(p[0] for p in pairs) * Hq * D * 4)


# ------------------------------------------------------------------ in 64 bits

def _exact_turn(x, w, pos, f, sections, R, il, back=None):
    """One tensor [T, H, D] in 64 bits: its normed and rotated rows, or, given the gradient of those, its gradients."""
    x, w, T = x.double(), w.double(), x.shape[0]
    ang = torch.empty(T, R // 2, dtype=torch.float64, device=x.device)
    p = 0
    for a, n in enumerate(sections):
        ang[:, p:p + n] = pos[:, a:a + 1].double() * f[p:p + n].double()
        p += n
    turn = torch.polar(torch.ones_like(ang), ang)[:, None]          # rotation as a complex product
    r = (x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + EPS).pow(-0.5)

    def rotated(y, by):
        z = torch.complex(y[..., 0:R:2], y[..., 1:R:2]) if il else torch.complex(y[..., :R // 2], y[..., R // 2:R])
        z = z * by
        y = y.clone()
        if il:
            y[..., 0:R:2], y[..., 1:R:2] = z.real, z.imag
        else:
            y[..., :R // 2], y[..., R // 2:R] = z.real, z.imag
        return y

    if back is None:
        return rotated(x * r * w, turn)
    g = rotated(back.double(), turn.conj())
    dot = (g * w * x).sum(-1, keepdim=True)
    return r * g * w - r.pow(3) * x * dot / x.shape[-1], torch.einsum("thd,thd,thx->d", g, x, r)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] != "attend":
        at = (s["positions"], s["inv_freq"], s["sections"], case["R"], case["interleaved"])
    if case["op"] == "norm_rope":
        res = dict(q=_exact_turn(s["q"], s["q_weight"], *at), k=_exact_turn(s["k"], s["k_weight"], *at))
        if case["train"]:
            res["dq"], res["dq_weight"] = _exact_turn(s["q"], s["q_weight"], *at, back=s["dq_out"])
            res["dk"], res["dk_weight"] = _exact_turn(s["k"], s["k_weight"], *at, back=s["dk_out"])
        return res
    q_len, kv_len = _lengths(case)
    page = case["page"]
    if case["op"] == "append":
        kc, vc = s["k_cache"].double(), s["v_cache"].double()
        k = _exact_turn(s["k"], s["k_weight"], *at) / s["k_scale"]
        v = s["v"].double() / s["v_scale"]
        if case["cache"] == "e4m3":
            k, v = k.clamp(-448.0, 448.0), v.clamp(-448.0, 448.0)
        t = 0
        for b, (n, m) in enumerate(zip(q_len, kv_len)):
            i = torch.arange(m - n, m, device=k.device)
            pg = s["block_table"][b][i // page].long()
            kc[pg, :, i % page] = k[t:t + n]
            vc[pg, :, i % page] = v[t:t + n]
            t += n
        return dict(q=_exact_turn(s["q"], s["q_weight"], *at), k_cache=kc, v_cache=vc)
    Hq, G = case["Hq"], case["Hq"] // case["Hk"]
    if sum(q * n for q, n in zip(q_len, kv_len)) * Hq * case["D"] > 40e10:
        return None                                                # over about 20 s in 64 bits
    out = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.empty(s["q"].shape[:2], dtype=torch.float64, device="cuda")
    t = 0
    for b, (n, m) in enumerate(zip(q_len, kv_len)):
        pg = s["block_table"][b][:-(-m // page)].long()
        for h in range(case["Hk"]):
            kk, vv = ((c[:, h].view(torch.uint8)[pg].view(c.dtype) if case["cache"] == "e4m3" else c[:, h][pg])
                      .double().reshape(-1, case["D"])[:m] * f
                      for c, f in ((s["k_cache"], s["k_scale"]), (s["v_cache"], s["v_scale"])))
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
