"""Attention over a cache with page scales against its definition (tests/scaled_ref.py)."""
import numpy as np
import pytest

import scaled_ref as sref
import token_ref as ref
from test_token_ops_gpu import ATTEND, CHUNKED, MANY, SHARED, attend_inputs, cu_of, freqs, i32, poison, positions_of, rand, shares, within

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

F16, BF16 = torch.float16, torch.bfloat16


@pytest.fixture(scope="module")
def A():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    from depth_weighted_scatter_gb300 import attention

    return attention


def coded(case):
    return case[:8] + ("e4m3",) + case[9:]


def inputs(case, seed=0, pad=0, spread=1.5):
    x = attend_inputs(coded(case), seed=seed, pad=pad)
    del x["k_scale"], x["v_scale"]
    n, Hk = x["k_cache"].shape[:2]
    # keys' pages differ so that scores stay of the order of 1, values' by a factor of exp(spread) and more
    x["k_scales"] = torch.exp(0.4 * rand(seed + 50, n, Hk)) / 32
    x["v_scales"] = torch.exp(spread * rand(seed + 51, n, Hk)) / 24
    return x


NAMES = ("q", "k_cache", "v_cache", "k_scales", "v_scales", "block_table", "kv_len", "cu_q")


def attend(A, x, **more):
    x = {**x, **more}
    args = [x.pop(n) for n in NAMES]
    return A.paged_attention_scaled(*args, return_lse=True, **x)


def check(A, x, **more):
    out, lse = attend(A, x, **more)
    r = dict(x)
    scale = r.pop("scale", x["q"].shape[2] ** -0.5)
    want, want_lse, tol, lse_tol, done = sref.attention(*[r.pop(n) for n in NAMES], scale=scale, **r)
    within(out[done.cuda()], want[done], tol[done], "out")
    within(lse[done.cuda()], want_lse[done], lse_tol[done], "lse")
    return out, lse


def poison_all(x):
    """NaN codes in slots that no request reaches, and NaN, infinite, negative and zero scales on pages without any."""
    poison(x)
    tb, page = x["block_table"].cpu(), x["k_cache"].shape[2]
    used = {int(tb[b, j]) for b, n in enumerate(x["kv_len"].tolist()) for j in range(-(-n // page))}
    bad = [float("nan"), float("inf"), -1.0, 0.0, -float("inf")]
    for i, p in enumerate(sorted(set(range(x["k_cache"].shape[0])) - used)):
        x["k_scales"][p], x["v_scales"][p] = bad[i % 5], bad[(i + 2) % 5]


@pytest.mark.parametrize("case", ATTEND, ids=lambda c: str(c)[:70])
def test_attention(A, case):
    x = inputs(case)
    poison_all(x)
    out, lse = check(A, x)
    again = attend(A, x)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])
    only = A.paged_attention_scaled(*[x[n] for n in NAMES], **{k: v for k, v in x.items() if k not in NAMES})
    assert torch.equal(out, only)


def check_rows(x, out, lse, b, rows):
    """Token i and key head h of request b, in FP64 on the GPU; bounds: scaled_ref, and FP32 chains over the keys as in
    test_token_edges_gpu."""
    cu, kv_len, page, D = x["cu_q"].tolist(), x["kv_len"].tolist(), x["k_cache"].shape[2], x["q"].shape[2]
    G, dtype = x["q"].shape[1] // x["k_cache"].shape[1], x["q"].dtype
    n, m = cu[b + 1] - cu[b], kv_len[b]
    pg = x["block_table"][b, :-(-m // page)].long()
    scale = x.get("scale", D ** -0.5)
    for i, h in rows:
        pos = m - n + i
        hi, lo = (pos + 1 if x["causal"] else m), (max(0, pos - x["window"] + 1) if x["window"] else 0)
        if hi <= lo:                                        # nothing is seen
            assert (out[cu[b] + i, h * G:(h + 1) * G] == 0).all() and (lse[cu[b] + i, h * G:(h + 1) * G] == -float("inf")).all()
            continue
        kc, vc = (x[c].view(torch.uint8)[pg, h].view(x[c].dtype).float().reshape(-1, D)[lo:hi].double() for c in ("k_cache", "v_cache"))
        ks, f = (x[c][pg, h].double().repeat_interleave(page)[lo:hi] for c in ("k_scales", "v_scales"))
        k = kc * ks[:, None]
        r = slice(h * G, (h + 1) * G)
        q = x["q"][cu[b] + i, r].double()
        z = q @ k.T * scale
        d = (D + 8) * 2.0 ** -23 * scale * (q.abs() @ k.abs().T).max(-1).values
        d = d + 2.0 ** -22 * 1.4427 * z.abs().max(-1).values + 2.0 ** -22 * f.log2().abs().max()
        want = torch.logsumexp(z, -1)
        p = torch.exp(z - want[:, None])
        o, mag = (p * f) @ vc, (p * f) @ vc.abs()
        sub = 2.0 ** (-32 if dtype == F16 else -38) * vc.abs().sum(0)[None] * (p * f).max(-1, keepdim=True).values
        sums = (hi - lo) / 16 * 2.0 ** -23 + 2.0 ** -18
        u = ref.U[dtype]
        within(out[cu[b] + i, r], o.cpu(), ((u + 2 * d[:, None] + sums) * mag + sub + u * o.abs() + ref.tiny(dtype)).cpu(), f"out {b} {i} {h}")
        within(lse[cu[b] + i, r], want.cpu(), (d + sums + 2.0 ** -22 * want.abs()).cpu(), f"lse {b} {i} {h}")


def sampled(A, x, case, seed):
    """Rows from all over, and the same bits again."""
    poison_all(x)
    out, lse = attend(A, x)
    again = attend(A, x)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])
    assert not out.isnan().any() and not lse.isnan().any()
    rng = np.random.default_rng(seed)
    for b, n in enumerate(case[0]):
        if n:
            check_rows(x, out, lse, b, [(i, int(rng.integers(0, case[3]))) for i in sorted({0, n - 1, n // 2, *rng.integers(0, n, 6).tolist()})])
    assert A.bevpool_attention_timeouts() == 0


@pytest.mark.parametrize("case", CHUNKED + SHARED + MANY, ids=lambda c: str(c)[:70])
def test_many_rows(A, case):
    """Tiles whose keys are cut into chunks, that are shared out among CTAs, more of them than the GPU has SMs."""
    if case in SHARED:
        assert shares(A, coded(case))
    sampled(A, inputs(case, seed=600), case, 7)


FEW, TILES = ([1, 3], [2000, 700], 8, 2, 128, True, 0, BF16, "", 16, False), ([70, 33], [700, 290], 6, 2, 64, True, 0, F16, "", 32, True)


@pytest.mark.parametrize("q_len", [1, 40, 600])
@pytest.mark.parametrize("D, dtype, page", [(64, F16, 64), (128, BF16, 16), (128, F16, 256), (64, BF16, 32)])
def test_uniform_scales_are_those_of_the_plain_cache(A, q_len, D, dtype, page):
    """With one scale for all pages both attentions do the same, but for where the values' scale enters."""
    case = ([q_len, 1], [900, 640], 8, 2, D, True, 0, dtype, "e4m3", page, False)
    x = inputs(case, seed=30)
    x["k_scales"].fill_(1 / 32.0)
    x["v_scales"].fill_(0.25)
    out, lse = check(A, x)
    plain = {k: v for k, v in x.items() if k not in NAMES}
    want, want_lse = A.paged_attention(*[x[n] for n in NAMES if "scales" not in n], k_scale=1 / 32.0, v_scale=0.25, return_lse=True, **plain)
    # weights a power of two apart round alike; the scale of a softmax in progress may differ
    assert torch.allclose(out.float(), want.float(), rtol=4 * ref.U[dtype], atol=ref.U[dtype] * float(want.abs().max()))
    assert torch.allclose(lse, want_lse, rtol=0, atol=1e-4)


@pytest.mark.parametrize("far", [2.0 ** 20, 2.0 ** 44])
@pytest.mark.parametrize("case", [FEW, TILES], ids=["few", "tiles"])
def test_pages_far_apart(A, case, far):
    """Values' scales far apart: the sums are those of the softmax all the same, and a page of small values beside one of
    zeros under a large scale keeps its bits."""
    x = inputs(case, seed=40, spread=0.3)
    page = case[9]
    for b, n in enumerate(case[1]):
        for j in range(-(-n // page)):
            p = int(x["block_table"][b, j])
            x["v_scales"][p] *= (8.0, 8.0 / far, 2.0 ** -6)[j % 3]          # fp16 holds what the largest add up to
    check(A, x)
    for b, n in enumerate(case[1]):                          # the large ones' codes are zeros: small values are all there is
        for j in range(0, -(-n // page), 3):
            x["v_cache"].view(torch.uint8)[int(x["block_table"][b, j])] = 0
    check(A, x)


@pytest.mark.parametrize("case", [FEW, TILES], ids=["few", "tiles"])
def test_scales_outside_their_range(A, case):
    """They count as the nearest bound, NaN as the lower."""
    x = inputs(case, seed=45, spread=0.3)
    x["k_scales"][::5] = 0.0
    x["k_scales"][1::7] = float("nan")
    x["v_scales"][::4] = float("nan")
    x["v_scales"][2::6] = -3.0
    x["v_scales"][3::9] = 2.0 ** -80
    check(A, x)
    y = inputs(case, seed=46)
    y["v_scales"].fill_(float("inf"))
    z = dict(y, v_scales=torch.full_like(y["v_scales"], 2.0 ** 48))
    assert all(torch.equal(a, b) for a, b in zip(attend(A, y), attend(A, z)))


@pytest.mark.parametrize("case", [ATTEND[2], ATTEND[3], ATTEND[8], ATTEND[11]], ids=lambda c: str(c)[:70])
def test_holes_in_the_table(A, case):
    """Keys on a page that is -1 or past the pool are not seen."""
    x = inputs(case, seed=300)
    n, t = x["k_cache"].shape[0], x["block_table"]
    for b, m in enumerate(x["kv_len"].tolist()):
        used = -(-m // x["k_cache"].shape[2])
        t[b, used // 2 if used >= 2 else 0] = (-1, n, 2 ** 31 - 1, -2 ** 31)[b % 4]
    check(A, x)


@pytest.mark.parametrize("case", [ATTEND[5], ATTEND[6], ATTEND[8], ATTEND[9], ATTEND[12], ATTEND[13]], ids=lambda c: str(c)[:70])
def test_nan_under_the_mask(A, case):
    """A key and value of NaN that only later tokens see leave the earlier tokens' results as they are."""
    x = inputs(case, seed=200)
    q_len, kv_len, page = case[0], case[1], case[9]
    for b in range(len(q_len)):
        if q_len[b] >= 2:
            j = kv_len[b] - 1                               # seen by the last token alone
            for c in ("k_cache", "v_cache"):
                x[c].view(torch.uint8)[int(x["block_table"][b, j // page]), :, j % page] = 0x7F
    got = attend(A, x)
    r = dict(x)
    want, want_lse, tol, lse_tol, done = sref.attention(*[r.pop(n) for n in NAMES], scale=x["q"].shape[2] ** -0.5, **r)
    keep = done & want.isfinite().all(-1).all(-1)
    assert int(keep.sum()) >= sum(max(n - 1, 0) for n in q_len)
    within(got[0][keep.cuda()], want[keep], tol[keep], "out")
    within(got[1][keep.cuda()], want_lse[keep], lse_tol[keep], "lse")
    assert got[0][(done & ~keep).cuda()].isnan().any() or not (done & ~keep).any()


@pytest.mark.parametrize("case", [ATTEND[2], ATTEND[8]], ids=lambda c: str(c)[:70])
def test_bounds_cut_and_rows_outside_requests_stay(A, case):
    x = inputs(case, seed=400, pad=3)
    x["max_kv_len"], x["max_q_len"] = 100, max(1, max(case[0]) // 2)
    got, _ = check(A, x, out=torch.full_like(x["q"], 7.0))
    r = dict(x)
    *_, done = sref.attention(*[r.pop(n) for n in NAMES], scale=1.0, **r)
    assert (got[~done.cuda()] == 7.0).all() and int((~done).sum()) >= 3


@pytest.mark.parametrize("case", [ATTEND[1], ATTEND[5], ATTEND[9], ATTEND[10]], ids=lambda c: str(c)[:70])
def test_large_scores(A, case):
    x = inputs(case, seed=500)
    x["scale"] = 3.0
    check(A, x)


@pytest.mark.parametrize("q_len", [1, 40])
@pytest.mark.parametrize("power", [60, -60])
def test_query_magnitudes(A, q_len, power):
    x = inputs(([q_len] * 2, [90, 200], 4, 1, 128, True, 0, BF16, "", 16, False), seed=800)
    x["q"] = x["q"] * 2.0 ** power
    x["scale"] = 128 ** -0.5 * 2.0 ** -power
    check(A, x)


@pytest.mark.parametrize("page, D, dtype, token_major", [(256, 128, F16, True), (256, 64, BF16, False), (16, 64, BF16, True),
                                                         (32, 128, F16, False), (128, 128, BF16, True)])
def test_page_sizes_and_layouts(A, page, D, dtype, token_major):
    for q_len in ([70, 33], [1, 2]):
        x = inputs((q_len, [700, 290], 6, 2, D, True, 0, dtype, "", page, token_major), seed=700)
        poison_all(x)
        check(A, x)
        x["block_table"][0, 1] = -1
        check(A, x)


def test_caches_past_32_bits(A):
    """Pages whose codes start past 2^32 bytes, and past 2^31 elements."""
    n_pages, Hk, page, D = 2200, 16, 256, 512 // 4
    cache = torch.zeros(n_pages, Hk, page, D, dtype=torch.uint8, device="cuda")
    assert cache.numel() > 2 ** 30
    wide = torch.zeros(n_pages, Hk, 4 * page, D, dtype=torch.uint8, device="cuda")[:, :, :page]     # 4.6 GB apart
    assert wide.stride(0) * (n_pages - 1) > 2 ** 32
    q_len, kv_len = [1, 40], [700, 300]
    pages = [n_pages - 1, 3, n_pages - 2], [n_pages - 3, 1]
    table = i32([list(pages[0]), list(pages[1]) + [-1]])
    small = rand(1, 5, Hk, page, D, scale=30.0).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    where = [*pages[0], *pages[1]]
    for i, p in enumerate(where):
        wide[p] = small[i]
    ks, vs = torch.ones(n_pages, Hk, device="cuda"), torch.ones(n_pages, Hk, device="cuda")
    fs = [torch.exp(0.3 * rand(2 + i, 5, Hk)) / 32 for i in range(2)]
    ks[where], vs[where] = fs[0], fs[1]
    q = rand(5, 41, 16, D, dtype=F16)
    args = dict(max_q_len=40, max_kv_len=700, return_lse=True)
    got = A.paged_attention_scaled(q, wide, wide, ks, vs, table, i32(kv_len), cu_of(q_len), **args)
    near = A.paged_attention_scaled(q, small, small, fs[0].contiguous(), fs[1].contiguous(), i32([[0, 1, 2], [3, 4, -1]]), i32(kv_len), cu_of(q_len), **args)
    assert all(torch.equal(a, b) for a, b in zip(got, near))


@pytest.mark.parametrize("q_len, kv_len", [([1, 1], [9000, 5000]), ([4], [9000]), ([70], [9000])])
def test_workspace_of_the_caller(A, q_len, kv_len):
    """One of the size that is named serves; a smaller one is refused."""
    from depth_weighted_scatter_gb300.bevpool import BevpoolError

    x = inputs((q_len, kv_len, 8, 2, 128, True, 0, BF16, "", 16, False), seed=60)
    size = A.bevpool_paged_attention_scaled_workspace_size(len(q_len), sum(q_len), 8, 2, 128, max(q_len), max(kv_len), 0)
    own = torch.empty(size, dtype=torch.uint8, device="cuda")
    assert all(torch.equal(a, b) for a, b in zip(attend(A, x, workspace=own), attend(A, x)))
    with pytest.raises(BevpoolError):
        attend(A, x, workspace=own[:size - 256])


@pytest.mark.parametrize("q_len, Hq", [([2, 1], 4), ([1, 1], 20), ([40, 1], 4)])
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("value", [float("inf"), float("nan"), 1e38])
def test_queries_that_are_not_finite(A, q_len, Hq, dtype, value):
    """Rows of infinite or NaN queries are NaN, also where queries become codes or fp16; the others are not touched, and the
    largest finite ones serve."""
    if value == 1e38 and dtype == F16:
        value = 65504.0
    x = inputs((q_len, [300, 90], Hq, 2, 64, True, 0, dtype, "", 16, False), seed=70)
    want = attend(A, x)
    x["q"][1, 2, 5] = value
    out, lse = attend(A, x)
    keep = torch.ones(sum(q_len), Hq, dtype=torch.bool)
    keep[1, 2] = False
    assert torch.equal(out[keep.cuda()], want[0][keep.cuda()]) and torch.equal(lse[keep.cuda()], want[1][keep.cuda()])
    if value < 1e39 and value == value:
        # scores of the order of 1: a small scale, and keys' scales near the least
        x["scale"] = 2.0 ** -77 if dtype == BF16 else 2.0 ** -20
        if dtype == BF16:
            x["k_scales"] *= 2.0 ** -42
        check(A, x)
    else:
        assert out[1, 2].isnan().all() and lse[1, 2].isnan()


def test_refusals_on_the_gpu(A):
    from depth_weighted_scatter_gb300.bevpool import BevpoolError

    z = lambda *s, dtype=torch.float16: torch.zeros(*s, dtype=dtype, device="cuda")  # noqa: E731
    f32, u8, i = torch.float32, torch.uint8, torch.int32
    good = dict(q=z(3, 4, 64), k_cache=z(4, 2, 16, 64, dtype=u8), v_cache=z(4, 2, 16, 64, dtype=u8), k_scales=z(4, 2, dtype=f32),
                v_scales=z(4, 2, dtype=f32), block_table=z(3, 2, dtype=i), kv_len=z(3, dtype=i), cu_q=z(4, dtype=i), max_q_len=1, max_kv_len=4)
    assert A.paged_attention_scaled(**good).shape == good["q"].shape
    for bad in [dict(k_scales=z(4, 3, dtype=f32)), dict(v_scales=z(3, 2, dtype=f32)), dict(k_scales=z(4, 2)), dict(v_scales=z(2, 4, dtype=f32).t()),
                dict(v_scales=z(4, 2, dtype=f32).cpu()), dict(k_scales=None), dict(k_cache=z(4, 2, 16, 64), v_cache=z(4, 2, 16, 64)),
                dict(scale=0.0), dict(scale=1e30), dict(window=-1), dict(window=3, causal=False), dict(max_q_len=-1), dict(out=z(3, 4, 64).bfloat16()),
                dict(q=z(3, 3, 64)), dict(workspace=z(1, dtype=u8).cpu())]:
        with pytest.raises(BevpoolError):
            A.paged_attention_scaled(**{**good, **bad})
    with pytest.raises(BevpoolError, match="gradients"):
        A.paged_attention_scaled(**{**good, "v_scales": z(4, 2, dtype=f32).requires_grad_()})
    torch.cuda.synchronize()


# ------------------------------------------------------------------ the operators together

@pytest.mark.parametrize("dtype, D, page", [(BF16, 128, 16), (F16, 64, 32)])
def test_plan_append_attend(A, dtype, D, page):
    """Requests of prompts and single tokens whose pages are planned, filled and read, some of them ended or cut on the way;
    the attention against one over the unrounded keys and values that each request has kept.  A code is within half a step
    of its value: 2^-4 of it, or 2^-10 scales of its page, scales at most twice 1 / 448 of the page's largest; again at each
    growth of a page's scale, whose steps halve each time before: twice that in all."""
    B, Hq, Hk, cap, W = 3, 4, 2, 40, 12
    dev = [i32([0] * B), i32([0] * B), torch.full((B, W), -1, dtype=torch.int32, device="cuda"),
           torch.randperm(cap, generator=torch.Generator().manual_seed(1)).to(torch.int32).cuda(), i32([cap])]
    shape = (cap, Hk, page, D)
    kc, vc = (torch.zeros(shape, dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.zeros(cap, Hk, device="cuda") for _ in range(2))
    f = freqs(D)
    kept = [[torch.zeros(0, Hk, D, dtype=torch.float64)] * 2 for _ in range(B)]
    steps = [([40, 1, 0], None), ([1, 1, 1], None), ([1, 30, 1], [0, 0, 0]), ([1, 1, 17], [1, 0, -1]), ([2, 0, 1], [0, -1, 0]), ([1, 9, 1], None)]
    for step, (q_len, drop) in enumerate(steps):
        T = sum(q_len) + 1                                  # a row of padding
        plan = A.plan_pages(i32(q_len), *dev, page_size=page, n_tokens=T, drop=None if drop is None else i32(drop))
        dev = [plan.kv_len, plan.first, plan.block_table, plan.free_pages, plan.n_free]
        assert plan.missing.item() == 0
        qkv = rand(10 + step, T, Hq + 2 * Hk, D, dtype=dtype)
        k, v = qkv[:, Hq:Hq + Hk], qkv[:, Hq + Hk:]
        q = A.kv_append_scaled(k, v, kc, vc, ks, vs, plan.block_table, plan.kv_len, plan.cu_q, plan.positions, f, q=qkv[:, :Hq])
        lens = plan.kv_len.tolist()
        out, lse = A.paged_attention_scaled(q, kc, vc, ks, vs, plan.block_table, plan.kv_len, plan.cu_q, max_q_len=max(q_len), max_kv_len=W * page,
                                            return_lse=True)
        cos, sin = ref.cos_sin(plan.positions, f, [D // 2])
        kt = ref.norm_rope(k, None, cos, sin, False, 1e-6)[0]
        t = 0
        for b, n in enumerate(q_len):
            had = [x.clone() for x in kept[b]]
            if drop is not None and drop[b]:
                cut = len(had[0]) if drop[b] < 0 else min(drop[b] * page, len(had[0]))
                had = [x[cut:] for x in had]
            kept[b] = [torch.cat([had[0], kt[t:t + n]]), torch.cat([had[1], v[t:t + n].cpu().double()])]
            assert len(kept[b][0]) == lens[b]
            K, V = kept[b]
            for i in range(n):
                m = lens[b] - n + i + 1
                for h in range(Hk):
                    rows = slice(h * (Hq // Hk), (h + 1) * (Hq // Hk))
                    qs = q[t + i, rows].cpu().double()

                    def err(x):                             # of the codes' values, and of the rotation before them
                        top = torch.stack([c.abs().max().expand(len(c)) for c in x[:m, h].split(page)] if m else []).flatten() if m % page == 0 else \
                            torch.cat([c.abs().max().expand(len(c)) for c in x[:lens[b], h].split(page)])[:m]
                        return 2 * torch.maximum(2.0 ** -4 * x[:m, h].abs(), 2.0 ** -10 * top[:, None] / 224) + 2.0 ** -16 * x[:m, h].abs()

                    s = qs @ K[:m, h].T * D ** -0.5
                    ds = (qs.abs() @ err(K).T) * D ** -0.5 + (D + 8) * 2.0 ** -23 * D ** -0.5 * (qs.abs() @ K[:m, h].abs().T)
                    p = torch.softmax(s, -1)
                    grow = torch.exp(ds + ds.amax(-1, keepdim=True)) - 1              # how far a weight may be off, relatively
                    bound = (p * grow) @ (V[:m, h].abs() + err(V)) + p @ err(V) + 2 * ref.U[dtype] * (p @ V[:m, h].abs()) + 2.0 ** -12
                    assert ((out[t + i, rows].cpu().double() - p @ V[:m, h]).abs() <= bound).all(), (step, b, i, h)
                    assert ((lse[t + i, rows].cpu().double() - torch.logsumexp(s, -1)).abs() <= ds.amax(-1) + 2.0 ** -12).all()
            t += n


def test_operators_in_a_graph(A):
    """A decoding step of plan, append and attention captured once and replayed gives what the calls give; two captured
    graphs and their eager calls share nothing."""
    B, Hq, Hk, D, page, cap, W = 5, 8, 2, 64, 16, 60, 10
    f = freqs(D)

    def setup(seed):
        order = torch.randperm(cap, generator=torch.Generator().manual_seed(seed)).to(torch.int32).cuda()
        dev = [i32([0] * B), i32([5] * B), torch.full((B, W), -1, dtype=torch.int32, device="cuda"), order, i32([cap])]
        caches = [torch.zeros(cap, Hk, page, D, dtype=torch.uint8, device="cuda") for _ in range(2)] + [torch.ones(cap, Hk, device="cuda") for _ in range(2)]
        return dev, caches

    def step(dev, caches, q_len, qkv):
        plan = A.plan_pages(q_len, *dev, page_size=page, n_tokens=qkv.shape[0])
        q = A.kv_append_scaled(qkv[:, Hq:Hq + Hk], qkv[:, Hq + Hk:], *caches, plan.block_table, plan.kv_len, plan.cu_q, plan.positions, f, q=qkv[:, :Hq])
        out = A.paged_attention_scaled(q, *caches, plan.block_table, plan.kv_len, plan.cu_q, max_q_len=2, max_kv_len=W * page)
        for old, new in zip(dev, [plan.kv_len, plan.first, plan.block_table, plan.free_pages, plan.n_free]):
            old.copy_(new)
        return out

    q_len = i32([1, 2, 1, 0, 1])
    graphs = []
    for seed in (1, 2):
        dev, caches = setup(seed)
        x = torch.zeros(5, Hq + 2 * Hk, D, dtype=F16, device="cuda")
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step(dev, caches, q_len, x)
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = step(dev, caches, q_len, x)
        fresh_dev, fresh_caches = setup(seed)
        for a, b in zip(dev + caches, fresh_dev + fresh_caches):
            a.copy_(b)
        graphs.append((graph, x, out, dev, caches, fresh_dev, fresh_caches))
    for t in range(25):
        for i, (graph, x, out, *_rest) in enumerate(graphs):
            x.copy_(rand(100 * i + t, *x.shape, dtype=F16))
        for graph, *_rest in graphs:
            graph.replay()
        for i, (graph, x, out, dev, caches, dev2, caches2) in enumerate(graphs):
            want = step(dev2, caches2, q_len, x)
            assert torch.equal(out, want), (t, i)
            for a, b in zip(dev + caches, dev2 + caches2):
                assert torch.equal(a, b), (t, i)
