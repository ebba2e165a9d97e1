"""Attention and append with page scales at their edges: queries of zeros, scales
far apart in tiles of bf16 heads, caches past 32 bits."""
import pytest

import scaled_ref as sref
import token_ref as ref
from test_scaled_attention_gpu import A, BF16, F16, NAMES, attend, check, check_rows, inputs  # noqa: F401
from test_token_ops_gpu import cu_of, freqs, i32, make_pages, positions_of, rand, within

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def least_time(call, n=5):
    """ms of the fastest of n calls, after one."""
    call()
    best = float("inf")
    for _ in range(n):
        start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        start.record()
        call()
        end.record()
        end.synchronize()
        best = min(best, start.elapsed_time(end))
    return best


@pytest.mark.parametrize("power", [None, -100], ids=["zeros", "tiny"])
@pytest.mark.parametrize("D, page, causal", [(128, 16, True), (128, 64, True), (64, 128, True), (64, 16, False)])
def test_padded_rows_take_no_longer(A, D, page, causal, power):  # noqa: F811
    """Rows of zeros (or of next to nothing) over pages of zeros, as a padded prompt's, whose keys have the least scale: the
    mean of the values, in the time of any other rows.  A masked score times a factor that had become 0 would be NaN, and
    such rows are taken again key by key, 32 of a warp one after the other: more than ten times as long."""
    x = inputs(([2000], [2000], 8, 2, D, causal, 0, BF16, "", page, False), seed=900)
    usual = least_time(lambda: attend(A, x))
    x["q"] = torch.zeros_like(x["q"]) if power is None else x["q"] * 2.0 ** power
    x["k_cache"].view(torch.uint8).zero_()
    x["k_scales"].fill_(2.0 ** -48)
    out, lse = attend(A, x)
    check_rows(x, out, lse, 0, [(i, i % 2) for i in (0, 1, 777, 1998, 1999)])
    padded = least_time(lambda: attend(A, x))
    assert padded < 3 * usual, (padded, usual)


@pytest.mark.parametrize("D, page", [(128, 16), (64, 64), (128, 256)])
def test_small_queries_of_large_keys(A, D, page):  # noqa: F811
    """Tiles of bf16 rows of 2^-60 to 2^-110, keys' scales near the largest: scores from 1 down to nothing."""
    x = inputs(([70, 33], [300, 290], 6, 2, D, True, 0, BF16, "", page, False), seed=910)
    power = -60 - torch.arange(x["q"].shape[0], device="cuda") % 51
    x["q"] = (x["q"].float() * torch.exp2(power.float())[:, None, None]).to(BF16)
    x["k_scales"] = (x["k_scales"] * 2.0 ** 51).clamp(max=2.0 ** 48)
    check(A, x)


def token_rows(x, b, i, h, least):
    """(out, bound) of token i of request b under key head h, in FP64.  Bounds as in scaled_ref, the weights being fp16: u =
    2^-11 relatively, and `least` of the largest weight times scale that the token sees below that."""
    cu, kv_len, page, D = x["cu_q"].tolist(), x["kv_len"].tolist(), x["k_cache"].shape[2], x["q"].shape[2]
    G, dtype = x["q"].shape[1] // x["k_cache"].shape[1], x["q"].dtype
    n, m = cu[b + 1] - cu[b], kv_len[b]
    hi = m - n + i + 1
    pg = x["block_table"][b, :-(-m // page)].long()
    kc, code = (x[c].view(torch.uint8)[pg, h].view(torch.float8_e4m3fn).float().reshape(-1, D)[:hi].double() for c in ("k_cache", "v_cache"))
    ks, f = (x[c][pg, h].double().repeat_interleave(page)[:hi] for c in ("k_scales", "v_scales"))
    q = x["q"][cu[b] + i, h * G:(h + 1) * G].double()
    k, scale = kc * ks[:, None], D ** -0.5
    s = q @ k.T * scale
    d = (D + 8) * 2.0 ** -23 * scale * (q.abs() @ k.abs().T).max(-1).values
    d = d + 2.0 ** -22 * 1.4427 * s.abs().max(-1).values + 2.0 ** -22 * f.log2().abs().max()
    w = torch.softmax(s, -1) * f
    o, mag = w @ code, w @ code.abs()
    return o, (2.0 ** -11 + 2 * d[:, None] + 2.0 ** -18) * mag + least * w.max(-1, keepdim=True).values * code.abs().sum(0)[None] \
        + ref.U[dtype] * o.abs() + ref.tiny(dtype)


# more than 16 rows a key head: tiles; 12 and 6: the two few-rows kernels
@pytest.mark.parametrize("far", [20, 24, 28, 30, 33, 36, 44])
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("q_len, D, page", [([70, 33], 64, 32), ([70, 33], 128, 128), ([4, 3], 64, 16), ([2, 1], 128, 64)])
def test_how_far_small_values_last(A, q_len, D, page, dtype, far):  # noqa: F811
    """Values' pages 2^far apart, the large ones' codes zeros: small values are all there is.  They are as exact as others down
    to 2^-21 of the largest weight times scale (few rows: 2^-28), and off by 2^-32 (2^-39) of that one below, whatever the
    heads' type."""
    x = inputs((q_len, [700, 290], 6, 2, D, True, 0, dtype, "", page, False), seed=920, spread=0.3)
    least = 2.0 ** -39 if max(q_len) * 3 <= 16 else 2.0 ** -32
    for b, n in enumerate([700, 290]):
        for j in range(-(-n // page)):
            p = int(x["block_table"][b, j])
            x["v_scales"][p] *= 8.0 if j % 2 == 0 else 8.0 * 2.0 ** -far
            if j % 2 == 0:
                x["v_cache"].view(torch.uint8)[p] = 0
    x["v_scales"] *= 2.0 ** (far // 2)                       # fp16 outputs hold them
    x["v_scales"].clamp_(max=2.0 ** 48)
    out, _ = attend(A, x)
    for b in range(2):
        for i in {0, q_len[b] // 2, q_len[b] - 1}:
            for h in range(2):
                want, tol = token_rows(x, b, i, h, least)
                within(out[int(x["cu_q"][b]) + i, 3 * h:3 * h + 3], want.cpu(), tol.cpu(), f"{b} {i} {h}")


@pytest.mark.parametrize("T, page", [(60, 16), (40000, 64), (40000, 256)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_angles_of_the_append(A, T, page, interleaved):  # noqa: F811
    """cos and sin are off by 2^-20 at most.  Pairs (1, 0) come out as (cos, sin), rounded to fp16: by 2^-11 of them, which
    for those below 2^-10 is half of the bound or less.  (The product of position and frequency, exact but for 2^-53 of
    itself, adds 2^-29 below 2^24 radians.)"""
    D = 64
    seqs = 1 if T > 100 else T                               # few tokens a request: a warp a page and head
    g = torch.Generator().manual_seed(T)
    pos = torch.randint(-(1 << 24), 1 << 24, (T,), generator=g).to(torch.int32).cuda()
    f = torch.rand(D // 2, generator=g).cuda()
    q = torch.zeros(T, 1, D, dtype=F16, device="cuda")
    first, second = (slice(0, D, 2), slice(1, D, 2)) if interleaved else (slice(0, D // 2), slice(D // 2, D))
    q[..., first] = 1.0
    pages = -(-(T // seqs) // page)
    cache = [torch.zeros(seqs * pages, 1, page, D, dtype=torch.uint8, device="cuda") for _ in range(2)]
    scales = [torch.ones(seqs * pages, 1, device="cuda") for _ in range(2)]
    table = torch.arange(seqs * pages, dtype=torch.int32, device="cuda").view(seqs, pages)
    out = A.kv_append_scaled(q, q, *cache, *scales, table, i32([T // seqs] * seqs), cu_of([T // seqs] * seqs), pos, f, q=q, interleaved=interleaved)
    cos, sin = ref.cos_sin(pos, f, [D // 2])
    for got, want in ((out[:, 0, first], cos), (out[:, 0, second], sin)):
        assert T < 100 or int((want.abs() < 2.0 ** -10).sum()) > 500
        within(got, want, 2.0 ** -20 + 2.0 ** -11 * want.abs() + 2.0 ** -25 + 2.0 ** -29, "angles")


@pytest.mark.parametrize("page, D, Hq, Hk", [(128, 64, 8, 8), (256, 64, 3, 2), (128, 128, 32, 8), (256, 128, 5, 1)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_long_pages_in_part_and_whole(A, page, D, Hq, Hk, interleaved):  # noqa: F811
    """Pages of which a call fills a few slots, as many as a group has rows, and all: the first two have their rows on their
    way in shared memory, the last their angles, in one launch."""
    q_len, kv_len = [64, page, 2 * page + 3, 65, 1, 7 * page], [64, page, 3 * page + 1, page + 1, 40, 7 * page]
    T, dtype = sum(q_len), BF16 if D == 128 else F16
    kc, vc, table = make_pages(1, kv_len, page, Hk, D, dtype, "e4m3")
    ks, vs = (torch.exp(rand(8 + i, kc.shape[0], Hk)) / 100 for i in range(2))
    before = [(c.float().cpu().double(), s.cpu().clone()) for c, s in ((kc, ks), (vc, vs))]
    qkv, pos, f, w = rand(2, T, Hq + 2 * Hk, D, dtype=dtype), positions_of(3, T, 1), freqs(D), 1 + 0.2 * rand(4, D)
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hk], qkv[:, Hq + Hk:]
    q_out = A.kv_append_scaled(k, v, kc, vc, ks, vs, table, i32(kv_len), cu_of(q_len), pos, f, interleaved=interleaved, q=q, q_weight=w, k_weight=w)
    cos, sin = ref.cos_sin(pos, f, [D // 2])
    want, mag = ref.norm_rope(q, w, cos, sin, interleaved, 1e-6)
    within(q_out, want, ref.U[dtype] * want.abs() + 2.0 ** -18 * mag + ref.tiny(dtype), "q")
    want_k, mag = ref.norm_rope(k, w, cos, sin, interleaved, 1e-6)
    runs = sref.page_runs(cu_of(q_len).cpu().numpy(), kv_len, table.cpu().numpy(), page, kc.shape[0])
    x = v.cpu().double()
    sref.check_append(runs, want_k, 2.0 ** -18 * mag, *before[0], kc.float().cpu().double(), ks.cpu(), False, "k")
    sref.check_append(runs, x, torch.zeros_like(x), *before[1], vc.float().cpu().double(), vs.cpu(), True, "v")


FAR_PAGES, FAR_HEADS, FAR_PAGE, FAR_D = 2200, 16, 256, 128
FAR = [3, FAR_PAGES - 1, FAR_PAGES - 2, 1, FAR_PAGES - 3]   # pages that the tests use


@pytest.fixture(scope="module")
def far():
    """Caches of codes whose pages are 2 MB apart, the last ones past 2^32 bytes."""
    caches = [torch.zeros(FAR_PAGES, FAR_HEADS, 4 * FAR_PAGE, FAR_D, dtype=torch.uint8, device="cuda")[:, :, :FAR_PAGE] for _ in range(2)]
    assert caches[0].stride(0) * FAR[4] > 2 ** 32
    return caches


def near(seed):
    """Codes and scales of five pages."""
    codes = rand(seed, 5, FAR_HEADS, FAR_PAGE, FAR_D, scale=30.0).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    return codes, torch.exp(0.3 * rand(seed + 1, 5, FAR_HEADS)) / 4000


def placed(far, codes, scales):
    """Those pages in the wide caches, and their scales among all."""
    for cache, c in zip(far, codes):
        for i, p in enumerate(FAR):
            cache[p] = c[i]
    res = [torch.ones(FAR_PAGES, FAR_HEADS, device="cuda") for _ in range(2)]
    for all_, s in zip(res, scales):
        all_[FAR] = s
    return far, res


def table_of(pages):
    return i32([pages[:3], pages[3:] + [-1]])


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("q_len, G", [([1, 3], 1), ([1, 6], 2), ([1, 40], 1)], ids=["codes", "few", "tiles"])
def test_attention_over_pages_past_32_bits(A, far, q_len, G, dtype):  # noqa: F811
    """Each of the three kernels: the bits of the same codes in a small cache."""
    codes, scales = zip(near(1), near(3))
    wide, wide_scales = placed(far, codes, scales)
    q, kv_len = rand(5, sum(q_len), FAR_HEADS * G, FAR_D, dtype=dtype), i32([700, 300])
    args = dict(max_q_len=max(q_len), max_kv_len=700, return_lse=True)
    got = A.paged_attention_scaled(q, *wide, *wide_scales, table_of(FAR), kv_len, cu_of(q_len), **args)
    want = A.paged_attention_scaled(q, *codes, *scales, table_of([0, 1, 2, 3, 4]), kv_len, cu_of(q_len), **args)
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and got[0].abs().amax() > 0


@pytest.mark.parametrize("q_len, kv_len", [([2, 1], [514, 300]), ([200, 20], [700, 290]), ([300, 20], [700, 290])],
                         ids=["tokens", "pages", "pages read twice"])
def test_append_to_pages_past_32_bits(A, far, q_len, kv_len):  # noqa: F811
    """Pages that hold tokens and whose scales grow among them: the codes and scales of the same append to a small cache."""
    T, f, pos = sum(q_len), freqs(FAR_D), positions_of(8, sum(q_len), 1)
    k, v = (rand(6 + i, T, FAR_HEADS, FAR_D, dtype=F16) for i in range(2))
    codes, scales = zip(near(1), near(3))
    wide, wide_scales = placed(far, codes, scales)
    before = [s.clone() for s in scales]
    A.kv_append_scaled(k, v, *wide, *wide_scales, table_of(FAR), i32(kv_len), cu_of(q_len), pos, f)
    A.kv_append_scaled(k, v, *codes, *scales, table_of([0, 1, 2, 3, 4]), i32(kv_len), cu_of(q_len), pos, f)
    for a, b, c, d, was in zip(wide, codes, wide_scales, scales, before):
        assert torch.equal(a[FAR], b) and torch.equal(c[FAR], d)
        assert (d[4] / was[4]).log2().amax() >= 1           # the last page, past 2^32 bytes, holds tokens and has grown
