"""The token operators where a call is easy to get wrong: host bounds far above
the lengths on the device, heads that do not fill a step, weights far below the
largest.  Definitions and bounds: tests/token_ref.py."""
import numpy as np
import pytest

import token_ref as ref
from test_token_ops_gpu import MANY, attend, attend_inputs, cu_of, freqs, i32, make_pages, norm_rope_inputs, poison, rand, within

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

F16, BF16 = torch.float16, torch.bfloat16


@pytest.fixture(scope="module")
def A():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    from depth_weighted_scatter_gb300 import attention

    return attention


# ------------------------------------------------------------------ bounds far above the lengths

@pytest.mark.parametrize("case, most", [
    # every request's keys lie in one chunk although the bound makes many: few rows, chunked tiles, shared tiles
    (([1, 1, 1], [60, 5, 33], 8, 2, 128, True, 0, BF16, "same", 16, False), 60000),
    (([2], [64], 4, 1, 64, True, 0, F16, "e4m3", 64, False), 131072),
    (([70, 33], [100, 90], 6, 2, 128, True, 0, BF16, "same", 16, True), 30000),
    (([1100, 1], [128, 0], 8, 8, 64, False, 0, F16, "same", 32, False), 8000),
], ids=["few", "few_e4m3", "chunked", "shared"])
def test_attention_is_done_when_the_next_kernel_reads_it(A, case, most):
    """What comes next in the stream sees the results, call after call."""
    x = attend_inputs(case, seed=2000)
    x["max_kv_len"] = most
    pages = -(-most // case[9])                             # the table has room for the bound; past the lengths there is no page
    x["block_table"] = torch.nn.functional.pad(x["block_table"], (0, pages - x["block_table"].shape[1]), value=-1).contiguous()
    assert A.bevpool_paged_attention_workspace_size(len(case[0]), sum(case[0]), *case[2:5], max(case[0]), most, 0) > 0
    args = (x.pop("q"), x.pop("k_cache"), x.pop("v_cache"), x.pop("block_table"), x.pop("kv_len"), x.pop("cu_q"))
    want, _, tol, _, _ = ref.attention(*args, scale=case[4] ** -0.5, **x)
    out, seen = torch.empty_like(args[0]), []
    for _ in range(200):
        out.fill_(float("nan"))
        A.paged_attention(*args, out=out, **x)
        seen.append(out.clone())
    within(seen[0], want, tol, "out")
    assert all(torch.equal(s, seen[0]) for s in seen)


# ------------------------------------------------------------------ the caller's workspace

def test_workspace_of_the_caller(A):
    """One of the size that is named serves; views that do not own their bytes, and other devices, are refused."""
    from depth_weighted_scatter_gb300.bevpool import BevpoolError

    x = attend_inputs(([1], [3000], 8, 2, 128, True, 0, BF16, "same", 16, False), seed=2100)
    args = (x.pop("q"), x.pop("k_cache"), x.pop("v_cache"), x.pop("block_table"), x.pop("kv_len"), x.pop("cu_q"))
    size = A.bevpool_paged_attention_workspace_size(1, 1, 8, 2, 128, 1, 3000, 0)
    own = torch.empty(size, dtype=torch.uint8, device="cuda")
    assert torch.equal(A.paged_attention(*args, workspace=own, **x), A.paged_attention(*args, **x))
    q, pos = args[0].expand(5, 8, 128), torch.arange(5, dtype=torch.int32, device="cuda")
    f, w = torch.ones(64, device="cuda"), torch.ones(128, device="cuda")
    need = A.bevpool_qk_norm_rope_backward_workspace_size(5, 8, 8, 128)
    own = torch.empty(need, dtype=torch.uint8, device="cuda")
    got = A.qk_norm_rope_backward(q, q, q, q, pos, f, q_weight=w, workspace=own)
    want = A.qk_norm_rope_backward(q, q, q, q, pos, f, q_weight=w)
    assert all(torch.equal(a, b) for a, b in zip(got[:3], want))
    wide = torch.empty(2, size, dtype=torch.uint8, device="cuda")
    for bad in (torch.empty(size, dtype=torch.uint8), wide[:1, :1].expand(1, size), wide[:, :size // 2], own[:1].expand(need)):
        with pytest.raises(BevpoolError, match="workspace"):
            A.paged_attention(*args, workspace=bad, **x)
        with pytest.raises(BevpoolError, match="workspace"):
            A.qk_norm_rope_backward(q, q, q, q, pos, f, q_weight=w, workspace=bad)


# ------------------------------------------------------------------ heads that do not fill a step

@pytest.mark.parametrize("eps", [0.0, 1e-30])
@pytest.mark.parametrize("case", [
    # T, Hq, Hk, D, R, axes, interleaved, dtype: a step holds 32 / (lanes of a row) heads
    (5, 3, 1, 128, 128, 1, False, BF16),
    (700, 7, 1, 128, 96, 2, True, F16),
    (5, 7, 2, 64, 64, 3, True, F16),
    (3000, 5, 1, 64, 32, 1, False, BF16),
    (9, 9, 3, 32, 32, 1, False, F16),
    (9, 4, 2, 80, 80, 1, True, BF16),                       # heads fill the steps, lanes the rows do not
    (4, 3, 1, 256, 256, 1, False, F16),
], ids=str)
def test_norm_rope_backward_without_eps(A, case, eps):
    """Places of a step without a head add nothing to the weights' gradients: no real row is zero, so eps = 0 is as
    good as any."""
    T, Hq, Hk, D, R, axes, il, dtype = case
    x = norm_rope_inputs(case, seed=70)
    x["eps"] = eps
    dy = dict(q=rand(71, T, Hq, D, dtype=dtype), k=rand(72, T, Hk, D, dtype=dtype))
    args = {k: v for k, v in x.items() if k not in ("q", "k", "positions", "inv_freq")}
    got = A.qk_norm_rope_backward(dy["q"], dy["k"], x["q"], x["k"], x["positions"], x["inv_freq"], **args)
    out = A.qk_norm_rope(x["q"], x["k"], x["positions"], x["inv_freq"], **args)
    cos, sin = ref.cos_sin(x["positions"], x["inv_freq"], x["sections"])
    for i, name in enumerate("qk"):
        want, mag = ref.norm_rope(x[name], x[name + "_weight"], cos, sin, il, eps)
        within(out[i], want, ref.U[dtype] * want.abs() + 2.0 ** -18 * mag + ref.tiny(dtype), name)
        dx, mag, dw, dw_mag = ref.norm_rope_back(dy[name], x[name], x[name + "_weight"], cos, sin, il, eps)
        within(got[i], dx, ref.U[dtype] * dx.abs() + 2.0 ** -16 * mag + ref.tiny(dtype), "d" + name)
        within(got[2 + i], dw, 2.0 ** -16 * dw_mag, "d" + name + "_weight")


# ------------------------------------------------------------------ weights far below the largest

def check_rows(x, out, lse, b, i, h):
    """Token i of request b, the query heads of key head h, in FP64 on the GPU (no holes in the table).  The bound is
    token_ref's but for three terms.  fp16 weights carry a factor of 2^7 at least: what subnormal ones lose is 2^-25 of
    2^7 times the largest, 2^-32 of it each.  The sums of n keys are FP32 chains of n / 64 + 16 additions, and products of
    16 keys added up n / 16 times, possibly with truncation: (n / 16) * 2^-23 and 2^-18 cover both."""
    cu, kv_len, page, D = x["cu_q"].tolist(), x["kv_len"].tolist(), x["k_cache"].shape[2], x["q"].shape[2]
    G, dtype = x["q"].shape[1] // x["k_cache"].shape[1], x["q"].dtype
    n, m = cu[b + 1] - cu[b], kv_len[b]
    pos = m - n + i
    hi, lo = (pos + 1 if x["causal"] else m), (max(0, pos - x["window"] + 1) if x["window"] else 0)
    pg = x["block_table"][b, :-(-m // page)].long()

    def keys(c, scale):
        c = c.view(torch.uint8)[pg, h].view(c.dtype) if c.element_size() == 1 else c[pg, h]
        return c.float().reshape(-1, D)[lo:hi].double() * scale

    k, v = keys(x["k_cache"], x.get("k_scale", 1.0)), keys(x["v_cache"], x.get("v_scale", 1.0))
    rows = slice(h * G, (h + 1) * G)
    q = x["q"][cu[b] + i, rows].double()
    scale = x.get("scale", D ** -0.5)
    z = q @ k.T * scale
    d = (D + 8) * 2.0 ** -23 * scale * (q.abs() @ k.abs().T).max(-1).values
    want = torch.logsumexp(z, -1)
    p = torch.exp(z - want[:, None])
    o, mag = p @ v, p @ v.abs()
    sub = 2.0 ** -32 * v.abs().sum(0)[None] * p.max(-1, keepdim=True).values if dtype == F16 else 0.0
    sums = (hi - lo) / 16 * 2.0 ** -23 + 2.0 ** -18
    u = ref.U[dtype]
    within(out[cu[b] + i, rows], o.cpu(), ((u + 2 * d[:, None] + sums) * mag + sub + u * o.abs() + ref.tiny(dtype)).cpu(),
           f"out {b} {i} {h}")
    within(lse[cu[b] + i, rows], want.cpu(), (d + sums + 2.0 ** -22 * want.abs()).cpu(), f"lse {b} {i} {h}")


@pytest.mark.parametrize("tail", ["alike", "spread"])
@pytest.mark.parametrize("case", [
    # q_len, kv_len, Hq, Hk, D, causal, window, dtype, cache, page, token_major
    ([1], [20000], 4, 1, 64, True, 0, F16, "same", 16, False),          # few rows
    ([2, 1], [20000, 9000], 4, 2, 128, True, 0, F16, "e4m3", 64, False),
    ([600] * 8, [5000] * 8, 16, 8, 64, True, 0, F16, "same", 32, False),       # tiles
    ([1300] * 2, [4000] * 2, 16, 16, 128, True, 0, F16, "same", 64, False),
    ([70], [20000], 4, 1, 64, True, 0, F16, "same", 16, False),         # chunked
    ([70], [20000], 4, 1, 128, False, 0, F16, "e4m3", 64, False),
    ([2100, 10], [5000, 4900], 10, 10, 64, True, 0, F16, "e4m3", 64, False),   # shared
    ([1100] * 2, [6000] * 2, 10, 10, 128, False, 0, F16, "same", 64, False),
], ids=[str(i) for i in range(8)])
def test_attention_weights_far_below_the_largest(A, case, tail):
    """The first key takes nearly all of a row's weight and its value is zero: the result is what the others add up to.
    They weigh about 2^-21 each, all alike, or about 2^-26, spread."""
    x = attend_inputs(case, seed=2200)
    kv_len, page, e4m3 = case[1], case[9], case[8] == "e4m3"
    x["scale"] = 0.125
    x["q"][..., 0] = 4.0                                    # a key's first element says what it weighs
    ks, vs = (1 / 12.0, 1 / 32.0) if e4m3 else (1.0, 1.0)
    if e4m3:
        x.update(k_scale=ks, v_scale=vs)
    heights = dict(alike=28.84, spread=36.0)[tail] / ks

    def put(name, fn):
        c = x[name].float()
        fn(c)
        x[name].copy_(c.to(x[name].dtype))

    def keys(c):
        c.mul_(0.0 if tail == "alike" else 0.3)
        c[..., 0] = 0.0
        for b in range(len(kv_len)):
            c[int(x["block_table"][b, 0]), :, 0] = 0.0
            c[int(x["block_table"][b, 0]), :, 0, 0] = heights

    def values(c):
        c.abs_().mul_(0.25).add_(6.0 / vs)
        for b in range(len(kv_len)):
            c[int(x["block_table"][b, 0]), :, 0] = 0.0

    put("k_cache", keys)
    put("v_cache", values)
    out, lse = attend(A, x)
    for b, n in enumerate(case[0]):
        for i in sorted({0, n // 3, n - 1}):
            check_rows(x, out, lse, b, i, (i + b) % case[3])
    assert out[:case[0][0]].abs().amax(-1).amin() > 2.0 ** -13          # sums that fp16 holds to all of its bits


@pytest.mark.parametrize("case", MANY, ids=[str(i) for i in range(len(MANY))])
def test_attention_many_tiles_small_contributions(A, case):
    """The largest calls held to what their own weights can lose: an allowance for subnormal fp16 weights is of the
    largest weight, which is a small part of a sum over thousands of keys."""
    x = attend_inputs(case, seed=2300)
    poison(x)
    out, lse = attend(A, x)
    rng = np.random.default_rng(11)
    for b, n in enumerate(case[0]):
        for i in sorted({0, n - 1, *rng.integers(0, n, 3).tolist()}):
            for h in {0, int(rng.integers(0, case[3]))}:
                check_rows(x, out, lse, b, i, h)


# ------------------------------------------------------------------ tensors that require gradients

def test_gradients_are_not_dropped(A):
    """With grad mode on a tensor that requires gradients is refused, whatever its place; without, it is taken."""
    from depth_weighted_scatter_gb300.bevpool import BevpoolError

    q, k = rand(1, 3, 4, 64, dtype=F16), rand(2, 3, 2, 64, dtype=F16)
    pos, f, w = torch.arange(3, dtype=torch.int32, device="cuda"), torch.ones(32, device="cuda"), torch.ones(64, device="cuda")
    c = rand(3, 4, 2, 16, 64, dtype=F16)
    table, n = torch.zeros(1, 1, dtype=torch.int32, device="cuda"), torch.full((1,), 3, dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 3], dtype=torch.int32, device="cuda")
    want = A.qk_norm_rope(q, k, pos, f, q_weight=w)
    at = dict(max_q_len=3, max_kv_len=3)
    attended = A.paged_attention(q, c, c, table, n, cu, **at)
    for name, args in (("q", (q.clone().requires_grad_(), k, pos, f)), ("inv_freq", (q, k, pos, f.clone().requires_grad_()))):
        with pytest.raises(BevpoolError, match=name + ": gradients"):
            A.qk_norm_rope(*args, q_weight=w)
        with torch.no_grad():
            got = A.qk_norm_rope(*args, q_weight=w)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and not got[0].requires_grad
    g = c.clone().requires_grad_()
    with pytest.raises(BevpoolError, match="v_cache: gradients"):
        A.paged_attention(q, c, g, table, n, cu, **at)
    with torch.no_grad():
        assert torch.equal(A.paged_attention(q, c, g, table, n, cu, **at), attended)


# ------------------------------------------------------------------ E4M3 codes of exact values

def e4m3_of(x):
    """Codes' values of FP64 numbers: nearest, even where halfway, saturating; from the format's definition."""
    a = x.abs().clamp(max=448.0)
    step = torch.exp2(torch.floor(torch.log2(a.clamp(min=2.0 ** -6))) - 3)              # of the code's binade
    return torch.copysign(torch.round(a / step) * step, x)                              # torch.round: halves to even


@pytest.mark.parametrize("k_scale, v_scale", [(63 / 4096, 7 / 4096), (15 / 4096, 61 / 4096), (1 / 64, 2.0), (3e-3, 0.1)])
@pytest.mark.parametrize("il, D, R", [(False, 64, 64), (True, 128, 128), (False, 80, 64)])
def test_append_e4m3_rounds_the_quotient(A, k_scale, v_scale, il, D, R):
    """Keys without norm at position 0 and values are exact, so their codes are those of value / scale, rounded once: a
    value halfway between two codes goes to the even one."""
    T, page = 64, 32
    halves = torch.tensor([(1 + (2 * i + 1) / 16) * 2.0 ** e for i in range(8) for e in range(-6, 8)], dtype=torch.float64)
    kc, vc, table = make_pages(1, [T], page, 2, D, F16, "e4m3")
    x = []
    for seed, scale in ((1, k_scale), (2, v_scale)):
        s = float(torch.tensor(scale, dtype=torch.float32))
        v = rand(seed, T, 2, D, dtype=F16).double().cpu()
        exact = torch.where(torch.rand(T, 2, D, generator=torch.Generator().manual_seed(seed)) < 0.8,
                            (halves * s)[torch.randint(0, len(halves), (T, 2, D), generator=torch.Generator().manual_seed(seed))], v)
        h = exact.half()
        h[0, 0, :4] = torch.tensor([float("inf"), -float("inf"), 65504.0, -0.0], dtype=F16)
        x.append(h.cuda())
    A.kv_append(*x, kc, vc, table, i32([T]), cu_of([T]), torch.zeros(T, dtype=torch.int32, device="cuda"), freqs(R),
                interleaved=il, k_scale=k_scale, v_scale=v_scale)
    pg = table[0].long().cpu()
    ties = 0
    for name, got, h, scale in (("k", kc, x[0], k_scale), ("v", vc, x[1], v_scale)):
        q = h.float().cpu() / torch.tensor(scale, dtype=torch.float32)                  # one rounding
        want = e4m3_of(q.double())
        got = got.float().cpu()[pg].transpose(1, 2).reshape(-1, 2, D)[:T].double()
        if name == "k":                                     # an infinity's partner: inf * 0
            want, got = want[1:], got[1:]
        assert torch.equal(got, want), name
        ties += int(torch.isin(q.double(), halves).sum())
    assert ties > 0 or k_scale == 3e-3


# ------------------------------------------------------------------ caches of one page or one head

@pytest.mark.parametrize("n_pages, Hk, q_len", [(1, 1, 3), (1, 2, 40), (5, 1, 3), (5, 1, 40)])
def test_caches_that_differ_in_the_stride_of_an_axis_of_one_entry(A, n_pages, Hk, q_len):
    """Two caches lie alike where they do along every axis of more than one entry."""
    page, D, n = 64, 64, 60 if n_pages == 1 else 300
    kc, vc = rand(1, n_pages, Hk, page, D, dtype=F16), rand(2, n_pages, Hk, page, D, dtype=F16)
    strides = (vc.stride(0) if n_pages > 1 else 8, vc.stride(1) if Hk > 1 else 40, D, 1)
    v2 = vc.as_strided(vc.shape, strides)                   # the same elements
    assert torch.equal(v2, vc) and v2.stride() != kc.stride()
    q, k = rand(3, q_len, 2 * Hk, D, dtype=F16), rand(4, q_len, Hk, D, dtype=F16)
    table = torch.arange(n_pages, dtype=torch.int32, device="cuda")[None]
    at = (table, i32([n]), cu_of([q_len]))
    want = A.paged_attention(q, kc, vc, *at, max_q_len=q_len, max_kv_len=n)
    assert torch.equal(A.paged_attention(q, kc, v2, *at, max_q_len=q_len, max_kv_len=n), want)
    assert torch.equal(A.paged_attention(q, kc.as_strided(kc.shape, strides), vc, *at, max_q_len=q_len, max_kv_len=n), want)
    pos = torch.arange(q_len, dtype=torch.int32, device="cuda")
    k1, v1 = kc.clone(), vc.clone()
    A.kv_append(k, k, k1, v1, *at, pos, freqs(D))
    A.kv_append(k, k, kc, v2, *at, pos, freqs(D))
    assert torch.equal(kc, k1) and torch.equal(vc, v1)


# ------------------------------------------------------------------ the count of waits that ran out

def test_timeouts_are_counted_to_the_end(A):
    """The count is that of all work enqueued so far, on streams that do not wait for the default one too."""
    x = attend_inputs(([300], [700], 4, 2, 128, True, 0, BF16, "same", 16, False), seed=2500)
    attend(A, x)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(200_000_000)                      # about a tenth of a second
        attend(A, x)
    assert not side.query()
    assert A.bevpool_attention_timeouts() == 0
    assert side.query()
