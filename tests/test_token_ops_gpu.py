"""The token operators against their definitions in FP64 (tests/token_ref.py,
which derives the bounds used here)."""
import numpy as np
import pytest

import token_ref as ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

F16, BF16 = torch.float16, torch.bfloat16


@pytest.fixture(scope="module")
def A():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    from depth_weighted_scatter_gb300 import attention

    return attention


def rand(seed, *shape, dtype=torch.float32, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale).to(dtype).cuda()


def freqs(R, theta=10000.0):
    p = torch.arange(R // 2, dtype=torch.float64)
    return torch.pow(theta, -2 * p / R).float().cuda()


def sections_of(R, axes):
    P = R // 2
    return {1: [P], 2: [P // 2, P - P // 2], 3: [P // 4, P // 4, P - 2 * (P // 4)], 4: [0, 3, P - 4, 1]}[axes]


def positions_of(seed, T, axes, most=5000):
    g = torch.Generator().manual_seed(seed)
    p = torch.randint(0, most, (T, axes), generator=g, dtype=torch.int32)
    return p.cuda()


def within(got, want, tol, what):
    got, want, tol = got.detach().cpu().double(), want.double(), torch.as_tensor(tol, dtype=torch.float64)
    bad = ~((got - want).abs() <= tol) & ~(got == want)
    if bad.any():
        i = bad.nonzero()[0].tolist()
        pytest.fail(f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {i}: {got[tuple(i)]} for "
                    f"{want[tuple(i)]}, bound {tol.expand_as(got)[tuple(i)]}")


# ------------------------------------------------------------------ norms and rotation

NORM_ROPE = [
    # T, Hq, Hk, D, R, axes, interleaved, dtype
    (1, 1, 1, 32, 16, 1, False, F16),
    (1, 32, 8, 128, 128, 1, False, BF16),
    (3, 7, 1, 80, 80, 3, False, F16),
    (5, 5, 3, 96, 48, 2, True, BF16),
    (33, 8, 8, 64, 64, 3, True, F16),
    (257, 9, 2, 256, 256, 1, False, BF16),
    (2500, 3, 1, 40, 32, 4, True, F16),
    (2500, 4, 2, 128, 64, 4, False, F16),
]


def norm_rope_inputs(case, seed=0):
    T, Hq, Hk, D, R, axes, il, dtype = case
    qkv = rand(seed, T, Hq + 2 * Hk, D, dtype=dtype)
    return dict(q=qkv[:, :Hq], k=qkv[:, Hq:Hq + Hk], positions=positions_of(seed + 1, T, axes), inv_freq=freqs(R),
                sections=sections_of(R, axes), q_weight=1 + 0.2 * rand(seed + 2, D), k_weight=1 + 0.2 * rand(seed + 3, D),
                interleaved=il, eps=1e-6)


def call(A, x, **more):
    x = {**x, **more}
    return A.qk_norm_rope(x.pop("q"), x.pop("k"), x.pop("positions"), x.pop("inv_freq"), **x)


@pytest.mark.parametrize("weights", [True, False])
@pytest.mark.parametrize("case", NORM_ROPE, ids=str)
def test_norm_rope_forward(A, case, weights):
    x = norm_rope_inputs(case)
    if not weights:
        x["q_weight"] = x["k_weight"] = None
    got = call(A, x)
    cos, sin = ref.cos_sin(x["positions"], x["inv_freq"], x["sections"])
    for name, y in zip("qk", got):
        want, mag = ref.norm_rope(x[name], x[name + "_weight"], cos, sin, x["interleaved"], x["eps"])
        within(y, want, ref.U[y.dtype] * want.abs() + 2.0 ** -18 * mag + ref.tiny(y.dtype), name)


@pytest.mark.parametrize("weights", ["both", "q", "none"])
@pytest.mark.parametrize("case", NORM_ROPE, ids=str)
def test_norm_rope_backward(A, case, weights):
    T, Hq, Hk, D, R, axes, il, dtype = case
    x = norm_rope_inputs(case, seed=10)
    if weights != "both":
        x["k_weight"] = None
    if weights == "none":
        x["q_weight"] = None
    dy = dict(q=rand(20, T, Hq, D, dtype=dtype), k=rand(21, Hk, T, D, dtype=dtype).transpose(0, 1))
    args = {k: v for k, v in x.items() if k not in ("q", "k", "positions", "inv_freq")}
    got = A.qk_norm_rope_backward(dy["q"], dy["k"], x["q"], x["k"], x["positions"], x["inv_freq"], **args)
    again = A.qk_norm_rope_backward(dy["q"], dy["k"], x["q"], x["k"], x["positions"], x["inv_freq"], **args)
    cos, sin = ref.cos_sin(x["positions"], x["inv_freq"], x["sections"])
    for i, name in enumerate("qk"):
        dx, mag, dw, dw_mag = ref.norm_rope_back(dy[name], x[name], x[name + "_weight"], cos, sin, il, x["eps"])
        within(got[i], dx, ref.U[dtype] * dx.abs() + 2.0 ** -16 * mag + ref.tiny(dtype), "d" + name)
        assert torch.equal(got[i], again[i])
        if dw is None:
            assert got[2 + i] is None
        else:
            within(got[2 + i], dw, 2.0 ** -16 * dw_mag, "d" + name + "_weight")
            assert torch.equal(got[2 + i], again[2 + i])


@pytest.mark.parametrize("case", [NORM_ROPE[2], NORM_ROPE[3]], ids=str)
def test_norm_rope_backward_against_differences(A, case):
    """The directional derivative of <dy, forward> by central differences of the FP64 forward, against the kernel's
    gradients.  The step's own error is below 1e-7 of the terms; the gradients' bound is their elements' bound."""
    T, Hq, Hk, D, R, axes, il, dtype = case
    x = norm_rope_inputs(case, seed=30)
    dy = dict(q=rand(31, T, Hq, D, dtype=dtype), k=rand(32, T, Hk, D, dtype=dtype))
    args = {k: v for k, v in x.items() if k not in ("q", "k", "positions", "inv_freq")}
    got = A.qk_norm_rope_backward(dy["q"], dy["k"], x["q"], x["k"], x["positions"], x["inv_freq"], **args)
    cos, sin = ref.cos_sin(x["positions"], x["inv_freq"], x["sections"])
    for i, name in enumerate("qk"):
        x0, w0, g = x[name].cpu().double(), x[name + "_weight"].cpu().double(), dy[name].cpu().double()
        vx, vw = (torch.randn(s, generator=torch.Generator().manual_seed(33 + i), dtype=torch.float64)
                  for s in (x0.shape, w0.shape))

        def loss(e, ex, ew):
            return float((ref.norm_rope(x0 + e * ex * vx, w0 + e * ew * vw, cos, sin, il, x["eps"])[0] * g).sum())

        _, mag, _, dw_mag = ref.norm_rope_back(g, x0, w0, cos, sin, il, x["eps"])
        e = 1e-5
        slope = (loss(e, 1, 0) - loss(-e, 1, 0)) / (2 * e)
        dx = got[i].cpu().double()
        tol = ((ref.U[dtype] * dx.abs() + 2.0 ** -16 * mag + ref.tiny(dtype)) * vx.abs()).sum() + 1e-7 * (mag * vx.abs()).sum()
        assert abs(slope - float((dx * vx).sum())) <= float(tol)
        slope = (loss(e, 0, 1) - loss(-e, 0, 1)) / (2 * e)
        tol = 2.0 ** -16 * (dw_mag * vw.abs()).sum()
        assert abs(slope - float((got[2 + i].cpu().double() * vw).sum())) <= float(tol)


@pytest.mark.parametrize("il", [False, True])
def test_norm_rope_far_and_negative_positions(A, il):
    """Every int32 position turns by its exact angle, to the accuracy of near ones."""
    pos = torch.tensor([0, 1, -1, 131071, 16777217, -16777217, 2 ** 31 - 1, -2 ** 31, 99999999], dtype=torch.int32).cuda()
    T = pos.numel()
    x = norm_rope_inputs((T, 2, 1, 64, 64, 1, il, F16), seed=40)
    x["positions"] = pos
    x["inv_freq"] = torch.cat([freqs(64)[:29], torch.tensor([7.5, -0.25, 6.2831855]).cuda()])
    got = call(A, x)
    cos, sin = ref.cos_sin(pos, x["inv_freq"], x["sections"])
    for name, y in zip("qk", got):
        want, mag = ref.norm_rope(x[name], x[name + "_weight"], cos, sin, il, x["eps"])
        within(y, want, ref.U[F16] * want.abs() + 2.0 ** -18 * mag + ref.tiny(F16), name)


@pytest.mark.parametrize("case", [NORM_ROPE[1], NORM_ROPE[7]], ids=str)
def test_norm_rope_in_place_and_other_stream(A, case):
    x = norm_rope_inputs(case, seed=50)
    want = call(A, x)
    y = {**x, "q": x["q"].clone(), "k": x["k"].clone()}
    got = call(A, y, q_out=y["q"], k_out=y["k"])
    assert got[0].data_ptr() == y["q"].data_ptr()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    on = call(A, x, stream=s)
    s.synchronize()
    by_handle = call(A, x, stream=s.cuda_stream)
    torch.cuda.synchronize()
    for a, b, c, d in zip(want, got, on, by_handle):
        assert torch.equal(a, b) and torch.equal(a, c) and torch.equal(a, d)


def test_norm_rope_rows_of_zeros_and_special_values(A):
    """A zero row stays zero through eps; an infinity or NaN stays in its own row."""
    case = (4, 2, 2, 64, 32, 1, False, BF16)
    x = norm_rope_inputs(case, seed=60)
    base = call(A, x)
    q = x["q"].clone()
    q[1] = 0
    q[2, 0, 63] = float("inf")
    q[3, 1, 5] = float("nan")
    got, _ = call(A, x, q=q)
    assert torch.equal(got[0], base[0][0]) and not got[1].any()
    assert torch.equal(got[2, 1], base[0][2, 1]) and torch.equal(got[3, 0], base[0][3, 0])
    assert got[3, 1].isnan().all()
    turned, _ = call(A, x, q=q, q_weight=None)             # without a norm an unturned infinity is one element
    assert turned[2, 0, 63] == float("inf") and turned[2, 0, :63].isfinite().all()


def test_norm_rope_no_tokens(A):
    x = norm_rope_inputs((0, 2, 1, 64, 64, 1, False, F16))
    q, k = call(A, x)
    assert q.shape == (0, 2, 64) and k.shape == (0, 1, 64)
    args = {k: v for k, v in x.items() if k not in ("q", "k", "positions", "inv_freq")}
    dq, dk, dqw, dkw = A.qk_norm_rope_backward(q, k, x["q"], x["k"], x["positions"], x["inv_freq"], **args)
    assert dq.shape == q.shape and not dqw.any() and not dkw.any()


# ------------------------------------------------------------------ paged cache

def make_pages(seed, kv_len, page, Hk, D, dtype, cache, spare=2, token_major=False, fill=1.0):
    """Two caches of random rows and a block table of shuffled pages (-1 past a request's last)."""
    n = [max(1, -(-m // page)) for m in kv_len]
    total = sum(n) + spare
    order = torch.randperm(total, generator=torch.Generator().manual_seed(seed)).to(torch.int32)
    table = torch.full((len(kv_len), max(n)), -1, dtype=torch.int32)
    at = 0
    for b, m in enumerate(n):
        table[b, :m] = order[at:at + m]
        at += m
    shape = (total, page, Hk, D) if token_major else (total, Hk, page, D)
    pools = []
    for i in range(2):
        x = rand(seed + 1 + i, *shape, scale=fill)
        x = (x * 32).clamp(-448, 448).to(torch.float8_e4m3fn) if cache == "e4m3" else x.to(dtype)
        pools.append(x.transpose(1, 2) if token_major else x)
    return pools[0], pools[1], table.cuda()


def i32(x):
    return torch.tensor(x, dtype=torch.int32).cuda()


def cu_of(q_len):
    return i32(np.concatenate([[0], np.cumsum(q_len)]).tolist())


APPEND = [
    # q_len, kv_len, Hq, Hk, D, R, axes, interleaved, dtype, cache, page, token_major
    ([1], [1], 4, 1, 64, 64, 1, False, F16, "same", 16, False),
    ([1, 1, 1], [700, 16, 17], 32, 8, 128, 128, 1, False, BF16, "same", 16, False),
    ([5, 0, 40], [5, 33, 71], 3, 3, 80, 64, 3, True, F16, "e4m3", 32, True),
    ([129, 64], [500, 64], 8, 2, 128, 96, 1, False, BF16, "e4m3", 128, False),
    ([3000, 1], [3001, 257], 2, 2, 64, 64, 3, True, F16, "same", 256, True),
    ([1] * 70, list(range(1, 71)), 0, 2, 256, 256, 2, False, BF16, "same", 64, False),
]


@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("case", APPEND, ids=lambda c: str(c)[:60])
def test_append(A, case, norm):
    q_len, kv_len, Hq, Hk, D, R, axes, il, dtype, cache, page, token_major = case
    T, pad = sum(q_len), 2                                  # two rows past the last request
    kc, vc, table = make_pages(1, kv_len, page, Hk, D, dtype, cache, token_major=token_major)
    qkv = rand(2, T + pad, Hq + 2 * Hk, D, dtype=dtype)
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hk], qkv[:, Hq + Hk:]
    pos, f, sec = positions_of(3, T + pad, axes), freqs(R), sections_of(R, axes)
    w = dict(q_weight=1 + 0.2 * rand(4, D), k_weight=1 + 0.2 * rand(5, D)) if norm else dict(q_weight=None, k_weight=None)
    scales = dict(k_scale=1 / 48.0, v_scale=0.03) if cache == "e4m3" else {}
    raw = lambda c: c.contiguous().view(torch.uint8 if cache == "e4m3" else torch.int16).cpu().clone()  # noqa: E731
    before = raw(kc), raw(vc)
    q_out = A.kv_append(k, v, kc, vc, table, i32(kv_len), cu_of(q_len), pos, f, sections=sec, interleaved=il,
                        q=q if Hq else None, **w, **scales)
    after = raw(kc), raw(vc)
    cos, sin = ref.cos_sin(pos, f, sec)
    if Hq:
        want, mag = ref.norm_rope(q, w["q_weight"], cos, sin, il, 1e-6)
        within(q_out, want, ref.U[dtype] * want.abs() + 2.0 ** -18 * mag + ref.tiny(dtype), "q")
    else:
        assert q_out is None
    want_k, mag_k = ref.norm_rope(k, w["k_weight"], cos, sin, il, 1e-6)
    cu, tb = cu_of(q_len).cpu().numpy(), table.cpu().numpy()
    touched = torch.zeros(kc.shape[0], page, dtype=torch.bool)
    at = [(t, ref.place_of(cu, kv_len, tb, page, kc.shape[0], t)) for t in range(T + pad)]
    at = [(t, p) for t, p in at if p is not None]
    assert len(at) == T
    ts, pg, sl = (torch.tensor(x) for x in ([t for t, _ in at], [p[0] for _, p in at], [p[1] for _, p in at]))
    touched[pg, sl] = True
    for name, got, want, mag, s in (("k", kc, want_k, mag_k, scales.get("k_scale", 1.0)),
                                    ("v", vc, v.cpu().double(), v.cpu().double().abs(), scales.get("v_scale", 1.0))):
        g = got.cpu().float()[pg, :, sl]
        x, m = want[ts] / s, mag[ts] / s
        if cache == "e4m3":
            x = x.clamp(-448, 448)
            within(g, x, torch.maximum(x.abs() * 2.0 ** -4, torch.tensor(2.0 ** -10, dtype=torch.float64)) + 2.0 ** -18 * m, name)
        elif name == "v":
            assert torch.equal(g.double(), x)
        else:
            within(g, x, ref.U[dtype] * x.abs() + 2.0 ** -18 * m + ref.tiny(dtype), name)
    for b, a in zip(before, after):                         # every other slot keeps its bits
        keep = ~touched[:, None, :, None].expand(b.shape)
        assert torch.equal(b[keep], a[keep])


def test_append_skips_places_outside_the_table_and_bad_pages(A):
    """Holes, pages past the pool, places below zero and past the table write nothing and fault nothing."""
    Hk, D, page = 2, 64, 16
    kc, vc, _ = make_pages(1, [160], page, Hk, D, F16, "same")
    n_pages = kc.shape[0]
    table = i32([[0, -1, n_pages, 3], [1, 2, 2 ** 31 - 1, -2 ** 31]])
    q_len, kv_len = [70, 40], [60, 66]                      # request 0 starts at place -10, request 1 ends past page 3
    T = sum(q_len)
    k, v = rand(2, T, Hk, D, dtype=F16), rand(3, T, Hk, D, dtype=F16)
    before = kc.cpu().clone(), vc.cpu().clone()
    A.kv_append(k, v, kc, vc, table, i32(kv_len), cu_of(q_len), positions_of(4, T, 1), freqs(64))
    want = before[1].clone()
    for t in range(T):
        p = ref.place_of([0, 70, 110], kv_len, table.cpu().numpy(), page, n_pages, t)
        if p is not None:
            want[p[0], :, p[1]] = v[t].cpu()
    assert torch.equal(vc.cpu(), want)
    rows = (kc.cpu() != before[0]).any(-1).any(1)
    assert torch.equal(rows, (want != before[1]).any(-1).any(1))


def test_append_e4m3_saturates_and_keeps_nan(A):
    kc, vc, table = make_pages(1, [4], 16, 1, 32, F16, "e4m3")
    v = torch.tensor([[60000.0] * 32, [-60000.0] * 32, [float("nan")] * 32, [float("inf")] * 32], dtype=F16).cuda()[:, None]
    A.kv_append(torch.zeros_like(v), v, kc, vc, table, i32([4]), cu_of([4]), positions_of(2, 4, 1), freqs(32))
    got = vc.float()[int(table[0, 0]), 0, :4]
    assert (got[0] == 448).all() and (got[1] == -448).all() and got[2].isnan().all()
    assert (got[3] == 448).all()


# ------------------------------------------------------------------ attention

ATTEND = [
    # q_len, kv_len, Hq, Hk, D, causal, window, dtype, cache, page, token_major
    ([1], [1], 1, 1, 64, True, 0, F16, "same", 16, False),
    ([1], [777], 8, 8, 64, True, 0, F16, "same", 16, False),
    ([1, 1, 1, 1], [1, 16, 129, 2000], 32, 8, 128, True, 0, BF16, "same", 16, True),
    ([1, 1, 1], [5, 64, 1031], 14, 2, 64, False, 0, BF16, "e4m3", 64, False),
    ([1, 1], [3500, 65], 32, 4, 128, True, 0, F16, "e4m3", 256, True),
    ([2, 4, 3], [300, 4, 90], 28, 4, 128, True, 0, F16, "same", 32, False),
    ([4, 1, 0], [259, 40, 10], 8, 2, 128, True, 50, BF16, "same", 16, False),
    ([1], [600], 4, 4, 64, True, 1, F16, "e4m3", 32, False),
    ([7, 130, 31], [7, 400, 500], 8, 2, 128, True, 0, BF16, "same", 16, False),
    ([129, 20], [129, 300], 7, 7, 64, True, 0, F16, "same", 64, True),
    ([65, 33], [200, 333], 8, 1, 128, True, 0, BF16, "e4m3", 128, False),
    ([50, 90], [300, 100], 6, 3, 64, False, 0, F16, "e4m3", 16, False),
    ([300], [700], 4, 2, 128, True, 100, F16, "same", 128, False),
    ([100, 0, 64], [700, 9, 64], 4, 1, 64, True, 33, BF16, "same", 32, False),
    ([40, 3], [30, 0], 4, 2, 128, True, 0, BF16, "same", 16, False),     # rows before the first key: nothing is seen
    ([5, 40], [0, 0], 4, 2, 64, False, 0, F16, "same", 16, False),
]


def attend_inputs(case, seed=0, pad=0):
    q_len, kv_len, Hq, Hk, D, causal, window, dtype, cache, page, token_major = case
    kc, vc, table = make_pages(seed + 1, kv_len, page, Hk, D, dtype, cache, token_major=token_major)
    x = dict(q=rand(seed, sum(q_len) + pad, Hq, D, dtype=dtype, scale=1.5), k_cache=kc, v_cache=vc, block_table=table,
             kv_len=i32(kv_len), cu_q=cu_of(q_len), max_q_len=max(max(q_len), 1), max_kv_len=max(kv_len), causal=causal,
             window=window)
    if cache == "e4m3":
        x.update(k_scale=1 / 32.0, v_scale=1 / 24.0)
    return x


def attend(A, x, **more):
    x = {**x, **more}
    return A.paged_attention(x.pop("q"), x.pop("k_cache"), x.pop("v_cache"), x.pop("block_table"), x.pop("kv_len"),
                             x.pop("cu_q"), return_lse=True, **x)


def check_attend(A, x, **more):
    out, lse = attend(A, x, **more)
    r = {k: v for k, v in x.items()}
    want, want_lse, tol, lse_tol, done = ref.attention(scale=r.pop("scale", x["q"].shape[2] ** -0.5), **r)
    within(out[done.cuda()], want[done], tol[done], "out")
    within(lse[done.cuda()], want_lse[done], lse_tol[done], "lse")
    return out, lse


@pytest.mark.parametrize("case", ATTEND, ids=lambda c: str(c)[:70])
def test_attention(A, case):
    x = attend_inputs(case)
    out, lse = check_attend(A, x)
    again = attend(A, x)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])
    only = A.paged_attention(x["q"], x["k_cache"], x["v_cache"], x["block_table"], x["kv_len"], x["cu_q"],
                             **{k: v for k, v in x.items() if k not in ("q", "k_cache", "v_cache", "block_table", "kv_len",
                                                                        "cu_q")})
    assert torch.equal(out, only)


def poison(x):
    """NaN (every bit of a code) in each slot that no request's table reaches within its kv_len."""
    live = torch.zeros(x["k_cache"].shape[0], x["k_cache"].shape[2], dtype=torch.bool)
    tb, page = x["block_table"].cpu(), x["k_cache"].shape[2]
    for b, n in enumerate(x["kv_len"].cpu().tolist()):
        for j in range(n):
            live[tb[b, j // page], j % page] = True
    for name in ("k_cache", "v_cache"):
        c = x[name]
        if c.dtype == torch.float8_e4m3fn:
            y = c.view(torch.uint8)
            y.masked_fill_(~live[:, None, :, None].cuda(), 0x7F)
        else:
            c.masked_fill_(~live[:, None, :, None].cuda(), float("nan"))


@pytest.mark.parametrize("case", ATTEND, ids=lambda c: str(c)[:70])
def test_attention_nan_in_unused_slots(A, case):
    x = attend_inputs(case, seed=100)
    poison(x)
    check_attend(A, x)


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("case", [ATTEND[5], ATTEND[6], ATTEND[8], ATTEND[9], ATTEND[12], ATTEND[13]],
                         ids=lambda c: str(c)[:70])
def test_attention_special_values_under_the_mask(A, case, value):
    """A key and value that only later tokens see leave the earlier tokens' results as they are."""
    x = attend_inputs(case, seed=200)
    base = attend(A, x)
    q_len, kv_len, page = case[0], case[1], case[9]
    for b in range(len(q_len)):
        if q_len[b] < 2:
            continue
        j = kv_len[b] - 1                                   # seen by the last token alone
        pg = int(x["block_table"][b, j // page])
        x["k_cache"][pg, :, j % page] = value
        x["v_cache"][pg, :, j % page] = value
    got = attend(A, x)
    cu = np.concatenate([[0], np.cumsum(q_len)])
    for b in range(len(q_len)):
        if q_len[b] >= 2:
            rows = slice(int(cu[b]), int(cu[b + 1]) - 1)
            assert got[0][rows].isfinite().all()
    want, want_lse, tol, lse_tol, done = ref.attention(scale=x["q"].shape[2] ** -0.5, **x)
    keep = done & want.isfinite().all(-1).all(-1)
    within(got[0][keep.cuda()], want[keep], tol[keep], "out")
    within(got[1][keep.cuda()], want_lse[keep], lse_tol[keep], "lse")
    assert base[0].shape == got[0].shape


@pytest.mark.parametrize("case", [ATTEND[2], ATTEND[3], ATTEND[8], ATTEND[11]], ids=lambda c: str(c)[:70])
def test_attention_holes_in_the_table(A, case):
    """Keys on a page that is -1 or past the pool are not seen."""
    x = attend_inputs(case, seed=300)
    n = x["k_cache"].shape[0]
    t = x["block_table"]
    for b, m in enumerate(x["kv_len"].cpu().tolist()):
        used = -(-m // x["k_cache"].shape[2])
        if used >= 2:
            t[b, used // 2] = (-1, n, 2 ** 31 - 1, -2 ** 31)[b % 4]
        else:
            t[b, 0] = -1                                    # nothing left to see
    check_attend(A, x)


@pytest.mark.parametrize("case", [ATTEND[2], ATTEND[8]], ids=lambda c: str(c)[:70])
def test_attention_bounds_cut_and_rows_outside_requests_stay(A, case):
    x = attend_inputs(case, seed=400, pad=3)
    x["max_kv_len"] = 100
    x["max_q_len"] = max(1, max(case[0]) // 2)
    out = torch.full_like(x["q"], 7.0)
    got, _ = check_attend(A, x, out=out)
    *_, done = ref.attention(scale=1.0, **x)
    assert (got[~done.cuda()] == 7.0).all() and int((~done).sum()) >= 3


@pytest.mark.parametrize("case", [ATTEND[1], ATTEND[5], ATTEND[9], ATTEND[10]], ids=lambda c: str(c)[:70])
def test_attention_large_scores(A, case):
    """Scores far apart: one key takes the row; the running maximum rises along the keys, then falls."""
    x = attend_inputs(case, seed=500)
    x["scale"] = 3.0
    check_attend(A, x)


@pytest.mark.parametrize("q_len, G", [(1, 4), (40, 4)])
def test_attention_strided_rows_and_other_stream(A, q_len, G):
    """q and out as slices of wider tensors, head-major, on another stream."""
    Hk, D, page = 2, 128, 16
    kv = 203
    kc, vc, table = make_pages(1, [kv], page, Hk, D, BF16, "same")
    q = rand(5, Hk * G, q_len, D + 8, dtype=BF16)[..., :D].transpose(0, 1)
    x = dict(q=q, k_cache=kc, v_cache=vc, block_table=table, kv_len=i32([kv]), cu_q=cu_of([q_len]), max_q_len=q_len,
             max_kv_len=kv, causal=True, window=0)
    wide = torch.zeros(Hk * G, q_len, 2 * D, dtype=BF16, device="cuda")
    got, _ = check_attend(A, x, out=wide[..., D:].transpose(0, 1))
    assert not wide[..., :D].any()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    on, _ = attend(A, x, stream=s)
    s.synchronize()
    assert torch.equal(on, got)


def test_attention_offsets_past_32_bits(A):
    """A pool whose last pages start past 2^31 elements."""
    Hk, D, page = 2, 128, 256
    n_pages = (1 << 31) // (Hk * D * page) + 5
    kc, vc = (torch.zeros(n_pages, Hk, page, D, dtype=F16, device="cuda") for _ in range(2))
    table = i32([[n_pages - 1, 0, n_pages - 2], [n_pages - 4, n_pages - 3, 1]])
    for c in (kc, vc):
        for p in table.flatten().tolist():
            c[p] = rand(p % 100 + (c is vc), Hk, page, D, dtype=F16)
    k = rand(7, 2, Hk, D, dtype=F16)
    A.kv_append(k, k, kc, vc, table, i32([600, 700]), cu_of([1, 1]), positions_of(8, 2, 1), freqs(D))
    assert torch.equal(vc[n_pages - 2, :, 600 - 512 - 1], k[0]) and torch.equal(vc[1, :, 700 - 512 - 1], k[1])
    small = table.flatten().tolist()
    for q_len in (1, 70):
        q = rand(9, 2 * q_len, 4, D, dtype=F16)
        at = dict(kv_len=i32([600, 700]), cu_q=cu_of([q_len, q_len]), max_q_len=q_len, max_kv_len=700)
        big = A.paged_attention(q, kc, vc, table, **at)
        near = A.paged_attention(q, kc[small].contiguous(), vc[small].contiguous(), i32([[0, 1, 2], [3, 4, 5]]), **at)
        assert torch.equal(big, near)


def test_operators_in_a_graph(A):
    """Append and attention captured once and replayed for the next token: lengths are read on the device."""
    Hq, Hk, D, page, n0, steps = 8, 2, 64, 16, 30, 5
    kc, vc, table = make_pages(1, [64, 64], page, Hk, D, F16, "same")
    kv_len, cu = i32([n0, n0 + 9]), cu_of([1, 1])
    pos, f, w = kv_len.clone(), freqs(D), 1 + 0.1 * rand(2, D)
    qkv = rand(3, steps + 1, 2, Hq + 2 * Hk, D, dtype=F16)
    cur = qkv[0].clone()
    kc2, vc2 = kc.clone(), vc.clone()

    def step(kc, vc):
        q = A.kv_append(cur[:, Hq:Hq + Hk], cur[:, Hq + Hk:], kc, vc, table, kv_len, cu, pos, f, q=cur[:, :Hq], q_weight=w,
                        k_weight=w)
        return A.paged_attention(q, kc, vc, table, kv_len, cu, max_q_len=1, max_kv_len=64)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step(kc2, vc2)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    kv_len.add_(0)
    with torch.cuda.graph(graph):
        y = step(kc, vc)
    for i in range(steps):
        cur.copy_(qkv[i])
        if i:
            kv_len.add_(1)
            pos.add_(1)
        graph.replay()
        want = step(kc2, vc2)
        assert torch.equal(y, want)
    assert torch.equal(kc, kc2) and torch.equal(vc, vc2)


MANY = [
    # q_len, kv_len, Hq, Hk, D, causal, window, dtype, cache, page, token_major: several hundred row tiles and chunks
    ([700, 1300, 64, 900, 1111], [700, 1500, 4000, 901, 3333], 16, 16, 64, True, 0, F16, "same", 16, False),
    ([700, 1300, 64, 900, 1111], [700, 1500, 4000, 901, 3333], 16, 8, 128, True, 0, BF16, "same", 64, False),
    ([1300, 500, 1200], [2000, 3000, 1201], 12, 12, 64, False, 0, BF16, "e4m3", 64, True),
    ([1300, 500, 1200], [2000, 3000, 1201], 16, 8, 128, True, 600, F16, "e4m3", 32, False),
    ([300] * 9, [20000, 300, 5000, 9000, 301, 12000, 700, 16000, 8000], 4, 1, 64, True, 0, F16, "same", 128, False),
    ([90] * 12, [9000 - 700 * i for i in range(12)], 4, 2, 128, True, 0, BF16, "e4m3", 16, False),
    ([1] * 150, [1 + 37 * i for i in range(150)], 8, 4, 128, True, 0, BF16, "same", 16, False),
]


@pytest.mark.parametrize("case", MANY, ids=lambda c: str(c)[:70])
def test_attention_many_tiles(A, case):
    """More row tiles and chunks than the GPU has SMs; rows drawn from all over are held to their definition, and
    nothing that the call leaves changes when it is made again."""
    q_len, kv_len, Hq, Hk, D, causal, window, dtype, cache, page, _ = case
    x = attend_inputs(case, seed=600)
    poison(x)
    out, lse = attend(A, x)
    again = attend(A, x)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])
    assert out.isfinite().all() and lse.isfinite().all()
    ks, vs = x.get("k_scale", 1.0), x.get("v_scale", 1.0)
    u, cu, rng = ref.U[dtype], np.concatenate([[0], np.cumsum(q_len)]), np.random.default_rng(7)
    for b, (n, m) in enumerate(zip(q_len, kv_len)):
        pg = x["block_table"][b, :-(-m // page)].long()
        for i in sorted({0, n - 1, n // 2, *rng.integers(0, n, 5).tolist()}):
            pos = m - n + i
            hi, lo = (pos + 1 if causal else m), (max(0, pos - window + 1) if window else 0)
            for h in {0, Hk - 1, int(rng.integers(0, Hk))}:
                k, v = (c.float()[pg, h].reshape(-1, D)[lo:hi].double() * f if cache != "e4m3" else
                        c.view(torch.uint8)[pg, h].view(c.dtype).float().reshape(-1, D)[lo:hi].double() * f
                        for c, f in ((x["k_cache"], ks), (x["v_cache"], vs)))
                rows = slice(h * (Hq // Hk), (h + 1) * (Hq // Hk))
                q = x["q"][cu[b] + i, rows].double()
                z = q @ k.T * D ** -0.5
                d = (D + 8) * 2.0 ** -23 * D ** -0.5 * (q.abs() @ k.abs().T).max(-1).values
                want = torch.logsumexp(z, -1)
                p = torch.exp(z - want[:, None])
                o, mag = p @ v, p @ v.abs()
                sub = 2.0 ** -24 * v.abs().sum(0)[None] if dtype == F16 else 0.0
                within(out[cu[b] + i, rows], o.cpu(), ((u + 2 * d[:, None] + 2.0 ** -18) * mag + sub + u * o.abs()
                                                       + ref.tiny(dtype)).cpu(), f"out {b} {i} {h}")
                within(lse[cu[b] + i, rows], want.cpu(), (d + 2.0 ** -18 + 2.0 ** -22 * want.abs()).cpu(), "lse")
    assert A.bevpool_attention_timeouts() == 0


@pytest.mark.parametrize("page, D, dtype, cache, token_major", [(256, 128, BF16, "same", True), (256, 64, F16, "same", False),
                                                                (16, 64, BF16, "same", True), (32, 128, F16, "same", True),
                                                                (256, 128, F16, "e4m3", True)])
def test_attention_page_sizes_and_layouts(A, page, D, dtype, cache, token_major):
    """Many query rows over pages above and below a block, in either memory order, with holes among them."""
    case = ([70, 33], [700, 290], 6, 2, D, True, 0, dtype, cache, page, token_major)
    x = attend_inputs(case, seed=700)
    poison(x)
    check_attend(A, x)
    x["block_table"][0, 1] = -1
    check_attend(A, x)


@pytest.mark.parametrize("q_len", [1, 40])
@pytest.mark.parametrize("cache", ["same", "e4m3"])
@pytest.mark.parametrize("power", [60, -60])
def test_attention_query_magnitudes(A, q_len, cache, power):
    """bf16 queries far from 1 give the same attention when the scale takes their magnitude back."""
    case = ([q_len] * 2, [90, 200], 4, 1, 128, True, 0, BF16, cache, 16, False)
    x = attend_inputs(case, seed=800)
    x["q"] = x["q"] * 2.0 ** power
    x["scale"] = 128 ** -0.5 * 2.0 ** -power
    check_attend(A, x)


def test_append_and_attention_of_one_request_among_empty_ones(A):
    """Requests without tokens between others: their neighbours' rows are their own."""
    q_len, kv_len = [0, 3, 0, 0, 40, 0], [7, 50, 0, 9, 40, 1]
    case = (q_len, kv_len, 4, 2, 64, True, 0, F16, "same", 16, False)
    x = attend_inputs(case, seed=900)
    k, v = rand(901, 43, 2, 64, dtype=F16), rand(902, 43, 2, 64, dtype=F16)
    A.kv_append(k, v, x["k_cache"], x["v_cache"], x["block_table"], x["kv_len"], x["cu_q"], positions_of(903, 43, 1), freqs(64))
    tb = x["block_table"].cpu()
    for t, (b, place) in {0: (1, 47), 2: (1, 49), 3: (4, 0), 42: (4, 39)}.items():
        assert torch.equal(x["v_cache"][tb[b, place // 16], :, place % 16], v[t])
    check_attend(A, x)


# Long calls of few row tiles, their keys cut into chunks.
CHUNKED = [
    # q_len, kv_len, Hq, Hk, D, causal, window, dtype, cache, page, token_major
    ([300], [5000], 8, 2, 128, True, 0, BF16, "same", 16, False),                       # few tiles cut many times
    ([64], [20000], 4, 1, 64, False, 0, F16, "e4m3", 64, True),                         # one tile
    ([257, 0, 1, 900, 33], [1100, 1300, 1, 900, 4000], 8, 4, 64, True, 0, F16, "same", 32, True),
    ([257, 0, 1, 900, 33], [1100, 1300, 1, 900, 4000], 8, 4, 128, False, 0, BF16, "e4m3", 16, False),
    ([700, 1300], [3000, 1300], 16, 8, 64, True, 500, BF16, "same", 128, False),        # windows
    ([400] * 9, [1500, 0, 1025, 1, 90, 1400, 128, 129, 1279], 6, 3, 128, False, 0, F16, "same", 16, True),  # requests without keys
    ([1] * 40 + [600], [2000] * 41, 16, 4, 64, True, 0, BF16, "e4m3", 16, False),       # rows far below the longest
    ([50, 60], [1200, 1100], 12, 3, 128, True, 40, F16, "e4m3", 256, True),
    ([1500, 20], [1200, 1100], 8, 8, 64, True, 0, F16, "same", 16, False),              # more new tokens than keys
]


@pytest.mark.parametrize("case", CHUNKED, ids=[str(i) for i in range(len(CHUNKED))])
def test_attention_chunked_tiles(A, case):
    x = attend_inputs(case, seed=1000 + CHUNKED.index(case))
    poison(x)
    check_attend(A, x)


# Calls whose row tiles are shared out among CTAs: pieces of tiles, whole tiles and tiles that see nothing in one CTA.
SHARED = [
    ([1030, 0, 1, 300, 40], [3000, 7, 1, 300, 2990], 8, 8, 64, True, 0, F16, "same", 32, True),
    ([1030, 0, 1, 300, 40], [3300, 7, 1, 300, 2990], 8, 8, 128, False, 0, BF16, "e4m3", 16, False),
    ([300, 300, 300, 5, 5], [3500, 3400, 0, 128, 3500], 32, 8, 128, True, 0, BF16, "same", 16, True),    # one without keys
    ([2100, 10], [5000, 4900], 10, 10, 64, True, 0, BF16, "e4m3", 64, False),
    ([700, 1300], [4000, 3500], 32, 16, 64, True, 2200, BF16, "same", 128, False),                      # windows
    ([40] * 100, [7000] + [300] * 99, 4, 1, 64, True, 0, F16, "e4m3", 16, False),                       # one far longer
    ([1100] * 4, [3500, 900, 1099, 600], 10, 10, 64, True, 0, F16, "same", 256, True),                  # more tokens than keys
]


def shares(A, case):
    """Whether the call's workspace is that of shared tiles."""
    q_len, kv_len, Hq, Hk, D, _, window = case[:7]
    size = A.bevpool_paged_attention_workspace_size(len(q_len), sum(q_len), Hq, Hk, D, max(q_len), max(kv_len), window)
    tiles = -(-max(q_len) * (Hq // Hk) // 256) * Hk * len(q_len)
    return size == 152 * 512 * (D + 2) * 4 + tiles * 8


@pytest.mark.parametrize("case", SHARED, ids=[str(i) for i in range(len(SHARED))])
def test_attention_shared_tiles(A, case):
    assert shares(A, case)
    x = attend_inputs(case, seed=1300 + SHARED.index(case))
    poison(x)
    check_attend(A, x)


def test_attention_shared_tiles_repeat(A):
    """The same call gives the same bits, also beside another one on another stream."""
    x = attend_inputs(SHARED[2], seed=1100)
    y = attend_inputs(SHARED[3], seed=1101)

    def run(x):
        return attend(A, x)[0]

    first = run(x)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        for _ in range(3):
            run(y)
    again = [run(x) for _ in range(3)]
    torch.cuda.synchronize()
    for o in again:
        assert torch.equal(first, o)


def test_attention_shared_tiles_non_finite(A):
    """Infinities and NaN among keys that some rows of a shared tile see and others do not."""
    case = SHARED[0]
    assert shares(A, case)
    x = attend_inputs(case, seed=1200)
    for j, value in ((2500, float("inf")), (2900, float("nan"))):
        x["v_cache"][int(x["block_table"][0, j // 32]), :, j % 32] = value
    out, lse = attend(A, x)
    want, want_lse, tol, lse_tol, done = ref.attention(scale=64 ** -0.5, **x)
    assert torch.equal(out.isnan().cpu(), want.isnan()) and torch.equal(out.isinf().cpu(), want.isinf())
    fine = want.isfinite().all(-1).all(-1)
    assert int(fine.sum()) == 530 + 1 + 300 + 40
    within(out[fine.cuda()], want[fine], tol[fine], "out")
    within(lse[done.cuda()], want_lse[done], lse_tol[done], "lse")


@pytest.mark.parametrize("causal", [True, False])
def test_attention_whole_prompts(A, causal):
    """The same sizes, causal and not: tiles of all lengths and tiles that are alike are laid out differently."""
    case = ([2100], [2100], 20, 20, 64, causal, 0, BF16, "same", 16, False)
    assert shares(A, case)
    x = attend_inputs(case, seed=1400)
    poison(x)
    check_attend(A, x)
