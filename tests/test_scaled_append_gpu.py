"""The append with page scales against its definition (tests/scaled_ref.py)."""
import pytest

import scaled_ref as sref
import token_ref as ref
from test_token_ops_gpu import cu_of, freqs, i32, make_pages, positions_of, rand, sections_of, within

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

F16, BF16 = torch.float16, torch.bfloat16


@pytest.fixture(scope="module")
def A():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    from depth_weighted_scatter_gb300 import attention

    return attention


def values(cache):
    return cache.float().cpu().double()


def scales_of(seed, n_pages, Hk, spread=1.0):
    return torch.exp(spread * rand(seed, n_pages, Hk)) / 100


CASES = [
    # q_len, kv_len, Hq, Hk, D, R, axes, interleaved, dtype, page, token_major
    ([1], [1], 4, 1, 64, 64, 1, False, F16, 16, False),
    ([1, 1, 1, 1], [700, 16, 17, 33], 32, 8, 128, 128, 1, False, BF16, 16, False),         # a warp a page and head
    ([1, 7, 0, 3, 1, 1], [40, 50, 7, 3, 17, 100], 6, 3, 64, 32, 2, True, BF16, 32, True),
    ([2, 90, 0, 0] + [0] * 40, [40, 95, 7, 0] + [5] * 40, 4, 2, 128, 96, 3, False, F16, 64, False),   # more tokens than a warp's rows
    ([5, 0, 40], [5, 33, 71], 3, 3, 64, 48, 3, True, F16, 32, True),                       # a CTA a page
    ([129, 64], [500, 64], 8, 2, 128, 96, 1, False, BF16, 128, False),                     # pages read twice
    ([300, 513], [301, 700], 2, 1, 128, 128, 1, True, F16, 256, False),
    ([3000, 1], [3001, 257], 2, 2, 64, 64, 3, True, F16, 64, True),
    ([700], [731], 0, 7, 64, 16, 4, False, BF16, 16, False),
    ([40, 33], [30, 20], 4, 1, 64, 64, 1, False, F16, 16, False),                          # places below 0
]


@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("case", CASES, ids=lambda c: str(c)[:60])
def test_append(A, case, norm):
    q_len, kv_len, Hq, Hk, D, R, axes, il, dtype, page, token_major = case
    T, pad = sum(q_len), 3                                  # three rows past the last request
    kc, vc, table = make_pages(1, kv_len, page, Hk, D, dtype, "e4m3", token_major=token_major)
    ks, vs = scales_of(8, kc.shape[0], Hk), scales_of(9, kc.shape[0], Hk)
    qkv = rand(2, T + pad, Hq + 2 * Hk, D, dtype=dtype)
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hk], qkv[:, Hq + Hk:]
    pos, f, sec = positions_of(3, T + pad, axes), freqs(R), sections_of(R, axes)
    w = dict(q_weight=1 + 0.2 * rand(4, D), k_weight=1 + 0.2 * rand(5, D)) if norm else dict(q_weight=None, k_weight=None)
    before = [(values(c), s.cpu().clone()) for c, s in ((kc, ks), (vc, vs))]
    q_out = A.kv_append_scaled(k, v, kc, vc, ks, vs, table, i32(kv_len), cu_of(q_len), pos, f, sections=sec, interleaved=il,
                               q=q if Hq else None, **w)
    cos, sin = ref.cos_sin(pos, f, sec)
    if Hq:
        want, mag = ref.norm_rope(q, w["q_weight"], cos, sin, il, 1e-6)
        within(q_out, want, ref.U[dtype] * want.abs() + 2.0 ** -18 * mag + ref.tiny(dtype), "q")
    else:
        assert q_out is None
    want_k, mag = ref.norm_rope(k, w["k_weight"], cos, sin, il, 1e-6)
    runs = sref.page_runs(cu_of(q_len).cpu().numpy(), kv_len, table.cpu().numpy(), page, kc.shape[0])
    assert runs
    sref.check_append(runs, want_k, 2.0 ** -18 * mag, *before[0], values(kc), ks.cpu(), False, "k")
    x = v.cpu().double()
    sref.check_append(runs, x, torch.zeros_like(x), *before[1], values(vc), vs.cpu(), True, "v")


@pytest.mark.parametrize("many", [False, True])
@pytest.mark.parametrize("old, new", [(1.0, 1.0), (1.0, 1.01), (1.0, 37.0), (1.0, 2.0 ** -9), (2.0 ** -30, 1.0), (0.0, 1.0),
                                      (float("nan"), 1.0), (2.0 ** 60, 1.0), (1.0, 0.0)])
def test_a_page_that_holds_tokens(A, old, new, many):
    """The scale grows by powers of two where it has to, and stays where it holds; old scales outside the range count as its
    bounds; the earlier codes move with it."""
    Hk, D, page = 3, 64, 32
    q_len, kv_len = ([20, 5], [25, 31]) if many else ([2, 1], [7, 32])
    kc, vc, table = make_pages(5, kv_len, page, Hk, D, F16, "e4m3")
    ks, vs = torch.full((kc.shape[0], Hk), old, device="cuda"), torch.full((kc.shape[0], Hk), old, device="cuda")
    T = sum(q_len)
    k, v = (rand(s, T, Hk, D, dtype=F16).clamp(-1, 1) * new * 448 for s in (6, 7))
    k, v = ((x if not new else x.clamp(-65504, 65504)).to(F16) for x in (k, v))
    before = [(values(c), s.cpu().clone().nan_to_num(nan=0.0)) for c, s in ((kc, ks), (vc, vs))]
    A.kv_append_scaled(k, v, kc, vc, ks, vs, table, i32(kv_len), cu_of(q_len), torch.zeros(T, dtype=torch.int32, device="cuda"), freqs(D))
    runs = sref.page_runs(cu_of(q_len).cpu().numpy(), kv_len, table.cpu().numpy(), page, kc.shape[0])
    for x, (c, s), cache, scales, what in ((k, before[0], kc, ks, "k"), (v, before[1], vc, vs, "v")):
        x = x.cpu().double()                                # position 0 turns nothing: exact
        sref.check_append(runs, x, torch.zeros_like(x), c, s, values(cache), scales.cpu().nan_to_num(nan=0.0), True, what)


@pytest.mark.parametrize("many", [False, True])
def test_special_values(A, many):
    """Infinities become +-448 and NaN stays; neither counts in the scale.  Zeros get the least scale."""
    Hk, D, page, T = 2, 128, 64, 40 if many else 2
    kc, vc, table = make_pages(1, [T], page, Hk, D, BF16, "e4m3")
    ks, vs = scales_of(1, kc.shape[0], Hk), scales_of(2, kc.shape[0], Hk)
    v = rand(3, T, Hk, D, dtype=BF16)
    v[0, 0, :3] = torch.tensor([float("inf"), -float("inf"), float("nan")], dtype=BF16)
    v[:, 1] = 0.0
    v[T - 1, 1, 5] = float("nan")
    k = torch.full_like(v, float("nan"))
    k[:, 1] = float("inf")
    A.kv_append_scaled(k, v, kc, vc, ks, vs, table, i32([T]), cu_of([T]), torch.zeros(T, dtype=torch.int32, device="cuda"), freqs(D))
    p = int(table[0, 0])
    got, s = values(vc)[p, :, :T].transpose(0, 1), vs.cpu().double()[p]
    x = v.cpu().double()
    top = torch.where(x[:, 0].isfinite(), x[:, 0].abs(), 0.0).max()
    assert abs(s[0] - top / 448) <= 2.0 ** -24 * s[0] and s[1] == sref.LO
    assert got[0, 0, 0] == 448 and got[0, 0, 1] == -448 and got[0, 0, 2].isnan() and got[T - 1, 1, 5].isnan()
    fin = x.isfinite()
    assert torch.equal(got[fin], sref.e4m3_of((x.float() / s.float()[None, :, None]).double())[fin])
    assert (ks.cpu()[p].double() == sref.LO).all() and values(kc)[p, 0, :T].isnan().all()


def test_values_beyond_the_largest_scale(A):
    """bf16 values past 448 * 2^48 saturate; tiny ones get the least scale."""
    kc, vc, table = make_pages(1, [3], 16, 1, 64, BF16, "e4m3")
    ks, vs = scales_of(1, kc.shape[0], 1), scales_of(2, kc.shape[0], 1)
    k, v = torch.full((3, 1, 64), 1e30, dtype=BF16, device="cuda"), torch.full((3, 1, 64), 1e-30, dtype=BF16, device="cuda")
    A.kv_append_scaled(k, v, kc, vc, ks, vs, table, i32([3]), cu_of([3]), torch.zeros(3, dtype=torch.int32, device="cuda"), freqs(64))
    p = int(table[0, 0])
    assert ks[p, 0] == 2.0 ** 48 and vs[p, 0] == 2.0 ** -48
    assert (values(kc)[p, 0, :3] == 448).all() and (values(vc)[p, 0, :3] == 0).all()


@pytest.mark.parametrize("many", [False, True])
def test_bad_pages_and_places_write_nothing(A, many):
    """Holes, pages past the pool, places below zero and past the table."""
    Hk, D, page = 2, 64, 16
    kc, vc, _ = make_pages(1, [160], page, Hk, D, F16, "e4m3")
    n_pages = kc.shape[0]
    table = i32([[0, -1, n_pages, 3], [1, 2, 2 ** 31 - 1, -2 ** 31]] + [[-1] * 4] * (60 if not many else 0))
    q_len, kv_len = [70, 40] + [0] * (len(table) - 2), [60, 66] + [0] * (len(table) - 2)
    T = sum(q_len)
    k, v, q = rand(2, T, Hk, D, dtype=F16), rand(3, T, Hk, D, dtype=F16), rand(4, T, 3, D, dtype=F16)
    ks, vs = scales_of(1, n_pages, Hk), scales_of(2, n_pages, Hk)
    before = values(vc), vs.cpu().clone()
    pos = positions_of(4, T, 1)
    q_out = A.kv_append_scaled(k, v, kc, vc, ks, vs, table, i32(kv_len), cu_of(q_len), pos, freqs(D), q=q)
    runs = sref.page_runs(cu_of(q_len).cpu().numpy(), kv_len, table.cpu().numpy(), page, n_pages)
    x = v.cpu().double()
    sref.check_append(runs, x, torch.zeros_like(x), *before, values(vc), vs.cpu(), True, "v")
    cos, sin = ref.cos_sin(pos, freqs(D), [D // 2])
    want, mag = ref.norm_rope(q, None, cos, sin, False, 1e-6)
    within(q_out, want, ref.U[F16] * want.abs() + 2.0 ** -18 * mag + ref.tiny(F16), "q")


def test_token_by_token(A):
    """A page filled a token at a time: every token is within half a step of the final scale (and half a step of each
    growth's before) of its value."""
    Hk, D, page, n = 2, 64, 32, 45
    kc, vc, table = make_pages(1, [n], page, Hk, D, BF16, "e4m3")
    ks, vs = scales_of(1, kc.shape[0], Hk), scales_of(2, kc.shape[0], Hk)
    v = rand(3, n, Hk, D, dtype=BF16) * torch.exp2(torch.arange(n, device="cuda") % 7 - 3.0)[:, None, None].to(BF16)
    for t in range(n):
        A.kv_append_scaled(v[t:t + 1], v[t:t + 1], kc, vc, ks, vs, table, i32([t + 1]), cu_of([1]), i32([0]), freqs(D))
    for first in range(0, n, page):
        p, m = int(table[0, first // page]), min(page, n - first)
        x, s = v[first:first + m].cpu().double(), vs.cpu().double()[p]
        got = values(vc)[p, :, :m].transpose(0, 1) * s[None, :, None]
        # half a step when it was written and again at each growth, each step of a scale at most twice the one before
        tol = 2 * torch.maximum(2.0 ** -4 * x.abs(), 2.0 ** -10 * s[None, :, None]) * 1.0625
        assert ((got - x).abs() <= tol).all()
        assert (x.abs().amax((0, 2)) <= 448 * s * (1 + 2.0 ** -22)).all()


def test_other_stream_graph_and_strides(A):
    """Captured, replayed on new inputs and on a side stream: as called; slices and page-major caches are taken as they are."""
    q_len, kv_len, Hq, Hk, D, page = [33, 1, 17], [70, 20, 17], 4, 2, 128, 16
    T = sum(q_len)
    table0 = make_pages(1, kv_len, page, Hk, D, BF16, "e4m3")
    f, pos = freqs(D), positions_of(2, T, 1)
    n_pages = table0[0].shape[0]

    def fresh():
        kc, vc, _ = make_pages(1, kv_len, page, Hk, D, BF16, "e4m3", token_major=True)
        return kc, vc, scales_of(3, n_pages, Hk), scales_of(4, n_pages, Hk)

    x = rand(5, T, Hq + 2 * Hk, D, dtype=BF16)
    args = lambda: (x[:, Hq:Hq + Hk], x[:, Hq + Hk:])  # noqa: E731
    rest = (table0[2], i32(kv_len), cu_of(q_len), pos, f)
    state = fresh()
    stream = torch.cuda.Stream()
    q_out = torch.empty(T, Hq, D, dtype=BF16, device="cuda")
    stream.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        A.kv_append_scaled(*args(), *state, *rest, q=x[:, :Hq], q_out=q_out)
    torch.cuda.current_stream().wait_stream(stream)
    for seed in (6, 7):
        x.copy_(rand(seed, *x.shape, dtype=BF16))
        start = fresh()
        for a, b in zip(state, start):
            (a.view(torch.uint8) if a.dtype == torch.float8_e4m3fn else a).copy_(b.view(torch.uint8) if b.dtype == torch.float8_e4m3fn else b)
        graph.replay()
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        want = A.kv_append_scaled(*args(), *start, *rest, q=x[:, :Hq], stream=side)
        side.synchronize()
        assert torch.equal(want, q_out)
        for a, b in zip(state, start):
            assert torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


def test_refusals_on_the_gpu(A):
    from depth_weighted_scatter_gb300.bevpool import BevpoolError

    z = lambda *s, dtype=torch.float16: torch.zeros(*s, dtype=dtype, device="cuda")  # noqa: E731
    f32, u8, i = torch.float32, torch.uint8, torch.int32
    good = dict(k=z(3, 2, 64), v=z(3, 2, 64), k_cache=z(4, 2, 16, 64, dtype=u8), v_cache=z(4, 2, 16, 64, dtype=u8), k_scales=z(4, 2, dtype=f32),
                v_scales=z(4, 2, dtype=f32), block_table=z(3, 2, dtype=i), kv_len=z(3, dtype=i), cu_q=z(4, dtype=i), positions=z(3, dtype=i),
                inv_freq=z(32, dtype=f32))
    assert A.kv_append_scaled(**good) is None
    for bad in [dict(k_scales=z(4, 3, dtype=f32)), dict(v_scales=z(3, 2, dtype=f32)), dict(k_scales=z(4, 2)), dict(v_scales=z(2, 4, dtype=f32).t()),
                dict(k_scales=z(4, 2, dtype=f32).cpu()), dict(v_scales=1.0), dict(k_cache=z(4, 2, 16, 64), v_cache=z(4, 2, 16, 64)),
                dict(k=z(3, 4, 64)), dict(q_out=z(3, 4, 64)), dict(positions=z(3, 5, dtype=i)), dict(k_scales=z(4, 2, 1, dtype=f32)),
                dict(k=z(3, 2, 80), v=z(3, 2, 80), k_cache=z(4, 2, 16, 80, dtype=u8), v_cache=z(4, 2, 16, 80, dtype=u8))]:
        with pytest.raises(BevpoolError):
            A.kv_append_scaled(**{**good, **bad})
    with pytest.raises(BevpoolError, match="gradients"):
        A.kv_append_scaled(**{**good, "k_scales": z(4, 2, dtype=f32).requires_grad_()})
    torch.cuda.synchronize()
