"""The page plan against its definition (tests/page_plan_ref.py): whole numbers, equal."""
import random

import pytest

import page_plan_ref as ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def A():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    from depth_weighted_scatter_gb300 import attention

    return attention


def i32(x, *shape):
    return torch.tensor(x, dtype=torch.int32, device="cuda").reshape(*shape) if shape else torch.tensor(x, dtype=torch.int32, device="cuda")


def state(seed, B, W, cap, page, most):
    """A pool of cap pages, requests of up to `most` tokens on some of them."""
    rng = random.Random(seed)
    pages = list(range(cap))
    rng.shuffle(pages)
    kv, table = [], []
    for b in range(B):
        n = rng.choice([0, 1, page - 1, page, page + 1, rng.randint(0, most)])
        n = min(n, most, len(pages) * page, W * page)
        row = [pages.pop() for _ in range(ref.pages_for(n, page))]
        kv.append(n)
        table.append(row + [-1] * (W - len(row)))
    return dict(kv_len=kv, first=[rng.randint(0, 1000) for _ in range(B)], table=table,
                free=pages + [-1] * (cap - len(pages)), n_free=len(pages))


def run(A, x, q, **more):
    W = len(x["table"][0]) if x["table"] else 3
    drop = more.pop("drop", None)
    return A.plan_pages(i32(q), i32(x["kv_len"]), i32(x["first"]), i32(x["table"], len(x["table"]), W), i32(x["free"]), i32([x["n_free"]]),
                        drop=None if drop is None else i32(drop), **more)


def check(A, x, q, *, page_size, n_tokens, drop=None, **more):
    got = run(A, x, q, page_size=page_size, n_tokens=n_tokens, drop=drop, **more)
    want = ref.plan(q, x["kv_len"], x["first"], x["table"], x["free"], x["n_free"], page_size=page_size, n_tokens=n_tokens, drop=drop)
    for name, t in got._asdict().items():
        assert t.tolist() == want[name], name
    return got


# B, table pages, pool, page size, most tokens, most new tokens
SIZES = [(1, 1, 1, 16, 16, 1), (1, 7, 9, 16, 100, 5), (3, 40, 64, 32, 1000, 70), (64, 515, 5000, 16, 2000, 1),
         (31, 9, 500, 256, 2000, 300), (513, 12, 9000, 16, 150, 7), (1500, 5, 9000, 64, 200, 100), (4, 600, 1400, 64, 16384, 16384)]


@pytest.mark.parametrize("drops", ["none", "some", "ends"])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_plan(A, size, drops):
    B, W, cap, page, most, new = size
    x = state(B, B, W, cap, page, most)
    rng = random.Random(7)
    q = [rng.choice([0, 1, new, rng.randint(0, new)]) for _ in range(B)]
    drop = {"none": None, "some": [rng.choice([0, 1, 3, 10 ** 9]) for _ in range(B)],
            "ends": [rng.choice([0, 0, -1, 2]) for _ in range(B)]}[drops]
    for slack in (0, 13):
        check(A, x, q, page_size=page, n_tokens=sum(q) + slack, drop=drop)


def test_plan_after_plan(A):
    """A run of steps: every page is in one place at all times, and positions go on."""
    page, B, W, cap = 16, 5, 12, 48
    x = state(1, B, W, cap, page, 60)
    rng = random.Random(3)
    dev = [i32(x["kv_len"]), i32(x["first"]), i32(x["table"]), i32(x["free"]), i32([x["n_free"]])]
    seen = set()
    for step in range(60):
        q = [rng.choice([0, 1, 1, 5, 30]) for _ in range(B)]
        drop = [rng.choice([0, 0, 1, -1]) if rng.random() < 0.15 else 0 for _ in range(B)]
        got = A.plan_pages(i32(q), *dev, page_size=page, n_tokens=200, drop=i32(drop))
        want = ref.plan(q, x["kv_len"], x["first"], x["table"], x["free"], x["n_free"], page_size=page, n_tokens=200, drop=drop)
        for name, t in got._asdict().items():
            assert t.tolist() == want[name], (step, name)
        seen.add(min(got.missing.item(), 1))
        x = dict(kv_len=want["kv_len"], first=want["first"], table=want["block_table"], free=want["free_pages"], n_free=want["n_free"][0])
        dev = [got.kv_len, got.first, got.block_table, got.free_pages, got.n_free]
        used = [p for row in x["table"] for p in row if p >= 0] + x["free"][:x["n_free"]]
        assert sorted(used) == list(range(cap)), step
    assert seen == {-1, 0, 1}                                # every outcome was met


@pytest.mark.parametrize("what", ["pages", "row", "old_row", "rows", "pool", "huge"])
def test_what_does_not_fit_changes_nothing(A, what):
    x = state(5, 4, 6, 30, 16, 80)
    q, more = [3, 40, 0, 9], dict(page_size=16, n_tokens=60)
    drop = None
    if what == "pages":
        x["n_free"] = 1
    elif what == "row":
        q[2] = 97 - x["kv_len"][2] + 16 * 6
        more["n_tokens"] = 400
    elif what == "old_row":
        x["kv_len"][1] = 16 * 6 + 1
    elif what == "rows":
        more["n_tokens"] = 51
    elif what == "pool":
        x["n_free"], drop = 30, [-1, -1, -1, -1]
        x["kv_len"] = [16] * 4
    else:
        q[0], x["kv_len"][3] = 2 ** 31 - 1, 2 ** 31 - 1
    got = check(A, x, q, drop=drop, **more)
    assert got.missing.item() != 0 and got.kv_len.tolist() == x["kv_len"]


def test_lengths_and_counts_below_zero(A):
    x = state(6, 3, 8, 40, 16, 60)
    x["kv_len"][1] = -5
    x["table"][1] = [-1] * 8
    check(A, x, [-3, 4, 20], page_size=16, n_tokens=30)
    x["n_free"] = -2
    check(A, x, [0, 0, 100], page_size=16, n_tokens=130)


def test_positions_wrap_no_bits(A):
    """Positions near the ends of 32 bits; tokens before position 0."""
    x = state(8, 2, 8, 40, 16, 60)
    x["first"] = [2 ** 31 - 1 - 90, -70]
    check(A, x, [5, 6], page_size=16, n_tokens=11, drop=[1, 2])


def test_no_requests_and_the_most(A):
    got = A.plan_pages(i32([]), i32([]), i32([]), torch.zeros(0, 3, dtype=torch.int32, device="cuda"), i32([4, 2]), i32([2]),
                       page_size=16, n_tokens=3)
    assert got.cu_q.tolist() == [0] and got.slots.tolist() == [-1] * 3 and got.free_pages.tolist() == [4, 2]
    assert got.missing.item() == 0 and got.n_free.item() == 2
    from depth_weighted_scatter_gb300.bevpool import BevpoolError

    B = 16384
    x = dict(kv_len=[b % 33 for b in range(B)], first=[b for b in range(B)], n_free=B)
    it = iter(range(4 * B))
    x["table"] = [[next(it) if i * 16 < n else -1 for i in range(3)] for n in x["kv_len"]]
    rest = list(it)
    x["free"], x["n_free"] = rest, len(rest)
    check(A, x, [b % 3 for b in range(B)], page_size=16, n_tokens=B, drop=[-1 if b % 7 == 0 else b % 2 for b in range(B)])
    z = torch.zeros(B + 1, dtype=torch.int32, device="cuda")
    with pytest.raises(BevpoolError) as e:
        A.plan_pages(z, z, z, z[:, None].contiguous(), i32([0]), i32([1]), page_size=16, n_tokens=0)
    assert e.value.status == 3


def test_plan_in_a_graph_and_on_another_stream(A):
    """Captured once with its outputs copied back, a step can be replayed; given outputs are the ones written."""
    page, B, W, cap = 32, 7, 9, 80
    x = state(11, B, W, cap, page, 100)
    q = [1, 0, 5, 1, 1, 2, 1]
    dev = [i32(x["kv_len"]), i32(x["first"]), i32(x["table"]), i32(x["free"]), i32([x["n_free"]])]
    dq = i32(q)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    mine = A.plan_pages(dq, *dev, page_size=page, n_tokens=11)
    with torch.cuda.stream(stream):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            plan = A.plan_pages(dq, *dev, page_size=page, n_tokens=11, out=mine)
            for old, new in zip(dev, [plan.kv_len, plan.first, plan.block_table, plan.free_pages, plan.n_free]):
                old.copy_(new)
    torch.cuda.current_stream().wait_stream(stream)
    assert all(a is b for a, b in zip(plan, mine))
    for _ in range(4):
        want = ref.plan(q, x["kv_len"], x["first"], x["table"], x["free"], x["n_free"], page_size=page, n_tokens=11)
        graph.replay()
        for name, t in plan._asdict().items():
            assert t.tolist() == want[name], name
        x = dict(kv_len=want["kv_len"], first=want["first"], table=want["block_table"], free=want["free_pages"], n_free=want["n_free"][0])
    other = torch.cuda.Stream()
    torch.cuda.synchronize()
    for s in (other, other.cuda_stream):
        got = A.plan_pages(dq, *dev, page_size=page, n_tokens=11, stream=s)
        other.synchronize()
        want = ref.plan(q, x["kv_len"], x["first"], x["table"], x["free"], x["n_free"], page_size=page, n_tokens=11)
        assert got.slots.tolist() == want["slots"] and got.block_table.tolist() == want["block_table"]


def test_refusals_on_the_gpu(A):
    from depth_weighted_scatter_gb300.bevpool import BevpoolError

    x = state(2, 3, 4, 20, 16, 50)
    args = dict(q_len=i32([1, 1, 1]), kv_len=i32(x["kv_len"]), first=i32(x["first"]), block_table=i32(x["table"]), free_pages=i32(x["free"]),
                n_free=i32([x["n_free"]]), page_size=16, n_tokens=4)
    plan = A.plan_pages(**args)
    for bad in [dict(q_len=i32([1, 1])), dict(kv_len=args["kv_len"].long()), dict(first=args["first"].cpu()), dict(block_table=i32(x["table"]).t()),
                dict(block_table=i32(x["table"][0])), dict(n_free=i32([1, 2])), dict(page_size=24), dict(page_size=512), dict(page_size=0),
                dict(n_tokens=-1), dict(n_tokens=1 << 40), dict(drop=i32([1])), dict(drop=i32([1, 1, 1]).float()), dict(q_len=None),
                dict(free_pages=i32([])), dict(out=plan[:8]), dict(out=plan._replace(slots=plan.positions)),
                dict(out=plan._replace(kv_len=args["kv_len"])), dict(out=plan._replace(kv_len=plan.first)), dict(out=plan._replace(missing=None)),
                dict(out=plan._replace(free_pages=plan.free_pages[:19])), dict(out=plan._replace(block_table=plan.block_table.view(4, 3)))]:
        with pytest.raises(BevpoolError):
            A.plan_pages(**{**args, **bad})
    torch.cuda.synchronize()
