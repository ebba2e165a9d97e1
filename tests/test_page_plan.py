"""What the page plan refuses before any CUDA work, and its definition on a case
that is worked out by hand (no GPU needed)."""
import pytest

import page_plan_ref as ref

torch = pytest.importorskip("torch")

FAKE = 1 << 20   # never dereferenced: every call below fails validation first


@pytest.fixture(scope="module")
def A():
    from depth_weighted_scatter_gb300 import _build

    _build.build()
    from depth_weighted_scatter_gb300 import attention

    return attention


def test_c_refusals(A):
    args = dict(q_len=FAKE, kv_len=FAKE, first=FAKE, drop=FAKE, table=FAKE, free=FAKE, n_free=FAKE, n_seqs=3, table_pages=4, n_pool=9,
                n_tokens=5, page=16, cu_q=FAKE, positions=FAKE, slots=FAKE, kv_out=FAKE, first_out=FAKE, table_out=FAKE, free_out=FAKE,
                n_free_out=FAKE, missing=FAKE, stream=0)
    for name in ("q_len", "kv_len", "first", "table", "free", "n_free", "cu_q", "positions", "slots", "kv_out", "first_out", "table_out",
                 "free_out", "n_free_out", "missing"):
        for p in (0, FAKE + 2):
            assert A.bevpool_plan_pages(*{**args, name: p}.values()) == 1, name
    for change in (dict(n_seqs=-1), dict(table_pages=0), dict(n_pool=0), dict(n_tokens=-1), dict(page=0), dict(page=-16), dict(drop=FAKE + 1),
                   dict(slots=FAKE + 4), dict(table_pages=2 ** 31 - 1), dict(table_pages=2 ** 27, page=16)):
        assert A.bevpool_plan_pages(*{**args, **change}.values()) == 1, change
    for change in (dict(page=8), dict(page=48), dict(page=512), dict(n_seqs=16385)):
        assert A.bevpool_plan_pages(*{**args, **change}.values()) == 3, change


def test_helper_refuses_host_tensors(A):
    from depth_weighted_scatter_gb300.bevpool import BevpoolError

    z = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(BevpoolError, match="device"):
        A.plan_pages(z, z, z, torch.zeros(3, 4, dtype=torch.int32), z, z[:1], page_size=16, n_tokens=3)


def test_definition_by_hand():
    """Two requests on pages of 16: the first lets go of a page and grows, the second ends and starts anew."""
    got = ref.plan([3, 17], [30, 5], [100, 7], [[4, 9, -1], [2, -1, -1]], [6, 0, 1, -1, -1], 3, page_size=16, n_tokens=21, drop=[1, -1])
    # the stack becomes 6 0 1 4 2; the first keeps tokens 16..29 on page 9, 14 of them, and takes page 2 for its 17th place
    assert got["block_table"] == [[9, 2, -1], [4, 1, -1]]
    assert got["kv_len"] == [17, 17] and got["first"] == [116, 0] and got["cu_q"] == [0, 3, 20]
    assert got["positions"][:4] == [130, 131, 132, 0] and got["slots"][:4] == [9 * 16 + 14, 9 * 16 + 15, 2 * 16, 4 * 16]
    assert got["slots"][19:] == [16, -1] and got["free_pages"] == [6, 0, -1, -1, -1] and got["n_free"] == [2]
    assert ref.plan([50], [0], [0], [[-1] * 9], [1, 2, 3], 3, page_size=16, n_tokens=50)["missing"] == [1]
