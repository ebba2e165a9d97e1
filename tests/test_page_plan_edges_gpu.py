"""The page plan on tables that name a page more than once: as its documentation says."""
import pytest

import page_plan_ref as ref
from test_token_ops_gpu import i32

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def test_a_shared_page_goes_back_once_for_each_request():
    """Page numbers are not looked at: two requests that name page 3 give it back twice, which is why planned pages are not
    shared."""
    from depth_weighted_scatter_gb300 import attention as A

    q_len, kv_len, first, table, free, drop = [20, 0, 1], [32, 40, 0], [0, 0, 0], [[3, 1, -1], [3, 2, 4], [-1] * 3], [0, 5, -1, -1, -1, -1, -1], [1, -1, 0]
    want = ref.plan(q_len, kv_len, first, table, free, 2, page_size=16, n_tokens=21, drop=drop)
    got = A.plan_pages(i32(q_len), i32(kv_len), i32(first), i32(table), i32(free), i32([2]), page_size=16, n_tokens=21, drop=i32(drop))
    assert {k: v.tolist() for k, v in got._asdict().items()} == want
    assert want["missing"] == [0]
    handed = [p for row in want["block_table"] for p in row if p >= 0] + want["free_pages"][:want["n_free"][0]]
    assert handed.count(3) == 2
