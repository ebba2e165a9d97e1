"""Queries near the ends of bf16's range over caches of one type or one scale (those with page scales:
test_scaled_edges_gpu)."""
import pytest

from test_token_ops_gpu import A, BF16, attend_inputs, check_attend  # noqa: F401

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.mark.parametrize("q_len, Hq, D", [(1, 1, 64), (1, 4, 128), (3, 4, 64), (40, 4, 128)])
@pytest.mark.parametrize("cache", ["same", "e4m3"])
@pytest.mark.parametrize("power", [115, 101, -101, -105])
def test_largest_and_smallest_queries(A, q_len, Hq, D, cache, power):  # noqa: F811
    """The attention of queries of the order of 1, when the scale takes their magnitude back; a row of zeros among them is the
    mean of the values."""
    x = attend_inputs(([q_len] * 3, [90, 200, 17], Hq, 1, D, True, 0, BF16, cache, 16, False), seed=810)
    x["q"] = x["q"] * 2.0 ** power
    x["q"][0] = 0.0
    x["scale"] = D ** -0.5 * 2.0 ** -power
    check_attend(A, x)
