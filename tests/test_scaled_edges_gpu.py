"""Attention and append with page scales at their edges: queries of zeros, scales
far apart in tiles of bf16 heads, caches past 32 bits."""
import pytest

import scaled_ref as sref
import token_ref as ref
from test_scaled_attention_gpu import A, BF16, F16, NAMES, attend, check, check_rows, inputs  # noqa: F401
from test_token_ops_gpu import cu_of, freqs, i32, rand, within

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
