"""The fleet of the temporal attention example where its frames do not fit."""
import pytest

from test_temporal_example_gpu import ex  # noqa: F401

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def frames(ex, n, seed):  # noqa: F811
    return torch.cat([ex.pooled_frame(seed + i, Y=16, X=16) for i in range(n)])


def test_a_plan_that_does_not_fit_is_an_error(ex):  # noqa: F811
    """Without pages for a frame nothing is attended, so there are no rows to return; the state stays, and the next step that
    fits goes on from it."""
    fleet = ex.PlannedAttention(64, 16, 16, vehicles=2, frames=2)
    fleet.step(frames(ex, 2, 0), [True, True])
    free = fleet.state[4].clone()
    fleet.state[4].fill_(fleet.pages - 1)
    before = [s.clone() for s in fleet.state]
    with pytest.raises(RuntimeError, match="pages"):
        fleet.step(frames(ex, 1, 10), [False, True])
    assert all(torch.equal(a, b) for a, b in zip(before[:3], fleet.state[:3])) and torch.equal(before[4], fleet.state[4])
    fleet.state[4].copy_(free)
    y = fleet.step(frames(ex, 1, 10), [False, True])
    assert y.shape == (256, fleet.H, fleet.D) and y.isfinite().all()
    assert fleet.state[0].tolist() == [256, 512]


@pytest.mark.parametrize("n", [1, 3])
def test_cells_of_others_are_an_error(ex, n):  # noqa: F811
    """More or fewer cells than the vehicles that drive have: rows that no request takes would be returned as they are."""
    fleet = ex.PlannedAttention(64, 16, 16, vehicles=2, frames=2)
    with pytest.raises(ValueError, match="cells"):
        fleet.step(frames(ex, n, 0), [True, True])
    assert fleet.state[0].tolist() == [0, 0]
