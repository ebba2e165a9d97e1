"""The fleet of the temporal attention example: planned pages, a cache with page
scales, against a float64 attention over the codes that the cache holds."""
import pytest

import scaled_ref as sref
from test_temporal_example_gpu import ex  # noqa: F401
from test_token_ops_gpu import within

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def test_fleet(ex):  # noqa: F811
    Y = X = 16
    fleet = ex.PlannedAttention(64, Y, X, vehicles=3, frames=2)
    seen = [0, 0, 0]
    for t in range(5):
        drive = [True, t % 2 == 0, t > 2]
        bevs = torch.cat([ex.pooled_frame(10 * i + t, Y=Y, X=X) for i, on in enumerate(drive) if on])
        calls = []
        attend = ex.attention.paged_attention_scaled
        ex.attention.paged_attention_scaled = lambda *a, **k: calls.append((a, k)) or attend(*a, **k)
        try:
            y = fleet.step(bevs, drive)
        finally:
            ex.attention.paged_attention_scaled = attend
        seen = [min(n + on, 2) for n, on in zip(seen, drive)]
        assert fleet.state[0].tolist() == [n * Y * X for n in seen]
        assert fleet.state[4].item() == fleet.k_cache.shape[0] - sum(seen) * fleet.pages
        (a, k), = calls
        assert y.shape == (sum(drive) * Y * X, fleet.H, fleet.D)
        want, _, tol, _, done = sref.attention(*a, scale=fleet.D ** -0.5, **k)
        assert done.all()
        within(y, want, tol, f"frame {t}")
        # the newest frame's values are in the cache, within half a step of their page's scale
        v = (bevs @ fleet.project).view(-1, fleet.H + 2 * fleet.Hk, fleet.D)[:, fleet.H + fleet.Hk:].cpu().double()
        at = 0
        for i, on in enumerate(drive):
            if on:
                pages = fleet.state[2][i, (seen[i] - 1) * fleet.pages:seen[i] * fleet.pages].long().cpu()
                s = fleet.v_scales.cpu().double()[pages][:, :, None, None]
                got = (fleet.v_cache.float().cpu().double()[pages] * s).transpose(1, 2).reshape(-1, fleet.Hk, fleet.D)
                x = v[at:at + Y * X]
                step = (s.expand(-1, -1, ex.PAGE, 1)).transpose(1, 2).reshape(-1, fleet.Hk, 1)
                assert ((got - x).abs() <= torch.maximum(2.0 ** -4 * x.abs(), 2.0 ** -10 * step) * (1 + 2.0 ** -20)).all()
                at += Y * X
