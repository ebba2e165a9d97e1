"""The temporal attention example: each frame's output against the definition in
FP64 over the frames kept, and a falling training loss."""
import importlib.util
import os

import pytest

import token_ref as ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def ex():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    spec = importlib.util.spec_from_file_location("temporal_bev", os.path.join(ROOT, "examples", "temporal_bev.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_frames_attend_over_the_frames_kept(ex):
    """The keys are rounded to 16 bits twice on the way (rotation, cache); their scores move by at most the sum of
    2 * 2^-11 of |q k|, which the bound adds to the operators' own."""
    Y = X = 16
    model = ex.TemporalAttention(64, Y, X, frames=3)
    seen = []
    for t in range(5):
        bev = ex.pooled_frame(t, Y=Y, X=X)
        q, k, v = model.qkv(bev)
        cos, sin = ref.cos_sin(model.positions(), model.inv_freq, model.sections)
        y = model.step(bev)
        q = ref.norm_rope(q, model.q_weight, cos, sin, False, 1e-6)[0]
        k = ref.norm_rope(k, model.k_weight, cos, sin, False, 1e-6)[0]
        seen = (seen + [(k, v.cpu().double())])[-3:]
        K, V = torch.cat([s[0] for s in seen]), torch.cat([s[1] for s in seen])
        for h in range(0, model.H, 3):
            kh, vh = K[:, h // 2], V[:, h // 2]
            s = q[:, h] @ kh.T * model.D ** -0.5
            d = (4 * 2.0 ** -11 + (model.D + 8) * 2.0 ** -23) * model.D ** -0.5 * (q[:, h].abs() @ kh.abs().T).max(-1).values
            p = torch.softmax(s, -1)
            tol = (2.0 ** -11 + 2 * d[:, None] + 2.0 ** -18) * (p @ vh.abs()) + 2.0 ** -11 * (p @ vh).abs() + 2.0 ** -20
            assert ((y[:, h].cpu().double() - p @ vh).abs() <= tol).all(), (t, h)


def test_e4m3_frames_and_training(ex):
    model = ex.TemporalAttention(64, 16, 16, frames=2, cache_dtype=torch.float8_e4m3fn)
    for t in range(3):
        y = model.step(ex.pooled_frame(t, Y=16, X=16))
    assert y.isfinite().all() and y.any()
    bev = ex.pooled_frame(9, Y=16, X=16)
    q, k, _ = model.qkv(bev)
    target = ex.attention.qk_norm_rope(q, k, model.positions(), model.inv_freq, sections=model.sections,
                                       q_weight=2 * model.q_weight, k_weight=0.5 * model.k_weight)
    losses = [model.train_step(bev, *target, lr=0.5) for _ in range(6)]
    assert all(b < a for a, b in zip(losses, losses[1:])), losses
