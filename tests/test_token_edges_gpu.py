"""The token operators where a call is easy to get wrong: host bounds far above
the lengths on the device, heads that do not fill a step, weights far below the
largest.  Definitions and bounds: tests/token_ref.py."""
import pytest

import token_ref as ref
from test_token_ops_gpu import attend_inputs, norm_rope_inputs, rand, within

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

F16, BF16 = torch.float16, torch.bfloat16


@pytest.fixture(scope="module")
def A():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    from depth_weighted_scatter_gb300 import attention

    return attention


# ------------------------------------------------------------------ bounds far above the lengths

@pytest.mark.parametrize("case, most", [
    # every request's keys lie in one chunk although the bound makes many: few rows, chunked tiles, shared tiles
    (([1, 1, 1], [60, 5, 33], 8, 2, 128, True, 0, BF16, "same", 16, False), 60000),
    (([2], [64], 4, 1, 64, True, 0, F16, "e4m3", 64, False), 131072),
    (([70, 33], [100, 90], 6, 2, 128, True, 0, BF16, "same", 16, True), 30000),
    (([1100, 1], [128, 0], 8, 8, 64, False, 0, F16, "same", 32, False), 8000),
], ids=["few", "few_e4m3", "chunked", "shared"])
def test_attention_is_done_when_the_next_kernel_reads_it(A, case, most):
    """What comes next in the stream sees the results, call after call."""
    x = attend_inputs(case, seed=2000)
    x["max_kv_len"] = most
    pages = -(-most // case[9])                             # the table has room for the bound; past the lengths there is no page
    x["block_table"] = torch.nn.functional.pad(x["block_table"], (0, pages - x["block_table"].shape[1]), value=-1).contiguous()
    assert A.bevpool_paged_attention_workspace_size(len(case[0]), sum(case[0]), *case[2:5], max(case[0]), most, 0) > 0
    args = (x.pop("q"), x.pop("k_cache"), x.pop("v_cache"), x.pop("block_table"), x.pop("kv_len"), x.pop("cu_q"))
    want, _, tol, _, _ = ref.attention(*args, scale=case[4] ** -0.5, **x)
    out, seen = torch.empty_like(args[0]), []
    for _ in range(200):
        out.fill_(float("nan"))
        A.paged_attention(*args, out=out, **x)
        seen.append(out.clone())
    within(seen[0], want, tol, "out")
    assert all(torch.equal(s, seen[0]) for s in seen)


# ------------------------------------------------------------------ the caller's workspace

def test_workspace_of_the_caller(A):
    """One of the size that is named serves; views that do not own their bytes, and other devices, are refused."""
    from depth_weighted_scatter_gb300.bevpool import BevpoolError

    x = attend_inputs(([1], [3000], 8, 2, 128, True, 0, BF16, "same", 16, False), seed=2100)
    args = (x.pop("q"), x.pop("k_cache"), x.pop("v_cache"), x.pop("block_table"), x.pop("kv_len"), x.pop("cu_q"))
    size = A.bevpool_paged_attention_workspace_size(1, 1, 8, 2, 128, 1, 3000, 0)
    own = torch.empty(size, dtype=torch.uint8, device="cuda")
    assert torch.equal(A.paged_attention(*args, workspace=own, **x), A.paged_attention(*args, **x))
    q, pos = args[0].expand(5, 8, 128), torch.arange(5, dtype=torch.int32, device="cuda")
    f, w = torch.ones(64, device="cuda"), torch.ones(128, device="cuda")
    need = A.bevpool_qk_norm_rope_backward_workspace_size(5, 8, 8, 128)
    own = torch.empty(need, dtype=torch.uint8, device="cuda")
    got = A.qk_norm_rope_backward(q, q, q, q, pos, f, q_weight=w, workspace=own)
    want = A.qk_norm_rope_backward(q, q, q, q, pos, f, q_weight=w)
    assert all(torch.equal(a, b) for a, b in zip(got[:3], want))
    wide = torch.empty(2, size, dtype=torch.uint8, device="cuda")
    for bad in (torch.empty(size, dtype=torch.uint8), wide[:1, :1].expand(1, size), wide[:, :size // 2], own[:1].expand(need)):
        with pytest.raises(BevpoolError, match="workspace"):
            A.paged_attention(*args, workspace=bad, **x)
        with pytest.raises(BevpoolError, match="workspace"):
            A.qk_norm_rope_backward(q, q, q, q, pos, f, q_weight=w, workspace=bad)


# ------------------------------------------------------------------ heads that do not fill a step

@pytest.mark.parametrize("eps", [0.0, 1e-30])
@pytest.mark.parametrize("case", [
    # T, Hq, Hk, D, R, axes, interleaved, dtype: a step holds 32 / (lanes of a row) heads
    (5, 3, 1, 128, 128, 1, False, BF16),
    (700, 7, 1, 128, 96, 2, True, F16),
    (5, 7, 2, 64, 64, 3, True, F16),
    (3000, 5, 1, 64, 32, 1, False, BF16),
    (9, 9, 3, 32, 32, 1, False, F16),
    (9, 4, 2, 80, 80, 1, True, BF16),                       # heads fill the steps, lanes the rows do not
    (4, 3, 1, 256, 256, 1, False, F16),
], ids=str)
def test_norm_rope_backward_without_eps(A, case, eps):
    """Places of a step without a head add nothing to the weights' gradients: no real row is zero, so eps = 0 is as
    good as any."""
    T, Hq, Hk, D, R, axes, il, dtype = case
    x = norm_rope_inputs(case, seed=70)
    x["eps"] = eps
    dy = dict(q=rand(71, T, Hq, D, dtype=dtype), k=rand(72, T, Hk, D, dtype=dtype))
    args = {k: v for k, v in x.items() if k not in ("q", "k", "positions", "inv_freq")}
    got = A.qk_norm_rope_backward(dy["q"], dy["k"], x["q"], x["k"], x["positions"], x["inv_freq"], **args)
    out = A.qk_norm_rope(x["q"], x["k"], x["positions"], x["inv_freq"], **args)
    cos, sin = ref.cos_sin(x["positions"], x["inv_freq"], x["sections"])
    for i, name in enumerate("qk"):
        want, mag = ref.norm_rope(x[name], x[name + "_weight"], cos, sin, il, eps)
        within(out[i], want, ref.U[dtype] * want.abs() + 2.0 ** -18 * mag + ref.tiny(dtype), name)
        dx, mag, dw, dw_mag = ref.norm_rope_back(dy[name], x[name], x[name + "_weight"], cos, sin, il, eps)
        within(got[i], dx, ref.U[dtype] * dx.abs() + 2.0 ** -16 * mag + ref.tiny(dtype), "d" + name)
        within(got[2 + i], dw, 2.0 ** -16 * dw_mag, "d" + name + "_weight")
