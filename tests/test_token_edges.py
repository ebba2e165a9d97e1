"""What the tensor helpers of the token operators refuse before any CUDA work
(no GPU needed)."""
import pytest

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def A():
    from depth_weighted_scatter_gb300 import _build

    _build.build()
    from depth_weighted_scatter_gb300 import attention

    return attention


def calls(A):
    """Each helper that takes a workspace, as a function of its further arguments."""
    q, c = torch.zeros(3, 4, 64, dtype=torch.float16), torch.zeros(4, 4, 16, 64, dtype=torch.float16)
    pos, f, w = torch.zeros(3, dtype=torch.int32), torch.zeros(32), torch.ones(64)
    t, n, cu = torch.zeros(3, 2, dtype=torch.int32), torch.zeros(3, dtype=torch.int32), torch.zeros(4, dtype=torch.int32)
    return [lambda **kw: A.qk_norm_rope_backward(q, q, q, q, pos, f, q_weight=w, **kw),
            lambda **kw: A.paged_attention(q, c, c, t, n, cu, max_q_len=1, max_kv_len=4, **kw)]


@pytest.mark.parametrize("i", [0, 1])
def test_workspace_is_checked(A, i):
    """A workspace has to own the bytes that it counts, on the device: else the kernels write elsewhere."""
    from depth_weighted_scatter_gb300.bevpool import BevpoolError

    call = calls(A)[i]
    for ws, why in ((torch.zeros(1 << 20, dtype=torch.uint8), "device"),
                    (torch.zeros(1, dtype=torch.uint8).expand(1 << 40), "contiguous"),
                    (torch.zeros(64, 64)[:, :32], "contiguous")):
        with pytest.raises(BevpoolError, match="workspace: .*" + why):
            call(workspace=ws)


def test_gradients_are_not_dropped(A):
    """A tensor that requires gradients, or carries a tangent, is refused: the results would not be connected to it."""
    from depth_weighted_scatter_gb300.bevpool import BevpoolError

    q, c = torch.zeros(3, 4, 64, dtype=torch.float16), torch.zeros(4, 4, 16, 64, dtype=torch.float16)
    pos, f, w = torch.zeros(3, dtype=torch.int32), torch.zeros(32), torch.ones(64)
    t, n, cu = torch.zeros(3, 2, dtype=torch.int32), torch.zeros(3, dtype=torch.int32), torch.zeros(4, dtype=torch.int32)
    g = q.clone().requires_grad_()
    gw = w.clone().requires_grad_()
    calls = [lambda: A.qk_norm_rope(g, q, pos, f), lambda: A.qk_norm_rope(q, g, pos, f), lambda: A.qk_norm_rope(g * 2, q, pos, f),
             lambda: A.qk_norm_rope(q, q, pos, f, k_weight=gw), lambda: A.qk_norm_rope(q, q, pos, f, q_out=g),
             lambda: A.qk_norm_rope_backward(g, q, q, q, pos, f), lambda: A.qk_norm_rope_backward(q, q, q, q, pos, f, q_weight=gw),
             lambda: A.kv_append(q, g, c, c, t, n, cu, pos, f), lambda: A.kv_append(q, q, c, c, t, n, cu, pos, f, q=g),
             lambda: A.paged_attention(g, c, c, t, n, cu, max_q_len=1, max_kv_len=4)]
    for call in calls:
        with pytest.raises(BevpoolError, match="gradients are not recorded"):
            call()
        with torch.no_grad(), pytest.raises(BevpoolError) as e:         # refused for being on the host alone
            call()
        assert "gradients" not in str(e.value)
    import torch.autograd.forward_ad as fwd
    with fwd.dual_level(), torch.no_grad():
        dual = fwd.make_dual(w, torch.ones_like(w))
        with pytest.raises(BevpoolError, match="gradients are not recorded"):
            A.qk_norm_rope(q, q, pos, f, q_weight=dual)
