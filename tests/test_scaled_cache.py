"""The C entry points and tensor helpers of a cache with page scales reject bad
arguments on the host (no GPU needed)."""
import pytest

from test_token_abi import FAKE, HEADS_INVALID, HEADS_UNSUPPORTED, PAGES_INVALID, PAGES_UNSUPPORTED, ROTARY_INVALID, _sections, check, rows

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def A():
    from depth_weighted_scatter_gb300 import _build

    _build.build()
    from depth_weighted_scatter_gb300 import attention

    return attention


PAGES = dict(ps=4096, ss=128, hs=2048, ks=FAKE, vs=FAKE, n_pages=10, page=16, table=FAKE, table_pages=4, kv_len=FAKE, cu_q=FAKE, n_seqs=3)
SCALES_INVALID = [dict(ks=0), dict(vs=0), dict(ks=FAKE + 2), dict(vs=FAKE + 1)]


def append_args():
    return dict(dtype=0, **rows("k"), **rows("v"), **rows("q"), T=5, Hq=8, Hk=2, D=128, qw=FAKE, kw=FAKE, eps=1e-6, pos=FAKE, axes=2,
                sections=_sections(24, 40), R=128, freq=FAKE, il=0, **rows("qo"), kc=FAKE, vc=FAKE, **PAGES, stream=0)


def attend_args():
    return dict(dtype=0, **rows("q"), kc=FAKE, vc=FAKE, **PAGES, T=5, Hq=8, Hk=2, D=128, max_q=2, max_kv=64, scale=0.1, causal=1, window=0,
                **rows("o"), lse=FAKE, ws=FAKE, ws_bytes=1 << 40, stream=0)


def pages(changes):
    """Those that hold for codes: strides are multiples of 16 elements."""
    return [c for c in changes if "cache" not in c]


def test_append_refusals(A):
    check(A.bevpool_kv_append_scaled, append_args(),
          ROTARY_INVALID + HEADS_INVALID + pages(PAGES_INVALID) + SCALES_INVALID
          + [dict(k=0), dict(v=0), dict(v_hs=2), dict(qo=0), dict(q=FAKE + 4), dict(Hq=0), dict(hs=2056), dict(ss=8), dict(ss=136)],
          HEADS_UNSUPPORTED + pages(PAGES_UNSUPPORTED) + [dict(D=32), dict(D=96), dict(D=256)])
    assert A.bevpool_kv_append_scaled(*{**append_args(), "T": 0, "k": 0, "q": 0}.values()) == 0


def test_attention_refusals(A):
    check(A.bevpool_paged_attention_scaled, attend_args(),
          HEADS_INVALID + pages(PAGES_INVALID) + SCALES_INVALID
          + [dict(q=0), dict(o=0), dict(o=FAKE + 8), dict(q_ts=2), dict(Hk=3), dict(max_q=-1), dict(max_kv=-1), dict(scale=float("nan")),
             dict(scale=float("inf")), dict(scale=0.0), dict(scale=-1.0), dict(scale=2.0 ** 80), dict(scale=2.0 ** -79), dict(window=-1), dict(causal=0, window=5),
             dict(lse=FAKE + 2), dict(n_seqs=65536), dict(max_kv=2 ** 31 - 1), dict(max_q=2 ** 31 - 1), dict(T=1 << 28, Hq=32), dict(ss=136)],
          HEADS_UNSUPPORTED + pages(PAGES_UNSUPPORTED) + [dict(D=96), dict(D=256), dict(D=32)],
          [dict(ws=0, max_kv=100000), dict(ws=FAKE + 64, max_kv=100000), dict(ws_bytes=16, max_kv=100000)])
    for change in (dict(T=0, q=0), dict(n_seqs=0), dict(max_q=0)):
        assert A.bevpool_paged_attention_scaled(*{**attend_args(), **change}.values()) == 0


def test_helpers_refuse(A):
    """CPU tensors, and tensors that require gradients."""
    from depth_weighted_scatter_gb300.bevpool import BevpoolError

    q, c = torch.zeros(3, 4, 64, dtype=torch.float16), torch.zeros(4, 4, 16, 64, dtype=torch.uint8)
    s, pos, f = torch.zeros(4, 4), torch.zeros(3, dtype=torch.int32), torch.zeros(32)
    t, n, cu = torch.zeros(3, 2, dtype=torch.int32), torch.zeros(3, dtype=torch.int32), torch.zeros(4, dtype=torch.int32)
    g = s.clone().requires_grad_()
    for call in (lambda s: A.kv_append_scaled(q, q, c, c, s, s, t, n, cu, pos, f),
                 lambda s: A.paged_attention_scaled(q, c, c, s, s, t, n, cu, max_q_len=1, max_kv_len=4)):
        with pytest.raises(BevpoolError, match="device"):
            call(s)
        with pytest.raises(BevpoolError, match="gradients are not recorded"):
            call(g)
        with pytest.raises(BevpoolError, match="tensor"):
            call(1.0)


def test_workspace_sizes(A):
    """Chunks of few rows are cut for the kernel that reads them; others are those of the plain cache."""
    plain, scaled = A.bevpool_paged_attention_workspace_size, A.bevpool_paged_attention_scaled_workspace_size
    assert scaled(0, 5, 8, 2, 128, 2, 64, 0) == 0 and scaled(3, 5, 8, 3, 128, 2, 64, 0) == 0 and scaled(3, 5, 8, 2, 96, 2, 64, 0) == 0
    assert 0 < scaled(1, 1, 8, 2, 128, 1, 100000, 0) <= scaled(2, 2, 8, 2, 128, 1, 100000, 0)
    for sizes in ((2, 700, 16, 8, 64, 700, 5000, 0), (1, 3, 16, 4, 128, 3, 5000, 0)):      # tiles; nine to sixteen rows
        assert scaled(*sizes) == plain(*sizes) > 0
