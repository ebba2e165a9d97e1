"""The token operators' C entry points reject bad arguments on the host (no
GPU needed: these calls return before any CUDA work)."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

FAKE = 1 << 20   # never dereferenced: every call below fails validation first


@pytest.fixture(scope="module")
def A():
    from depth_weighted_scatter_gb300 import _build

    _build.build()
    from depth_weighted_scatter_gb300 import attention

    return attention


def _sections(*n):
    return (ctypes.c_int32 * len(n))(*n)


def rows(name):
    return {name: FAKE, name + "_ts": 1024, name + "_hs": 128}


def norm_args():
    return dict(dtype=0, **rows("q"), **rows("k"), T=5, Hq=8, Hk=2, D=128, qw=FAKE, kw=FAKE, eps=1e-6, pos=FAKE, axes=2,
                sections=_sections(24, 40), R=128, freq=FAKE, il=0, **rows("qo"), **rows("ko"), stream=0)


def back_args(A):
    return dict(dtype=3, **rows("gq"), **rows("gk"), **rows("q"), **rows("k"), T=5, Hq=8, Hk=2, D=128, qw=FAKE, kw=FAKE,
                eps=1e-6, pos=FAKE, axes=2, sections=_sections(24, 40), R=128, freq=FAKE, il=0, **rows("dq"), **rows("dk"),
                dqw=FAKE, dkw=FAKE, ws=FAKE, ws_bytes=A.bevpool_qk_norm_rope_backward_workspace_size(5, 8, 2, 128),
                stream=0)


PAGES = dict(ps=4096, ss=128, hs=2048, n_pages=10, page=16, table=FAKE, table_pages=4, kv_len=FAKE, cu_q=FAKE, n_seqs=3)


def append_args():
    return dict(dtype=0, cache=0, **rows("k"), **rows("v"), **rows("q"), T=5, Hq=8, Hk=2, D=128, qw=FAKE, kw=FAKE, eps=1e-6,
                pos=FAKE, axes=2, sections=_sections(24, 40), R=128, freq=FAKE, il=0, **rows("qo"), kc=FAKE, vc=FAKE,
                **PAGES, k_scale=1.0, v_scale=1.0, stream=0)


def attend_args():
    return dict(dtype=0, cache=0, **rows("q"), kc=FAKE, vc=FAKE, **PAGES, T=5, Hq=8, Hk=2, D=128, max_q=2, max_kv=64,
                scale=0.1, causal=1, window=0, k_scale=1.0, v_scale=1.0, **rows("o"), lse=FAKE, ws=FAKE,
                ws_bytes=1 << 40, stream=0)


def check(fn, args, invalid=(), unsupported=(), workspace=()):
    for changes, status in ((invalid, 1), (unsupported, 3), (workspace, 4)):
        for change in changes:
            assert set(change) <= set(args), change
            assert fn(*{**args, **change}.values()) == status, change


ROTARY_INVALID = [dict(pos=0), dict(pos=FAKE + 2), dict(freq=0), dict(sections=None), dict(axes=0), dict(axes=5),
                  dict(R=0), dict(R=8), dict(R=120), dict(R=144), dict(sections=_sections(24, 41)),
                  dict(sections=_sections(-1, 65)), dict(sections=_sections(65, -1)),
                  dict(sections=_sections(2 ** 31 - 1, 2 ** 31 - 1)), dict(eps=-1.0), dict(eps=float("nan")),
                  dict(eps=float("inf")), dict(kw=FAKE + 1)]
HEADS_UNSUPPORTED = [dict(D=24), dict(D=100), dict(D=264), dict(dtype=1), dict(dtype=2), dict(dtype=4), dict(dtype=-1)]
HEADS_INVALID = [dict(T=-1), dict(Hk=0), dict(Hk=-1), dict(Hk=65536), dict(D=0), dict(D=-8)]


def test_norm_rope_refusals(A):
    check(A.bevpool_qk_norm_rope, norm_args(),
          ROTARY_INVALID + HEADS_INVALID + [dict(q=0), dict(k=FAKE + 8), dict(qo=0), dict(ko=FAKE + 2), dict(q_ts=1020),
                                            dict(q_hs=-8), dict(ko_ts=4), dict(qo_hs=1 << 40), dict(Hq=0), dict(qw=FAKE + 2)],
          HEADS_UNSUPPORTED)


def test_norm_rope_backward_refusals(A):
    check(A.bevpool_qk_norm_rope_backward, back_args(A),
          ROTARY_INVALID + HEADS_INVALID + [dict(gq=0), dict(gk=FAKE + 8), dict(dq=0), dict(dk=FAKE + 4), dict(q=0),
                                            dict(gq_ts=3), dict(dqw=0), dict(dkw=0), dict(qw=0), dict(dqw=FAKE + 1)],
          HEADS_UNSUPPORTED,
          [dict(ws=0), dict(ws=FAKE + 64), dict(ws_bytes=back_args(A)["ws_bytes"] - 1)])
    size = A.bevpool_qk_norm_rope_backward_workspace_size
    assert size(0, 8, 2, 128) == 0 and size(-1, 8, 2, 128) == 0 and size(5, 8, 2, 100) == 0
    assert 0 < size(5, 8, 2, 128) <= size(50000, 8, 2, 128) == size(100000, 8, 2, 128)


PAGES_INVALID = [dict(kc=0), dict(vc=FAKE + 8), dict(ps=-8), dict(ps=4), dict(ss=1 << 40), dict(hs=12), dict(n_pages=0),
                 dict(page=0), dict(table=0), dict(table=FAKE + 2), dict(kv_len=0), dict(cu_q=0), dict(table_pages=0),
                 dict(table_pages=2 ** 31 - 1), dict(n_seqs=-1)]
PAGES_UNSUPPORTED = [dict(page=8), dict(page=48), dict(page=512), dict(cache=3), dict(cache=2)]


def test_append_refusals(A):
    check(A.bevpool_kv_append, append_args(),
          ROTARY_INVALID + HEADS_INVALID + PAGES_INVALID
          + [dict(k=0), dict(v=0), dict(v_hs=2), dict(qo=0), dict(q=FAKE + 4), dict(Hq=0),
             dict(cache=1, k_scale=0.0), dict(cache=1, v_scale=-1.0), dict(cache=1, k_scale=float("inf")),
             dict(cache=1, v_scale=float("nan")), dict(cache=1, v_scale=1e-45), dict(cache=1, ss=8)],
          HEADS_UNSUPPORTED + PAGES_UNSUPPORTED)


def test_attention_refusals(A):
    check(A.bevpool_paged_attention, attend_args(),
          HEADS_INVALID + PAGES_INVALID
          + [dict(q=0), dict(o=0), dict(o=FAKE + 8), dict(q_ts=2), dict(Hk=3), dict(max_q=-1), dict(max_kv=-1),
             dict(scale=float("nan")), dict(scale=float("inf")), dict(scale=0.0), dict(scale=-1.0), dict(window=-1),
             dict(causal=0, window=5), dict(lse=FAKE + 2), dict(cache=1, k_scale=0.0),
             dict(cache=1, v_scale=float("inf")), dict(n_seqs=65536), dict(max_kv=2 ** 31 - 1),
             dict(max_q=2 ** 31 - 1), dict(T=1 << 28, Hq=32)],
          HEADS_UNSUPPORTED + PAGES_UNSUPPORTED + [dict(D=96), dict(D=256), dict(D=32)])


def test_no_tokens_enqueue_nothing(A):
    """Zero tokens (or requests) are valid, whatever the pointers."""
    none = dict(q=0, k=0, T=0)
    assert A.bevpool_qk_norm_rope(*{**norm_args(), **none}.values()) == 0
    assert A.bevpool_kv_append(*{**append_args(), **none, "v": 0}.values()) == 0
    for change in (dict(T=0, q=0), dict(n_seqs=0), dict(max_q=0)):
        assert A.bevpool_paged_attention(*{**attend_args(), **change}.values()) == 0


def test_helpers_refuse(A):
    """The tensor helpers check types and shapes before the call (CPU tensors are refused)."""
    from depth_weighted_scatter_gb300.bevpool import BevpoolError

    def refused(fn, *args, **kw):
        with pytest.raises(BevpoolError):
            fn(*args, **kw)

    q = torch.zeros(3, 4, 64, dtype=torch.float16)
    pos, f = torch.zeros(3, dtype=torch.int32), torch.zeros(32)
    c = torch.zeros(4, 4, 16, 64, dtype=torch.float16)
    t, n, cu = torch.zeros(3, 2, dtype=torch.int32), torch.zeros(3, dtype=torch.int32), torch.zeros(4, dtype=torch.int32)
    # no CUDA tensors
    refused(A.qk_norm_rope, q, q, pos, f)
    refused(A.qk_norm_rope_backward, q, q, q, q, pos, f)
    refused(A.kv_append, q, q, c, c, t, n, cu, pos, f)
    refused(A.paged_attention, q, c, c, t, n, cu, max_q_len=1, max_kv_len=4)
    # no head tensors, no 16-bit type, no tensors
    refused(A.qk_norm_rope, q[0], q[0], pos, f)
    refused(A.qk_norm_rope, q.float(), q.float(), pos, f)
    refused(A.qk_norm_rope, [1.0], q, pos, f)
    refused(A.paged_attention, q, c, None, t, n, cu, max_q_len=1, max_kv_len=4)
    with pytest.raises(BevpoolError) as e:
        A.qk_norm_rope(q.double(), q, pos, f)
    assert e.value.status == 3


@pytest.mark.gpu
def test_helpers_refuse_on_the_gpu(A):
    """What does not match is refused before anything is enqueued."""
    from depth_weighted_scatter_gb300.bevpool import BevpoolError

    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")

    def refused(fn, *args, **kw):
        with pytest.raises(BevpoolError):
            fn(*args, **kw)

    z = lambda *s, dtype=torch.float16: torch.zeros(*s, dtype=dtype, device="cuda")  # noqa: E731
    q, k, pos, f = z(3, 4, 64), z(3, 2, 64), z(3, dtype=torch.int32), z(32, dtype=torch.float32)
    assert A.qk_norm_rope(q, k, pos, f)[0].shape == q.shape
    for bad in [(q, k[:2], pos, f), (q, k.bfloat16(), pos, f), (q, k.cpu(), pos, f), (q, z(3, 64, 2).transpose(1, 2), pos, f),
                (q, k, pos.long(), f), (q, k, pos[:2], f), (q, k, z(3, 5, dtype=torch.int32), f), (q, k, pos, f.double()),
                (q, k, pos, f[:4]), (q, k, pos.cpu(), f), (q, k, z(3, 2, dtype=torch.int32), f)]:
        refused(A.qk_norm_rope, *bad)
    for more in [dict(sections=[31]), dict(sections=[16, 16]), dict(q_weight=z(64)), dict(k_weight=z(32, dtype=torch.float32)),
                 dict(q_out=z(3, 2, 64)), dict(k_out=k.float()), dict(eps=-1.0)]:
        refused(A.qk_norm_rope, q, k, pos, f, **more)
    refused(A.qk_norm_rope_backward, k, k, q, k, pos, f)
    w = z(64, dtype=torch.float32)
    refused(A.qk_norm_rope_backward, q, k, q, k, pos, f, q_weight=w, workspace=z(16, dtype=torch.uint8))
    c, t, n, cu = z(4, 2, 16, 64), z(3, 2, dtype=torch.int32), z(3, dtype=torch.int32), z(4, dtype=torch.int32)
    assert A.paged_attention(q, c, c.clone(), t, n, cu, max_q_len=1, max_kv_len=4).shape == q.shape
    for bad in [(c, c[:3], t, n, cu), (c, c.float(), t, n, cu), (c.float(), c.float(), t, n, cu), (c, c, t, n, cu[:3]),
                (c, c, t, n.long(), cu), (c, c, t.t(), n, cu), (c, c, t[0], n, cu), (c[0], c[0], t, n, cu),
                (c, c.transpose(1, 2).contiguous().transpose(1, 2), t, n, cu), (c.bfloat16(), c.bfloat16(), t, n, cu),
                (z(4, 2, 24, 64), z(4, 2, 24, 64), t, n, cu), (z(4, 2, 16, 32), z(4, 2, 16, 32), t, n, cu),
                (z(4, 3, 16, 64), z(4, 3, 16, 64), t, n, cu)]:
        refused(A.paged_attention, q, *bad, max_q_len=1, max_kv_len=4)
        refused(A.kv_append, k, k, *bad, pos, f)
    for more in [dict(max_q_len=-1), dict(max_kv_len=1 << 40), dict(window=-1), dict(window=4, causal=False), dict(scale=0.0),
                 dict(out=q.bfloat16()), dict(out=z(3, 64, 4).transpose(1, 2))]:
        refused(A.paged_attention, q, c, c, t, n, cu, **{**dict(max_q_len=1, max_kv_len=4), **more})
    refused(A.kv_append, k, q, c, c, t, n, cu, pos, f)
    refused(A.kv_append, k, k, c, c, t, n, cu, pos, f, q_out=q)
    refused(A.kv_append, k, k, c.view(torch.uint8)[..., :64].contiguous(), c.view(torch.uint8)[..., :64].contiguous(), t, n, cu,
            pos, f, k_scale=0.0)
    torch.cuda.synchronize()
