"""How the attention over a cache with page scales cuts few rows' keys, seen from the workspace that it asks for (no GPU
needed)."""
import pytest

torch = pytest.importorskip("torch")

PLACES = 152 * 3                                            # CTAs that the GPU holds at a time


@pytest.fixture(scope="module")
def A():
    from depth_weighted_scatter_gb300 import _build

    _build.build()
    from depth_weighted_scatter_gb300 import attention

    return attention


def chunks(A, n_seqs, Hk, keys, D=128, rows=4):
    """Chunks of a request: the partial results of one are a row of D sums, a maximum and a sum for each query row."""
    size = A.bevpool_paged_attention_scaled_workspace_size(n_seqs, n_seqs, Hk * rows, Hk, D, 1, keys, 0)
    n, rest = divmod(size, n_seqs * Hk * rows * (D + 2) * 4)
    assert rest == 0
    return n or 1


@pytest.mark.parametrize("n_seqs, Hk", [(1, 1), (1, 8), (1, 16), (2, 8), (3, 8), (5, 7), (6, 8), (8, 8), (64, 1), (13, 4)])
@pytest.mark.parametrize("keys", [131072, 40000, 4097])
def test_few_pairs_are_one_wave(A, n_seqs, Hk, keys):
    """Up to 64 pairs of a request and key head: no more CTAs than the GPU holds, and, where keys allow, most of its places."""
    n = chunks(A, n_seqs, Hk, keys)
    ctas = n * n_seqs * Hk
    assert ctas <= PLACES
    if keys / n >= 640:                                     # chunks are multiples of 64 keys
        assert (n + 1) * n_seqs * Hk > 0.8 * PLACES


def test_many_pairs_are_waves_for_ragged_lengths(A):
    assert chunks(A, 64, 8, 8192) * 64 * 8 > 4 * PLACES
