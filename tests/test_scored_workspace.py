"""CPU: the workspace of scored batches is bounded by the splits there can be,
with a window as without one."""
import pytest

import quantized_kv_cache_append_gb300 as kvq

A = 1 << 32
TILE = 64          # cells a split has at least


@pytest.fixture(scope="module", autouse=True)
def _library():
    kvq.build()
    kvq.load_library()


def cache(n_kv, hd):
    return kvq.make_cache(kvq.KVQ_Q8, n_kv, hd, 64, 100000, A, 2 * A, 3 * A, 4 * A)


def most_bytes(n_seq, W, n_kv, G, hd, cells):
    """A partial (hd sums, maximum and weight sum) of every row for each tile a
    sequence can have, one more split than sequences, the table of first splits,
    three roundings to 256 bytes."""
    splits = max(n_seq * -(-cells // TILE), n_seq + 1)
    return n_kv * splits * G * W * (hd + 2) * 4 + 4 * (n_seq + 1) + 3 * 256


@pytest.mark.parametrize("n_seq", [2, 3, 16, 100, 128, 129, 300])
@pytest.mark.parametrize("n_kv,G,hd,W", [(1, 4, 128, 1), (8, 4, 128, 2), (2, 8, 256, 4), (32, 1, 64, 1)])
@pytest.mark.parametrize("window,max_ctx", [(64, 100000), (1, 100000), (0, 64), (0, 1000), (700, 100000), (100, 90)])
def test_bounded_by_the_splits_there_can_be(n_seq, n_kv, G, hd, W, window, max_ctx):
    got = kvq.kvq_scored_workspace_bytes(cache(n_kv, hd), kvq.make_scores(window=window), n_seq, W, n_kv * G, max_ctx)
    # (a window's cells may begin inside a tile: one tile more)
    cells = max_ctx if not 0 < window < max_ctx else min(max_ctx, window + W - 1 + TILE - 1)
    assert 0 < got <= most_bytes(n_seq, W, n_kv, G, hd, cells)


@pytest.mark.parametrize("n_seq", [2, 16, 128])
def test_a_window_bounds_it(n_seq):
    size = lambda window: kvq.kvq_scored_workspace_bytes(cache(1, 128), kvq.make_scores(window=window), n_seq, 1, 4, 1 << 20)
    assert size(64) < size(0) and size(64) <= size(1000) <= size(0)
