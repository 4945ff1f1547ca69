"""GPU: a NaN among the keys or queries of a list reaches every row that reads
it, and no other, whether the list's splits meet through the workspace, in a
cluster, or the list is one split."""
import math

import numpy as np
import pytest
import torch

import quantized_kv_cache_append_gb300 as kvq
from tests import plain_blocks as plain
from tests.test_gpu_blocks import dev, fill_pool, i32, lens_rows, queries, random_lists

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _library():
    if not torch.cuda.is_available():
        pytest.fail("the GPU suite needs a CUDA device")
    kvq.build()
    kvq.load_library()


@pytest.mark.parametrize("fmt", ["f16", "q8", "k8v4"])
@pytest.mark.parametrize("n_seq", [1, 40, 75, 310])
@pytest.mark.parametrize("hd,G", [(64, 4), (128, 8), (256, 2)])
def test_a_nan_reaches_the_rows_that_read_it_and_no_others(fmt, n_seq, hd, G):
    rng = np.random.default_rng(n_seq + hd)
    bs, n_sel, n_kv, n_blocks = 16, 32, 2, 40
    p, h = fill_pool(rng, fmt, n_blocks, n_kv, bs, hd)
    q = queries(rng, n_seq, 1, n_kv * G, hd)
    blocks, lens = random_lists(rng, n_seq, 1, n_kv, n_sel, n_blocks, bs)
    blk, head, slot = int(blocks[0, 0, 1, 7]), 1, 5       # a live cell of the first sequence's list
    lens[0, 0, 1] = n_sel * bs
    K, V = plain.pool_rows(fmt, h["k"], h["v"], h["ks"], h["vs"])
    sm = float(np.float32(1 / math.sqrt(hd)))

    def run(x):
        out = p.decode_selected(dev(x), i32(blocks), i32(lens), sm)
        torch.cuda.synchronize()
        return out.cpu().numpy()

    def check(out, rows):
        nan = np.isnan(out)
        assert (nan.all(-1) == rows).all() and (nan.any(-1) == rows).all()
        want, tol = plain.attention(fmt, K, V, q, blocks, lens, bs, sm)
        assert (np.abs(out - want).max(-1)[~rows] <= tol[~rows]).all()

    # a query
    x = q.copy()
    x[0, 0, 1, hd // 3] = np.nan
    x[n_seq - 1, 0, G, 0] = np.nan
    rows = np.isnan(x).any(-1) & (lens_rows(lens, q) > 0)
    check(run(x), rows)

    # a key (an int8 key's scale)
    if fmt == "f16":
        p.k[blk, head, slot, hd // 2] = float("nan")
    else:
        p.ks[blk, head, slot, 0] = float("nan")
    at = np.arange(n_sel)
    reads = ((blocks == blk) & (at * bs + slot < lens[..., None])).any(-1)
    reads[..., 1 - head] = False
    assert reads[0, 0, head]
    check(run(q), np.repeat(reads, G, -1))
