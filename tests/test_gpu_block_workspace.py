"""GPU: kvq_sparse_decode_attn in a workspace sized for another batch: any
size from 256 bytes up is served, and nothing past it is written."""
import math

import numpy as np
import pytest
import torch

import quantized_kv_cache_append_gb300 as kvq
from tests import plain_blocks as plain
from tests.test_gpu_blocks import dev, fill_pool, i32, queries, random_lists

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _library():
    if not torch.cuda.is_available():
        pytest.fail("the GPU suite needs a CUDA device")
    kvq.build()
    kvq.load_library()


@pytest.mark.parametrize("fmt", ["f16", "q8", "k8v4"])
@pytest.mark.parametrize("hd,G,bs,n_sel", [(64, 20, 16, 40), (128, 4, 64, 64), (128, 12, 16, 5), (256, 32, 32, 9)])
def test_a_batch_that_shrinks_keeps_its_workspace(fmt, hd, G, bs, n_sel):
    rng = np.random.default_rng(hd + G)
    n_kv, n_blocks = 2, n_sel + 3
    p, h = fill_pool(rng, fmt, n_blocks, n_kv, bs, hd)
    K, V = plain.pool_rows(fmt, h["k"], h["v"], h["ks"], h["vs"])
    sm = float(np.float32(1 / math.sqrt(hd)))
    full = kvq.kvq_sparse_workspace_bytes(p.cache, 400, 1, n_kv * G, n_sel)
    assert full == 256                               # in clusters
    for n_seq in (1, 3, 20):
        need = kvq.kvq_sparse_workspace_bytes(p.cache, n_seq, 1, n_kv * G, n_sel)
        q = queries(rng, n_seq, 1, n_kv * G, hd)
        blocks, lens = random_lists(rng, n_seq, 1, n_kv, n_sel, n_blocks, bs)
        lens[-1, 0, -1] = 0
        want, tol = plain.attention(fmt, K, V, q, blocks, lens, bs, sm)
        for size in sorted({full, max(256, need // 2), max(256, need - 1), need}):
            ws = torch.full((max(need, size) + 4096,), 0x5a, dtype=torch.uint8, device="cuda")
            out = torch.full(q.shape, float("nan"), device="cuda")
            st = kvq.kvq_sparse_decode_attn(p.cache, dev(q), n_seq, 1, n_kv * G, i32(blocks), i32(lens), n_sel, sm,
                                            out, ws, size)
            assert st == kvq.KVQ_OK, kvq.kvq_status_string(st)
            torch.cuda.synchronize()
            assert (np.abs(out.cpu().numpy() - want).max(-1) <= tol).all()
            assert (ws[size:] == 0x5a).all()
        assert kvq.kvq_sparse_decode_attn(p.cache, dev(q), n_seq, 1, n_kv * G, i32(blocks), i32(lens), n_sel, sm, out,
                                          ws, 255) == kvq.KVQ_ERR_WORKSPACE
