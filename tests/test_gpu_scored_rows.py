"""GPU: scored decode at every number of query rows a CTA is compiled for (up to
4, 8, 16 and 32 at the head dims that have them) and both refill schemes, against
the definition in 64 bits; the failure path where each warp fetches its own slice."""
import numpy as np
import pytest
import torch

import quantized_kv_cache_append_gb300 as kvq
from tests.test_gpu_scored import Case, dev, ints, slopes_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _library():
    if not torch.cuda.is_available():
        pytest.fail("the GPU suite needs a CUDA device")
    kvq.build()
    kvq.load_library()


# G, W: 3, 4, 5, 8, 9, 16, 17 and 32 rows
ROWS = [(3, 1), (2, 2), (5, 1), (8, 1), (2, 4), (3, 3), (4, 4), (17, 1), (8, 4)]


@pytest.mark.parametrize("fmt", ["f16", "q8", "k8v4"])
@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("G,W", ROWS)
@pytest.mark.parametrize("bs,lens", [(16, [1100]), (64, [700, 0, 33, 260]), (256, [65, 1500])])
def test_rows(bs, lens, G, W, hd, fmt):
    rng = np.random.default_rng([G, W, hd, bs])
    c = Case(rng, fmt, 2, G, hd, W, bs, lens)
    c.check(cap=20.0)
    c.check(window=130, slopes=slopes_of(2 * G), first=rng.integers(0, np.maximum(c.lens, 1)))


@pytest.mark.parametrize("fmt", ["f16", "q8", "k8v4"])
@pytest.mark.parametrize("hd,G,W", [(256, 2, 1), (256, 8, 1), (256, 4, 4), (256, 8, 4), (128, 8, 1), (128, 4, 4), (64, 4, 4),
                                    (64, 8, 4)])
@pytest.mark.parametrize("lens", [[700, 0, 300], [900], [60]])
def test_lost_waits_of_slices(lens, hd, G, W, fmt):
    rng = np.random.default_rng([hd, G, W])
    n = len(lens)
    c = Case(rng, fmt, 2, G, hd, W, 64, lens, max_ctx=1000)
    for scores in (kvq.make_scores(20.0), kvq.make_scores(0.0, 256, dev(slopes_of(2 * G)))):
        want = c.run(scores)
        q, out = dev(c.q), torch.zeros_like(want)
        ws = torch.empty(kvq.kvq_scored_workspace_bytes(c.pool.cache, scores, n, W, 2 * G, c.max_ctx), dtype=torch.uint8,
                         device="cuda")
        st = kvq.kvq_decode_attn_scored_lost_wait_test(
            c.pool.cache, scores, q, n, W, 2 * G, ints(c.lens), c.max_ctx, ints(c.table), c.table.shape[1], c.sm_scale, out,
            ws, ws.numel(), 3000, 16)
        assert st == kvq.KVQ_OK
        torch.cuda.synchronize()
        held = torch.tensor([L > 0 for L in lens], device="cuda")
        assert out[held].isnan().all() and not out[~held].any()
        assert torch.equal(c.run(scores), want) and bool(want[held].isfinite().all())
