"""GPU: the attention over block lists keeps the precision it is built for
where rounding bites: weights times small V scales, and int8 keys in sums that
nearly cancel.  One cell of each list has a value, so an output is that
cell's weight, times the value, over the row's sum."""
import numpy as np
import pytest
import torch

import quantized_kv_cache_append_gb300 as kvq
from quantized_kv_cache_append_gb300.pool import PagedPool
from tests.test_gpu_blocks import FMT, dev, i32

pytestmark = pytest.mark.gpu

BS, N = 64, 48          # lists of one block each, as many as blocks


@pytest.fixture(scope="module", autouse=True)
def _library():
    if not torch.cuda.is_available():
        pytest.fail("the GPU suite needs a CUDA device")
    kvq.build()
    kvq.load_library()


def one_value_pool(rng, fmt, hd, scale):
    """Block i: only cell at[i] has a value, in dim 3."""
    p = PagedPool(FMT[fmt], 1, hd, BS, N)
    at = rng.integers(0, BS, N)
    vs = np.full(tuple(p.vs.shape), scale, np.float16)
    if fmt == "q8":
        v = np.zeros((N, 1, BS, hd), np.int8)
        v[np.arange(N), 0, at, 3] = 127
        value = 127.0
    else:
        v = np.full((N, 1, BS, hd // 2), 0x88, np.uint8)     # code 8 is zero
        v[np.arange(N), 0, at, 1] = 0xf8
        value = 7.0 / hd                                     # rotated back: +- that in every dim
    p.v.copy_(dev(v))
    p.vs.copy_(dev(vs))
    return p, at, value * float(np.float16(scale))


def check(p, q, z, at, value, sm, tol):
    """z [N][G][BS]: the logits; tol: relative."""
    out = p.decode_selected(dev(q), i32(np.arange(N).reshape(N, 1, 1, 1)), i32(np.full((N, 1, 1), BS)), sm)
    torch.cuda.synchronize()
    w = np.exp(z - z.max(-1, keepdims=True))
    want = w[np.arange(N), :, at] / w.sum(-1) * value
    got = np.abs(out.cpu().numpy()[:, 0, :, 3].astype(np.float64))
    err = np.abs(got / want - 1).max()
    assert err <= tol, err


@pytest.mark.parametrize("fmt", ["q8", "k8v4"])
@pytest.mark.parametrize("hd,G", [(64, 4), (128, 4), (128, 12), (256, 8)])
def test_small_value_scales_keep_the_weights_precision(fmt, hd, G):
    # Logits 0 .. 1 from one product each.  In log2 units (below 1.5): q's fp16
    # halves 2^-22 and fp32 product 2^-24 relative, the subtraction from a
    # reference 8 below the maximum 2^-22: 3 * 2^-22 in all, so 2.1 * 2^-22 of p,
    # 2^-22 from the exponential; the same again in the row's sum; p times the
    # scale as fp16 halves 2^-21 (from 2^-12 * 2^8 * e^-1 up: the lo half's
    # smallest step, 2^-24, is off by 2^-25 of at least 2^-6: 2^-19); fp32
    # products and the last division 2^-22: below 2^-18 together.
    rng = np.random.default_rng(hd + G)
    p, at, value = one_value_pool(rng, fmt, hd, 1.37 * 2.0 ** -12)
    k = np.zeros((N, 1, BS, hd), np.int8)
    k[:, 0, :, 7] = rng.integers(0, 127, (N, BS))
    p.k.copy_(dev(k))
    p.ks.fill_(2.0 ** -7)
    q = np.zeros((N, 1, G, hd), np.float32)
    q[..., 7] = 1 - rng.random((N, 1, G)) * 0.3
    z = q[:, 0, :, 7, None].astype(np.float64) * k[:, :, :, 7] * 2.0 ** -7
    check(p, q, z, at, value, 1.0, 2.0 ** -18)


@pytest.mark.parametrize("hd,G", [(64, 4), (128, 4), (128, 12), (256, 8)])
def test_int8_keys_whose_products_cancel(hd, G):
    # Codes of +-1 against queries near 1: a logit is a small difference of
    # hd products.  Each of hd / 16 steps and of the additions that join
    # groups and halves is off by at most 2^-22 of the sum of |q k| (the
    # tensor cores add 16 products at 2^-23 and round once more): (hd / 16 +
    # 8) * 2^-22 of it.  The weight and the row's sum both carry that.
    rng = np.random.default_rng(hd + G)
    p, at, value = one_value_pool(rng, "q8", hd, 1.0)
    k = rng.choice([-1, 1], (N, 1, BS, hd)).astype(np.int8)
    p.k.copy_(dev(k))
    p.ks.fill_(1.0)
    q = (1 + 0.3 * rng.random((N, 1, G, hd))).astype(np.float32)
    sm = 0.125
    z = sm * np.einsum("ngd,ncd->ngc", q[:, 0].astype(np.float64), k[:, 0].astype(np.float64))
    sums = sm * np.abs(q).sum(-1).max()
    check(p, q, z, at, value, sm, 2 * (hd / 16 + 8) * 2.0 ** -22 * sums + 2.0 ** -18)
