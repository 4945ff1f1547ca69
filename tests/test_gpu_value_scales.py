"""GPU: attention over V scales up to fp16's largest, int8 and K8V4.  The V
scales are folded into the softmax weights, which then enter the tensor cores
as fp16 pairs: a weight times a scale has to stay in fp16's range.  Over block
lists and dense, against the plain 64-bit form of tests/plain_blocks.py."""
import math

import numpy as np
import pytest
import torch

import quantized_kv_cache_append_gb300 as kvq
from tests import plain_blocks as plain
from tests.test_gpu_blocks import dev, fill_pool, i32, queries, random_lists, tables

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _library():
    if not torch.cuda.is_available():
        pytest.fail("the GPU suite needs a CUDA device")
    kvq.build()
    kvq.load_library()


def set_scales(rng, p, h, kind, S):
    """V scales of magnitude S in some or all of the pool's cells."""
    vs = h["vs"]
    sign = rng.choice([-1.0, 1.0], vs.shape)
    if kind == "all":
        at = np.ones(vs.shape[:3], bool)
    elif kind == "some":
        at = rng.random(vs.shape[:3]) < 0.1
    else:                       # one 64-dim group or 32-dim block of one cell
        at = np.zeros(vs.shape[:3], bool)
        at[:, :, 3] = True
        sign[..., 1:] = 0
    h["vs"] = np.where(at[..., None] & (sign != 0), (S * sign), vs).astype(np.float16)
    p.vs.copy_(dev(h["vs"]))
    return at


def lowest_rounding(h, fmt, live_cells):
    """What fp16's smallest step (2^-24, off by half of it) may leave in a sum
    of weights (the largest 1) times scales times codes, per unit of the sum
    of the weights: at most one such rounding for each live cell."""
    return live_cells * 2.0 ** -25 * (127 if fmt == "q8" else 8)


def weights_sum(K, q, blocks, lens, bs, sm):
    """sum of exp(z - max z) per query row: [n_seq][W][n_q]."""
    n_seq, W, n_q, _ = q.shape
    n_kv = K.shape[1]
    G = n_q // n_kv
    l = np.ones((n_seq, W, n_q))
    for b in range(n_seq):
        for w in range(W):
            for g in range(n_kv):
                n = int(lens[b, w, g])
                if n == 0:
                    continue
                ids, slot = np.repeat(blocks[b, w, g], bs)[:n], np.arange(n) % bs
                z = sm * (q[b, w, g * G:(g + 1) * G].astype(np.float64) @ K[ids, g, slot].T)
                l[b, w, g * G:(g + 1) * G] = np.exp(z - z.max(1, keepdims=True)).sum(1)
    return l


def check_lists(fmt, p, h, q, blocks, lens):
    sm = float(np.float32(1 / math.sqrt(p.head_dim)))
    out = p.decode_selected(dev(q), i32(blocks), i32(lens), sm)
    torch.cuda.synchronize()
    out = out.cpu().numpy()
    K, V = plain.pool_rows(fmt, h["k"], h["v"], h["ks"], h["vs"])
    want, tol = plain.attention(fmt, K, V, q, blocks, lens, p.block_size, sm)
    tol = tol + lowest_rounding(h, fmt, blocks.shape[-1] * p.block_size) / weights_sum(K, q, blocks, lens,
                                                                                      p.block_size, sm)
    assert np.isfinite(out).all()
    err = np.abs(out - want).max(-1)
    assert (err <= tol).all(), (err / tol).max()


@pytest.mark.parametrize("fmt", ["q8", "k8v4"])
@pytest.mark.parametrize("S", [128, 128.125, 255, 255.875, 256, 1000, 65504])
@pytest.mark.parametrize("n_seq", [1, 75])      # splits through the workspace, and in clusters
def test_lists_with_large_value_scales(fmt, S, n_seq):
    rng = np.random.default_rng(int(8 * S) + n_seq)
    bs, n_sel, n_kv, G, hd = 16, 32, 2, 4, 128
    for kind in ("all", "some", "one"):
        p, h = fill_pool(rng, fmt, 40, n_kv, bs, hd)
        set_scales(rng, p, h, kind, S)
        blocks, lens = random_lists(rng, n_seq, 1, n_kv, n_sel, 40, bs)
        check_lists(fmt, p, h, queries(rng, n_seq, 1, n_kv * G, hd), blocks, lens)


@pytest.mark.parametrize("fmt", ["q8", "k8v4"])
@pytest.mark.parametrize("hd,G,bs", [(64, 1, 16), (64, 20, 64), (128, 8, 64), (128, 12, 16), (256, 4, 32), (256, 32, 16)])
def test_lists_with_large_value_scales_in_every_tile_shape(fmt, hd, G, bs):
    rng = np.random.default_rng(hd + G)
    n_kv, n_sel = 2, 320 // bs
    for S, kind in ((300, "all"), (65504, "some"), (4096, "one")):
        p, h = fill_pool(rng, fmt, n_sel + 3, n_kv, bs, hd)
        set_scales(rng, p, h, kind, S)
        for n_seq in (1, 40):
            blocks, lens = random_lists(rng, n_seq, 1, n_kv, n_sel, n_sel + 3, bs)
            check_lists(fmt, p, h, queries(rng, n_seq, 1, n_kv * G, hd), blocks, lens)


@pytest.mark.parametrize("fmt", ["q8", "k8v4"])
def test_a_list_of_one_cell_gives_its_value(fmt):
    rng = np.random.default_rng(9)
    bs, hd, n_kv, G = 16, 256, 1, 4
    for S in (255.5, 256, 65504, -65504):
        p, h = fill_pool(rng, fmt, 3, n_kv, bs, hd)
        h["vs"][:] = np.float16(S)
        p.vs.copy_(dev(h["vs"]))
        check_lists(fmt, p, h, queries(rng, 2, 1, G, hd), np.array([[[[2]]], [[[0]]]], np.int32),
                    np.ones((2, 1, 1), np.int64))


def ramp(rng, p, h, order, q_mean, rise):
    """Keys whose logits rise by `rise` (log2 units) along the cells in `order`
    (block, offset pairs) for queries of mean q_mean, with a little noise."""
    hd = p.head_dim
    n = len(order)
    unit = q_mean * hd / math.sqrt(hd) * math.log2(math.e)    # logit of a key of ones
    at = np.linspace(0, rise, n) / unit
    s = np.float16(rise / unit / 100)
    h["ks"][:] = s
    for i, (blk, c) in enumerate(order):
        h["k"][blk, :, c] = np.clip(np.rint(at[i] / float(s) + rng.normal(0, 1, (p.n_kv, hd))), -127, 127)
    for name in ("k", "ks"):
        getattr(p, name).copy_(dev(h[name]))


@pytest.mark.parametrize("fmt", ["q8", "k8v4"])
@pytest.mark.parametrize("rise", [7.5, 100.0])
def test_lists_whose_logits_rise_under_large_value_scales(fmt, rise):
    rng = np.random.default_rng(int(rise))
    bs, n_sel, n_kv, G, hd = 16, 40, 1, 4, 128
    for S, first in ((1000, 0), (65504, 0), (65504, 300), (65504, 620)):   # the first cell with such a scale
        p, h = fill_pool(rng, fmt, n_sel, n_kv, bs, hd)
        row = rng.permutation(n_sel)
        order = [(int(b), c) for b in row for c in range(bs)]
        ramp(rng, p, h, order, 1.0, rise)
        for b, c in order[first:]:
            h["vs"][b, :, c] = np.float16(S)
        p.vs.copy_(dev(h["vs"]))
        for n_seq in (1, 150):
            q = (1 + 0.1 * rng.standard_normal((n_seq, 1, n_kv * G, hd))).astype(np.float32)
            blocks = np.broadcast_to(row, (n_seq, 1, n_kv, n_sel)).astype(np.int32)
            lens = rng.integers(1, n_sel * bs + 1, (n_seq, 1, n_kv))
            lens.flat[0] = n_sel * bs
            check_lists(fmt, p, h, q, blocks, lens)


def check_dense(fmt, p, h, q, table, ctx, some=None):
    """some: so many sequences are compared (the first, the others spread)."""
    sm = float(np.float32(1 / math.sqrt(p.head_dim)))
    n_seq, W, n_q, hd = q.shape
    out = p.decode(dev(q), i32(ctx), int(max(ctx)), i32(table), sm)
    torch.cuda.synchronize()
    at = np.arange(n_seq) if some is None else np.unique(np.linspace(0, n_seq - 1, some).astype(int))
    out, q, table, ctx, n_seq = out.cpu().numpy()[at], q[at], table[at], np.asarray(ctx)[at], len(at)
    assert np.isfinite(out).all()
    K, V = plain.pool_rows(fmt, h["k"], h["v"], h["ks"], h["vs"])
    blocks = np.broadcast_to(table[:, None, None], (n_seq, W, p.n_kv, table.shape[1]))
    lens = np.maximum(0, ctx[:, None] - W + 1 + np.arange(W))[..., None].repeat(p.n_kv, 2)
    want, tol = plain.attention(fmt, K, V, q, blocks, lens, p.block_size, sm)
    # K enters q.k as 1152 + code here: a group of 64 dims is summed in fp32 at
    # up to (1152 + 127) sum |q| (4 steps and the 1152 sum |q| taken off, itself
    # a sum in 6 steps: 12 roundings of 2^-23 at most), times the K scale
    dz = 12 * 2.0 ** -23 * 1279 * np.abs(q).sum(-1) * float(np.abs(h["ks"].astype(np.float64)).max()) * sm
    spread = np.abs(V).max()
    tol = tol + 2 * dz * spread + lowest_rounding(h, fmt, table.shape[1] * p.block_size) / weights_sum(
        K, q, blocks, lens, p.block_size, sm)
    err = np.abs(out - want).max(-1)
    assert (err <= tol).all(), (err / tol).max()


@pytest.mark.parametrize("fmt", ["q8", "k8v4"])
@pytest.mark.parametrize("W,hd,G", [(1, 128, 4), (1, 64, 1), (3, 128, 4), (2, 64, 5), (1, 256, 8), (2, 256, 2)])
@pytest.mark.parametrize("rise", [3.0, 7.5, 60.0])
def test_dense_decode_whose_logits_rise_under_large_value_scales(fmt, W, hd, G, rise):
    # The reference maximum may lie up to 2^8 behind the row's own: weights up
    # to 256, times the scale.  Sequences enough that each is one split of all
    # its tiles (all of them read the same blocks).
    rng = np.random.default_rng(hd + W)
    bs, L, n_seq, n_kv = 32, 640, 320, 8
    nb = L // bs
    for S, first in ((260, 0), (1000, 0), (65504, 0), (65504, 300)):     # the first cell with such a scale
        p, h = fill_pool(rng, fmt, nb, n_kv, bs, hd)
        row = rng.permutation(nb)
        order = [(int(b), c) for b in row for c in range(bs)]
        ramp(rng, p, h, order, 1.0, rise)
        for b, c in order[first:]:
            h["vs"][b, :, c] = np.float16(S)
        p.vs.copy_(dev(h["vs"]))
        q = (1 + 0.1 * rng.standard_normal((n_seq, W, n_kv * G, hd))).astype(np.float32)
        ctx = rng.integers(L // 2, L + 1, n_seq)
        ctx[0] = L
        check_dense(fmt, p, h, q, np.broadcast_to(row, (n_seq, nb)).astype(np.int32), ctx, some=12)


@pytest.mark.parametrize("fmt", ["q8", "k8v4"])
@pytest.mark.parametrize("W,G", [(1, 4), (4, 8)])
def test_dense_decode_with_large_value_scales(fmt, W, G):
    rng = np.random.default_rng(W)
    bs, L, hd = 16, 1500, 128
    table, n_blocks = tables(rng, [L, 7, 333], bs)
    for S, kind in ((300, "all"), (65504, "some"), (4096, "one")):
        p, h = fill_pool(rng, fmt, n_blocks, 2, bs, hd)
        set_scales(rng, p, h, kind, S)
        check_dense(fmt, p, h, queries(rng, 3, W, 2 * G, hd), table, [L, 7, 333])
