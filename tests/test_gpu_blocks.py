"""GPU: kvq_bound_blocks and kvq_select_blocks bit for bit, and
kvq_sparse_decode_attn within a derived tolerance, against the plain 64-bit
forms of tests/plain_blocks.py; and the whole step together."""
import math

import numpy as np
import pytest
import torch

import quantized_kv_cache_append_gb300 as kvq
from quantized_kv_cache_append_gb300.pool import BlockBounds, PagedPool
from quantized_kv_cache_append_gb300.steps import StepPlanner
from tests import plain_blocks as plain

pytestmark = pytest.mark.gpu

FMT = {"f16": kvq.KVQ_F16, "q8": kvq.KVQ_Q8, "k8v4": kvq.KVQ_K8V4}


@pytest.fixture(scope="module", autouse=True)
def _library():
    if not torch.cuda.is_available():
        pytest.fail("the GPU suite needs a CUDA device")
    kvq.build()
    kvq.load_library()


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def i32(a):
    return dev(np.asarray(a, np.int32))


def tables(rng, lens, bs, spare=3):
    nb = [-(-int(L) // bs) for L in lens]
    perm = rng.permutation(sum(nb) + spare).astype(np.int32)
    t = np.full((len(lens), max(nb + [1])), -1, np.int32)
    at = 0
    for b, n in enumerate(nb):
        t[b, :n] = perm[at:at + n]
        at += n
    return t, sum(nb) + spare


def fill_pool(rng, fmt, n_blocks, n_kv, bs, hd):
    """A pool of random contents, written directly (host arrays returned too)."""
    p = PagedPool(FMT[fmt], n_kv, hd, bs, n_blocks)
    shape = (n_blocks, n_kv, bs)
    gain = np.where(rng.random(hd) < 0.05, 6.0, 1.0)
    h = {"vs": None, "ks": None}
    if fmt == "f16":
        h["k"] = (rng.standard_normal(shape + (hd,)) * gain).astype(np.float16)
        h["v"] = rng.standard_normal(shape + (hd,)).astype(np.float16)
    else:
        h["k"] = rng.integers(-127, 128, shape + (hd,)).astype(np.int8)
        h["ks"] = (rng.random(shape + (hd // 64,)) * 0.03 + 0.003).astype(np.float16)
        if fmt == "q8":
            h["v"] = rng.integers(-127, 128, shape + (hd,)).astype(np.int8)
            h["vs"] = (rng.random(shape + (hd // 64,)) * 0.03 + 0.003).astype(np.float16)
        else:
            h["v"] = rng.integers(0, 256, shape + (hd // 2,)).astype(np.uint8)
            h["vs"] = ((rng.random(shape + (hd // 32,)) - 0.5) * 4).astype(np.float16)
    for name in ("k", "v", "ks", "vs"):
        if h[name] is not None:
            getattr(p, name).copy_(dev(h[name]))
    return p, h


# ---------------------------------------------------------------- bounds
def plain_bounds(fmt, h, bounds, scales, table, start, lens, bs):
    with np.errstate(invalid="ignore", over="ignore"):
        K = h["k"].astype(np.float64)
        if fmt != "f16":
            K = K * np.repeat(h["ks"].astype(np.float64), 64, -1)
    codes, sc = bounds.copy(), scales.copy()
    for b in range(len(lens)):
        L = min(int(lens[b]), table.shape[1] * bs)
        if int(start[b]) >= L:
            continue
        for j in range(max(int(start[b]), 0) // bs, -(-L // bs)):
            blk = table[b, j]
            if 0 <= blk < len(codes):
                for n in range(K.shape[1]):
                    codes[blk, n], sc[blk, n] = plain.bounds_of(K[blk, n, :min(bs, L - j * bs)])
    return codes, sc


def check_bounds(rng, fmt, p, h, table, start, lens, use_start=True, max_new=None):
    n_blocks, n_kv, bs, hd = p.n_blocks, p.n_kv, p.block_size, p.head_dim
    bb = BlockBounds(p)
    old = rng.integers(-128, 128, bb.codes.shape).astype(np.int8)
    old_s = rng.random(bb.scales.shape).astype(np.float32)
    bb.codes.copy_(dev(old))
    bb.scales.copy_(dev(old_s))
    start, lens = np.asarray(start), np.asarray(lens)
    if max_new is None:
        max_new = int(max((lens - (start if use_start else 0)).max(), 0))
    p.bound(bb, i32(table), i32(lens), max_new, i32(start) if use_start else None)
    torch.cuda.synchronize()
    want = plain_bounds(fmt, h, old, old_s, table, start if use_start else np.zeros_like(lens), lens, bs)
    assert np.array_equal(bb.codes.cpu().numpy(), want[0])
    assert np.array_equal(bb.scales.cpu().numpy(), want[1])
    return want


@pytest.mark.parametrize("fmt", ["f16", "q8", "k8v4"])
@pytest.mark.parametrize("n_kv,hd,bs", [(2, 64, 16), (1, 64, 1024), (3, 128, 16), (2, 128, 64), (1, 128, 256),
                                        (1, 256, 16), (2, 256, 32), (1, 256, 128)])
def test_bounds_of_ragged_sequences(fmt, n_kv, hd, bs):
    rng = np.random.default_rng(hd + bs)
    lens = np.array([1, bs - 1, bs, bs + 1, 0, 3 * bs + 5])
    table, n_blocks = tables(rng, lens, bs)
    p, h = fill_pool(rng, fmt, n_blocks, n_kv, bs, hd)
    check_bounds(rng, fmt, p, h, table, np.zeros(6, int), lens, use_start=False)
    # the newest cells alone: mid-block, on a border, none, several blocks
    check_bounds(rng, fmt, p, h, table, [0, bs - 2, bs - 1, bs, 0, bs - 1], lens)
    check_bounds(rng, fmt, p, h, table, [1, bs - 1, bs, bs + 1, 0, 3 * bs + 5], lens, max_new=4)   # nothing new


@pytest.mark.parametrize("fmt", ["f16", "q8"])
def test_bounds_of_special_values(fmt):
    rng = np.random.default_rng(2)
    n_kv, hd, bs = 1, 128, 16
    table, n_blocks = tables(rng, [16 * 7], bs, spare=0)
    p, h = fill_pool(rng, fmt, n_blocks, n_kv, bs, hd)
    blk = table[0]
    if fmt == "f16":
        k = h["k"]
        k[blk[0]] = 0
        k[blk[1], 0, 3, :40] = np.nan                 # passed over
        k[blk[2], 0, :, 5] = np.nan                   # nothing left: 0
        k[blk[3], 0, 2, 7], k[blk[3], 0, 4, 70] = np.inf, -np.inf
        k[blk[4]] = np.float16(2.0 ** -24)            # the smallest subnormal
        k[blk[5]] = np.float16(-65504)
        k[blk[6], 0, :, :64] = np.float16(127 / 128)  # on the border of two scales
        k[blk[6], 0, :, 64:] = np.nextafter(np.float16(127 / 128), np.float16(2))
        k[blk[6], 0, 0, 3] = -0.0
    else:
        s = h["ks"]
        s[blk[0]] = 0
        s[blk[1]] = 65504                             # dequantised up to 8.3 million
        s[blk[2]] = np.float16(2.0 ** -24)
        h["k"][blk[3]] = 0
        s[blk[4]] = np.float16(2.0 ** -7)             # 127 * 2^-7: on the border
        h["k"][blk[4], 0, 0, :] = 127
        h["k"][blk[5]] = -127
    for name in ("k", "ks"):
        if h[name] is not None:
            getattr(p, name).copy_(dev(h[name]))
    check_bounds(rng, fmt, p, h, table, [0], [16 * 7], use_start=False)


def test_bounds_skip_foreign_ids_and_clamp_lengths():
    rng = np.random.default_rng(4)
    bs = 16
    table, n_blocks = tables(rng, [64, 64], bs)
    p, h = fill_pool(rng, "f16", n_blocks, 2, bs, 64)
    table[0, 1], table[0, 3], table[1, 2] = -1, n_blocks, 1 << 30
    check_bounds(rng, "f16", p, h, table, [0, 0], [64, 64])
    check_bounds(rng, "f16", p, h, table, [-5, 60], [1000, 64], max_new=64)       # past the row: clamped


def test_bounds_cover_what_max_new_covers_and_no_more():
    rng = np.random.default_rng(5)
    bs = 16
    table, n_blocks = tables(rng, [160], bs)
    p, h = fill_pool(rng, "q8", n_blocks, 2, bs, 64)
    bb = BlockBounds(p)
    bb.codes.fill_(55)
    p.bound(bb, i32(table), i32([160]), 30, i32([20]))       # cells 20 .. 49: blocks 1, 2, 3
    torch.cuda.synchronize()
    old = np.full(bb.codes.shape, 55, np.int8)
    want = plain_bounds("q8", h, old, np.zeros(bb.scales.shape, np.float32), table, [20], [64], bs)
    assert np.array_equal(bb.codes.cpu().numpy(), want[0])


def test_bounds_of_many_items():
    # more (block, head) items than one wave of warps or CTAs takes, per
    # layout of the work: persistent CTAs come round again
    rng = np.random.default_rng(6)
    for fmt, hd, bs, n in (("f16", 64, 16, 3000), ("q8", 64, 16, 3000), ("f16", 256, 32, 400), ("q8", 256, 64, 300)):
        lens = np.array([n * bs - 7])
        table, n_blocks = tables(rng, lens, bs)
        p, h = fill_pool(rng, fmt, n_blocks, 3, bs, hd)
        check_bounds(rng, fmt, p, h, table, [0], lens, use_start=False)


# ---------------------------------------------------------------- selection
def random_bounds(rng, n_blocks, n_kv, hd):
    hi = np.clip(np.rint(rng.normal(60, 30, (n_blocks, n_kv, 2, hd))), -127, 127).astype(np.int8)
    hi[:, :, 0] = np.minimum(hi[:, :, 1], np.clip(np.rint(rng.normal(-60, 30, hi[:, :, 0].shape)), -127, 127))
    scales = (2.0 ** rng.integers(-9, -3, (n_blocks, n_kv, hd // 64))).astype(np.float32)
    return hi, scales


def check_select(codes, scales, q, ctx, table, bs, n_blocks, n_sel, n_first, n_last, max_ctx=None, index=True):
    n_seq, W, n_q, hd = q.shape
    n_kv = codes.shape[1]
    p = PagedPool(kvq.KVQ_F16, n_kv, hd, bs, n_blocks)
    mk = lambda *s: torch.full(s, 77777, dtype=torch.int32, device="cuda")
    blocks, idx, lens = mk(n_seq, W, n_kv, n_sel), mk(n_seq, W, n_kv, n_sel), mk(n_seq, W, n_kv)
    st = kvq.kvq_select_blocks(p.cache, dev(codes), dev(scales), dev(q), n_seq, W, n_q, i32(ctx),
                               int(max(ctx)) if max_ctx is None else max_ctx, i32(table), table.shape[1],
                               n_sel, n_first, n_last, blocks, idx if index else None, lens)
    assert st == kvq.KVQ_OK, kvq.kvq_status_string(st)
    torch.cuda.synchronize()
    want = plain.select(codes, scales, q, ctx, table, bs, n_blocks, n_sel, n_first, n_last)
    assert np.array_equal(lens.cpu().numpy(), want[2])
    assert np.array_equal(blocks.cpu().numpy(), want[0])
    if index:
        assert np.array_equal(idx.cpu().numpy(), want[1])
    return want


def queries(rng, *shape):
    return rng.standard_normal(shape).astype(np.float32)


@pytest.mark.parametrize("n_seq,W,n_kv,G,hd,bs,hi,n_sel,first,last", [
    (1, 1, 1, 1, 64, 16, 16, 1, 0, 0), (1, 1, 8, 4, 128, 64, 32768, 64, 1, 2),
    (3, 1, 2, 2, 64, 16, 5000, 31, 1, 1), (2, 3, 3, 3, 128, 32, 4001, 17, 0, 3),
    (1, 4, 2, 8, 256, 16, 20011, 100, 2, 4), (2, 1, 1, 32, 256, 16, 3001, 9, 0, 0),
    (2, 17, 1, 5, 64, 16, 1500, 11, 1, 1), (1, 2, 1, 16, 128, 1024, 70000, 8, 1, 1),
    (40, 1, 8, 4, 128, 16, 900, 12, 1, 2), (2, 9, 2, 7, 128, 16, 1200, 30, 1, 2),
    (1, 1, 2, 1, 256, 16, 131072, 700, 0, 1), (2, 3, 1, 12, 128, 16, 1777, 20, 1, 1),
    (1, 2, 2, 20, 256, 32, 3333, 15, 0, 1), (1, 130, 1, 6, 64, 16, 1999, 13, 1, 2),
    (3, 5, 1, 9, 64, 16, 700, 6, 0, 0), (1, 3, 2, 8, 128, 16, 70001, 250, 1, 1),
])
def test_selection(n_seq, W, n_kv, G, hd, bs, hi, n_sel, first, last):
    rng = np.random.default_rng(hi + W)
    lens = rng.integers(max(1, hi // 3), hi + 1, n_seq)
    lens[0] = hi
    table, n_blocks = tables(rng, lens, bs)
    codes, scales = random_bounds(rng, n_blocks, n_kv, hd)
    check_select(codes, scales, queries(rng, n_seq, W, n_kv * G, hd), lens, table, bs, n_blocks, n_sel, first, last)


def test_selection_over_the_longest_row():
    rng = np.random.default_rng(8)
    bs, n = 16, 32768
    table, n_blocks = tables(rng, [n * bs], bs)
    codes, scales = random_bounds(rng, n_blocks, 1, 64)
    q = queries(rng, 1, 2, 3, 64)
    check_select(codes, scales, q, [n * bs], table, bs, n_blocks, 2000, 1, 4)
    check_select(codes, scales, q, [n * bs], table, bs, n_blocks, n + 5, 1, 4)      # every block


def test_selection_over_the_longest_row_of_many_wide_query_heads():
    rng = np.random.default_rng(18)
    bs, n = 16, 32768
    table, n_blocks = tables(rng, [n * bs - 5], bs)
    codes, scales = random_bounds(rng, n_blocks, 1, 256)
    check_select(codes, scales, queries(rng, 1, 3, 32, 256), [n * bs - 5], table, bs, n_blocks, 77, 0, 2)


def test_selection_orders_a_ragged_batch_without_mixing_it_up():
    # clusters start with the longer sequences when a batch takes several
    # waves: 70 and 129 sequences, empty and full ones among them
    rng = np.random.default_rng(19)
    bs = 16
    for n_seq, n_kv in ((70, 8), (129, 4)):
        lens = rng.integers(0, 1500, n_seq)
        lens[[0, 5, n_seq - 1]] = 0, 1500, 1
        lens[10:14] = [750, 749, 375, 374]      # on the classes' borders
        table, n_blocks = tables(rng, lens, bs)
        codes, scales = random_bounds(rng, n_blocks, n_kv, 64)
        check_select(codes, scales, queries(rng, n_seq, 1, n_kv, 64), lens, table, bs, n_blocks, 9, 1, 1)


def test_whole_number_sums_at_their_largest():
    # every product 127 * 127, all of one sign, and sums that differ by one
    bs, n, hd = 16, 64, 256
    codes = np.full((n, 1, 2, hd), 127, np.int8)
    codes[:, :, 0] = -127
    scales = np.full((n, 1, hd // 64), 2.0 ** -3, np.float32)
    for j in range(n):          # block j is short of the largest sum by j % 5 products' units
        codes[j, 0, 1, :j % 5] = 126
    q = np.full((1, 2, 2, hd), 127.0, np.float32)
    q[0, 1, :, ::2] = -127.0
    table = np.arange(n, dtype=np.int32)[None]
    for n_sel in (1, 12, 13, 26, 40):
        check_select(codes, scales, q, [n * bs], table, bs, n, n_sel, 0, 0)


def test_equal_scores_go_to_the_lower_block():
    rng = np.random.default_rng(5)
    bs, n = 16, 1000
    table, n_blocks = tables(rng, [n * bs - 3], bs)
    codes, scales = random_bounds(rng, n_blocks, 2, 128)
    q = queries(rng, 1, 1, 4, 128)
    codes[:], scales[:] = codes[:1], scales[:1]
    for n_sel, first, last in ((1, 0, 0), (7, 0, 0), (64, 1, 2), (999, 0, 1), (1000, 0, 0)):
        check_select(codes, scales, q, [n * bs - 3], table, bs, n_blocks, n_sel, first, last)
    pick = rng.integers(0, 5, n_blocks)          # five values, the threshold inside a long tie
    base, bsc = random_bounds(rng, 5, 2, 128)
    codes, scales = base[pick], bsc[pick]
    for n_sel in (2, 100, 333, 500, 801):
        check_select(codes, scales, q, [n * bs - 3], table, bs, n_blocks, n_sel, 1, 1)
    check_select(codes, scales, np.zeros_like(q), [n * bs - 3], table, bs, n_blocks, 100, 0, 0)   # all scores 0


def test_selection_of_short_contexts_and_windows():
    rng = np.random.default_rng(6)
    bs, n_kv, W = 16, 2, 5
    lens = np.array([0, 1, 3, 4, 5, 6, 16, 17, 20, 21, 100])       # some tokens see nothing
    table, n_blocks = tables(rng, lens, bs)
    codes, scales = random_bounds(rng, n_blocks, n_kv, 64)
    q = queries(rng, len(lens), W, n_kv * 2, 64)
    for n_sel, first, last in ((1, 0, 0), (2, 1, 1), (4, 0, 3), (9, 2, 2)):
        want = check_select(codes, scales, q, lens, table, bs, n_blocks, n_sel, first, last)
        assert (want[2][0] == 0).all() and (want[0][0] == -1).all()
    check_select(codes, scales, q, lens, table, bs, n_blocks, 3, 1, 1, index=False)
    check_select(codes, scales, q, lens, table, bs, n_blocks, 3, 1, 1, max_ctx=table.shape[1] * bs)


def test_selection_never_takes_a_foreign_block():
    rng = np.random.default_rng(7)
    bs, n = 16, 300
    table, n_blocks = tables(rng, [n * bs - 1, n * bs], bs)
    holes = rng.random(table.shape) < 0.4
    table[holes] = rng.choice([-1, n_blocks, 1 << 30, -(1 << 31)], holes.sum())
    table[0, 0] = table[0, n - 1] = -1           # the forced ones too
    table[1, 5:] = -1                            # hardly any left
    codes, scales = random_bounds(rng, n_blocks, 1, 128)
    q = queries(rng, 2, 1, 4, 128)
    for n_sel in (4, 60, 250):
        check_select(codes, scales, q, [n * bs - 1, n * bs], table, bs, n_blocks, n_sel, 2, 2)


def test_lists_that_hold_every_block():
    # nothing to score: rows at, below and one past the list's length, longer
    # than the CTA's threads, with holes, and beside rows that are scored
    rng = np.random.default_rng(14)
    bs, n_kv, W = 16, 2, 3
    for n_sel in (1, 4, 300, 700):
        lens = np.array([n_sel * bs, n_sel * bs + 1, n_sel * bs + 2, n_sel * bs + 3, bs, 1, 0, 5 * n_sel * bs])
        table, n_blocks = tables(rng, lens, bs)
        table[4, 0] = -1
        table[0, n_sel - 1] = n_blocks            # the last visible block is foreign
        table[1, ::3] = -1
        codes, scales = random_bounds(rng, n_blocks, n_kv, 64)
        check_select(codes, scales, queries(rng, len(lens), W, n_kv, 64), lens, table, bs, n_blocks, n_sel, 0, 1)
        check_select(codes, scales, queries(rng, len(lens), 1, n_kv * 4, 64), lens, table, bs, n_blocks, n_sel, 1, 0,
                     index=False)


def test_selection_with_special_queries():
    rng = np.random.default_rng(10)
    bs, n = 16, 200
    table, n_blocks = tables(rng, [n * bs], bs)
    codes, scales = random_bounds(rng, n_blocks, 1, 128)
    q = queries(rng, 1, 6, 2, 128)
    q[0, 0, 0, 5] = np.nan
    q[0, 1, 1, :] = np.nan
    q[0, 2, 0, 9], q[0, 2, 0, 90] = np.inf, -np.inf      # saturated codes at 2^60
    q[0, 3] *= 1e-30                                     # codes 0: all scores 0
    q[0, 4, 0, :64] = 127 / 128                          # on the border of two scales
    q[0, 4, 0, 64:] = np.nextafter(np.float32(127 / 128), np.float32(2))
    q[0, 5] *= 1e30                                      # past 127 * 2^60: saturated
    check_select(codes, scales, q, [n * bs], table, bs, n_blocks, 20, 0, 0)


# ---------------------------------------------------------------- attention
def check_attention(rng, fmt, p, h, q, blocks, lens, scale=None):
    sm = 1 / math.sqrt(p.head_dim) if scale is None else scale
    out = torch.full(q.shape, float("nan"), device="cuda")
    p.decode_selected(dev(q), i32(blocks), i32(lens), sm, out=out)
    torch.cuda.synchronize()
    K, V = plain.pool_rows(fmt, h["k"], h["v"], h["ks"], h["vs"])
    want, tol = plain.attention(fmt, K, V, q, blocks, lens, p.block_size, np.float64(np.float32(sm)))
    err = np.abs(out.cpu().numpy() - want).max(-1)
    assert np.isfinite(err).all()
    assert (err <= tol).all(), (err - tol).max()
    assert (out.cpu().numpy()[lens_rows(lens, q) <= 0] == 0).all()
    return out


def lens_rows(lens, q):
    """sel_lens per query row: [n_seq][W][n_q]."""
    return np.repeat(lens, q.shape[2] // lens.shape[2], 2)


def random_lists(rng, n_seq, W, n_kv, n_sel, n_blocks, bs):
    blocks = np.stack([rng.permutation(max(n_blocks, n_sel))[:n_sel] % n_blocks
                       for _ in range(n_seq * W * n_kv)]).reshape(n_seq, W, n_kv, n_sel)
    lens = rng.integers(0, n_sel * bs + 1, (n_seq, W, n_kv))
    lens.flat[0] = n_sel * bs
    return blocks, lens


@pytest.mark.parametrize("fmt", ["f16", "q8", "k8v4"])
@pytest.mark.parametrize("n_seq,W,n_kv,G,hd,bs,n_sel", [
    (1, 1, 1, 1, 64, 16, 1), (1, 1, 1, 4, 128, 64, 70), (1, 1, 8, 4, 128, 64, 9), (3, 1, 2, 3, 64, 16, 13),
    (2, 5, 3, 5, 128, 32, 7), (1, 17, 2, 2, 256, 16, 21), (2, 1, 2, 16, 128, 128, 4), (1, 2, 1, 32, 64, 256, 3),
    (1, 1, 2, 32, 256, 16, 40), (9, 2, 4, 8, 256, 16, 5), (1, 3, 1, 7, 128, 1024, 2),
    (2, 1, 1, 12, 256, 32, 6), (1, 2, 2, 20, 128, 16, 9), (1, 2, 1, 20, 256, 16, 12), (1, 150, 2, 4, 128, 16, 3),
    (1, 40, 1, 3, 64, 32, 5),
])
def test_attention_over_lists(fmt, n_seq, W, n_kv, G, hd, bs, n_sel):
    rng = np.random.default_rng(hd + bs + W)
    n_blocks = n_sel + 5
    p, h = fill_pool(rng, fmt, n_blocks, n_kv, bs, hd)
    blocks, lens = random_lists(rng, n_seq, W, n_kv, n_sel, n_blocks, bs)
    check_attention(rng, fmt, p, h, queries(rng, n_seq, W, n_kv * G, hd), blocks, lens)


@pytest.mark.parametrize("fmt", ["f16", "q8", "k8v4"])
def test_attention_lengths_holes_and_repeats(fmt):
    rng = np.random.default_rng(3)
    bs, n_sel, n_kv, hd = 16, 6, 2, 128
    p, h = fill_pool(rng, fmt, 8, n_kv, bs, hd)
    q = queries(rng, 4, 3, n_kv * 4, hd)
    blocks, lens = random_lists(rng, 4, 3, n_kv, n_sel, 8, bs)
    lens[0] = 0                                      # rows without a cell
    lens[1] = -4
    lens[2] = [[1, 2], [15, 16], [17, 1000]]         # one cell; past the list: clamped
    blocks[3, 0, :, 2] = [-1, 8]                     # a hole inside
    blocks[3, 1] = -1                                # nothing but holes
    blocks[3, 2, :, 1:] = 3                          # the same block again and again
    lens[3] = n_sel * bs
    out = check_attention(rng, fmt, p, h, q, blocks, lens)
    assert (out[3, 1] == 0).all()


def test_attention_ignores_what_lies_behind_a_list():
    # cells past sel_len inside the last block hold NaN and infinities
    rng = np.random.default_rng(12)
    bs, hd = 16, 64
    for fmt in ("f16", "q8", "k8v4"):
        p, h = fill_pool(rng, fmt, 4, 1, bs, hd)
        blocks = np.array([0, 2, 3], np.int32).reshape(1, 1, 1, 3)
        lens = np.full((1, 1, 1), 37)
        q = queries(rng, 1, 1, 4, hd)
        want = check_attention(rng, fmt, p, h, q, blocks, lens)
        bad = float("nan")
        if fmt == "f16":
            p.k[3, 0, 5:], p.v[3, 0, 5:] = float("inf"), bad
            p.k[1], p.v[1] = bad, bad
        else:
            p.ks[3, 0, 5:], p.vs[3, 0, 5:] = bad, float("-inf")
            p.ks[1], p.vs[1] = bad, bad
        out = p.decode_selected(dev(q), i32(blocks), i32(lens), 1 / math.sqrt(hd))
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_attention_over_every_block_is_the_dense_decode():
    rng = np.random.default_rng(13)
    bs, n_kv, G, hd, L, W = 32, 2, 4, 128, 3001, 2
    table, n_blocks = tables(rng, [L], bs)
    for fmt in ("f16", "q8", "k8v4"):
        p, h = fill_pool(rng, fmt, n_blocks, n_kv, bs, hd)
        q = dev(queries(rng, 1, W, n_kv * G, hd))
        bb = BlockBounds(p)
        p.bound(bb, i32(table), i32([L]), L)
        blocks, index, lens = p.select(bb, q, i32([L]), L, i32(table), table.shape[1])
        assert lens[0, :, 0].tolist() == [L - 1, L]
        assert torch.equal(blocks[0, 1, 1], i32(table)[0])
        a = p.decode_selected(q, blocks, lens, 0.088)
        b = p.decode(q, i32([L]), L, i32(table), 0.088)
        torch.cuda.synchronize()
        rel = ((a - b).norm() / b.norm()).item()
        assert rel < 4e-5      # two sums within the bounds of the attention tests


def clustered(p, n_seq, W, n_q, n_sel):
    """Whether a call's splits meet in clusters (it needs no partials then)."""
    return kvq.kvq_sparse_workspace_bytes(p.cache, n_seq, W, n_q, n_sel) == 256


@pytest.mark.parametrize("fmt", ["f16", "q8", "k8v4"])
@pytest.mark.parametrize("hd,G,bs", [(64, 4, 16), (128, 4, 16), (128, 8, 64), (256, 4, 16), (256, 32, 16)])
def test_attention_with_splits_through_clusters_and_through_the_workspace(fmt, hd, G, bs):
    # few lists and many: splits through the workspace, in clusters of
    # several sizes, and one split each; lists of every length, most splits of
    # the short ones empty
    rng = np.random.default_rng(hd + G)
    n_sel, n_kv, n_blocks = 512 // bs, 2, 40
    p, h = fill_pool(rng, fmt, n_blocks, n_kv, bs, hd)
    seen = set()
    for n_seq in (1, 20, 37, 75, 151, 310):
        n_q = n_kv * G
        seen.add(clustered(p, n_seq, 1, n_q, n_sel))
        if G == 32 and n_seq > 75:
            continue
        q = queries(rng, n_seq, 1, n_q, hd)
        blocks, lens = random_lists(rng, n_seq, 1, n_kv, n_sel, n_blocks, bs)
        check_attention(rng, fmt, p, h, q, blocks, lens)
    assert seen == {False, True}


@pytest.mark.parametrize("fmt", ["f16", "q8", "k8v4"])
def test_lost_copy_waits_give_nan_rows(fmt):
    # one wave's worth of lists in clusters, and a single one through the
    # workspace; an ordinary call on the same buffers is right afterwards
    rng = np.random.default_rng(30)
    bs, hd, n_kv, G, n_sel = 16, 128, 2, 4, 16
    p, h = fill_pool(rng, fmt, 20, n_kv, bs, hd)
    for n_seq in (1, 75, 310):
        q = queries(rng, n_seq, 1, n_kv * G, hd)
        blocks, lens = random_lists(rng, n_seq, 1, n_kv, n_sel, 20, bs)
        lens = np.maximum(lens, 1)
        out = torch.zeros(q.shape, device="cuda")
        ws = torch.empty(kvq.kvq_sparse_workspace_bytes(p.cache, n_seq, 1, n_kv * G, n_sel), dtype=torch.uint8,
                         device="cuda")
        st = kvq.kvq_sparse_decode_attn_lost_wait_test(p.cache, dev(q), n_seq, 1, n_kv * G, i32(blocks), i32(lens),
                                                       n_sel, 0.1, out, ws, ws.numel(), 4096, 16)
        assert st == kvq.KVQ_OK, kvq.kvq_status_string(st)
        torch.cuda.synchronize()
        assert torch.isnan(out).all()
        check_attention(rng, fmt, p, h, q, blocks, lens)


def test_methods_refuse_tensors_they_cannot_read():
    p = PagedPool(kvq.KVQ_F16, 2, 64, 16, 8)
    bb = BlockBounds(p)
    q = torch.zeros(1, 1, 4, 64, device="cuda")
    table, lens = i32([[0, 1, 2]]), i32([40])
    blocks, index, cells = p.select(bb, q, lens, 40, table, 2)
    bad_q = torch.zeros(1, 1, 64, 4, device="cuda").transpose(2, 3)
    for call in (lambda: p.select(bb, bad_q, lens, 40, table, 2), lambda: p.select(bb, q.half(), lens, 40, table, 2),
                 lambda: p.select(bb, q, lens.long(), 40, table, 2), lambda: p.select(bb, q, lens.cpu(), 40, table, 2),
                 lambda: p.select(bb, q, lens, 40, table.repeat(2, 1), 2),
                 lambda: p.bound(bb, table[:, ::2], lens, 40), lambda: p.bound(bb, table, lens, 40, i32([0, 0])),
                 lambda: p.decode_selected(bad_q, blocks, cells, 0.1),
                 lambda: p.decode_selected(q, blocks.long(), cells, 0.1),
                 lambda: p.decode_selected(q, blocks, cells[..., :1], 0.1),
                 lambda: p.decode_selected(q, blocks, cells, 0.1, workspace=torch.zeros(64, device="cuda")),
                 lambda: StepPlanner(2, 4, 16, 8, 16).plan(i32([1]))):
        with pytest.raises(kvq.KvqError):
            call()


# ---------------------------------------------------------------- together
@pytest.mark.parametrize("fmt", ["f16", "q8", "k8v4"])
def test_a_serving_loop(fmt):
    """Requests arrive, decode over chosen blocks and leave: plan, append,
    bound, select and attend each step from device arrays alone, checked
    against the plain forms on the pool's own contents."""
    rng = np.random.default_rng(21)
    n, bs, n_blocks, max_tok, n_kv, G, hd = 5, 16, 120, 160, 2, 4, 128
    width, n_sel = 30, 6
    planner = StepPlanner(n, width, bs, n_blocks, max_tok)
    p = PagedPool(FMT[fmt], n_kv, hd, bs, n_blocks)
    bb = BlockBounds(p)
    for step in range(8):
        new = np.array([[90, 0, 17, 33, 0], [1, 1, 1, 1, 0], [1, 50, 1, 1, 1], [1, 1, -1, 1, 1],
                        [1, 1, 40, 1, -1], [-1, 1, 1, 1, 0], [100, 1, 1, 1, 0], [1, 1, 1, 1, 0]][step])
        planner.plan(i32(new))
        k = rng.standard_normal((max_tok, n_kv, hd)).astype(np.float32)
        v = rng.standard_normal((max_tok, n_kv, hd)).astype(np.float32)
        p.append(dev(k), dev(v), planner.tok_seq, planner.tok_pos, planner.block_table)
        p.bound(bb, planner.block_table, planner.ctx_lens, 100, planner.ctx_start)
        q = queries(rng, n, 1, n_kv * G, hd)
        blocks, index, lens = p.select(bb, dev(q), planner.ctx_lens, width * bs, planner.block_table, n_sel, 1, 2)
        out = p.decode_selected(dev(q), blocks, lens, 1 / math.sqrt(hd))
        torch.cuda.synchronize()
        assert planner.info[3] == 0
        ctx, table = planner.ctx_lens.cpu().numpy(), planner.block_table.cpu().numpy()
        h = {m: None if getattr(p, m) is None else getattr(p, m).cpu().numpy() for m in ("k", "v", "ks", "vs")}
        codes, scales = plain_bounds(fmt, h, bb.codes.cpu().numpy(), bb.scales.cpu().numpy(), table,
                                     np.zeros(n, int), ctx, bs)
        assert np.array_equal(codes, bb.codes.cpu().numpy()) and np.array_equal(scales, bb.scales.cpu().numpy())
        want = plain.select(codes, scales, q, ctx, table, bs, n_blocks, n_sel, 1, 2)
        for a, b in zip((blocks, index, lens), want):
            assert np.array_equal(a.cpu().numpy(), b)
        K, V = plain.pool_rows(fmt, h["k"], h["v"], h["ks"], h["vs"])
        ref, tol = plain.attention(fmt, K, V, q, want[0], want[2], bs, np.float64(np.float32(1 / math.sqrt(hd))))
        assert (np.abs(out.cpu().numpy() - ref).max(-1) <= tol).all()


def test_a_step_on_a_side_stream_and_replayed_from_a_graph():
    rng = np.random.default_rng(22)
    n, bs, n_blocks, n_kv, G, hd, width, n_sel = 3, 16, 64, 2, 4, 64, 16, 4
    sm = 1 / math.sqrt(hd)
    s = torch.cuda.Stream()
    planner = StepPlanner(n, width, bs, n_blocks, 64)
    p = PagedPool(kvq.KVQ_Q8, n_kv, hd, bs, n_blocks)
    bb = BlockBounds(p)
    k, v = (torch.empty(64, n_kv, hd, device="cuda") for _ in range(2))
    q = torch.empty(n, 1, n_kv * G, hd, device="cuda")
    n_new = torch.empty(n, dtype=torch.int32, device="cuda")
    sel = tuple(torch.empty(x, dtype=torch.int32, device="cuda")
                for x in ((n, 1, n_kv, n_sel), (n, 1, n_kv, n_sel), (n, 1, n_kv)))
    out = torch.empty_like(q)
    ws = torch.empty(kvq.kvq_sparse_workspace_bytes(p.cache, n, 1, n_kv * G, n_sel), dtype=torch.uint8,
                     device="cuda")

    def step(stream=None):
        planner.plan(n_new, stream)
        p.append(k, v, planner.tok_seq, planner.tok_pos, planner.block_table, stream)
        p.bound(bb, planner.block_table, planner.ctx_lens, 20, planner.ctx_start, stream)
        p.select(bb, q, planner.ctx_lens, width * bs, planner.block_table, n_sel, out=sel, stream=stream)
        p.decode_selected(q, sel[0], sel[2], sm, out=out, workspace=ws, stream=stream)

    def feed(new):
        n_new.copy_(i32(new))
        for t in (k, v, q):
            t.copy_(dev(rng.standard_normal(tuple(t.shape)).astype(np.float32)))

    def verify():
        torch.cuda.synchronize()
        h = {m: getattr(p, m).cpu().numpy() for m in ("k", "v", "ks", "vs")}
        table, ctx = planner.block_table.cpu().numpy(), planner.ctx_lens.cpu().numpy()
        want = plain.select(bb.codes.cpu().numpy(), bb.scales.cpu().numpy(), q.cpu().numpy(), ctx, table, bs,
                            n_blocks, n_sel, 1, 1)
        for a, b in zip(sel, want):
            assert np.array_equal(a.cpu().numpy(), b)
        K, V = plain.pool_rows("q8", h["k"], h["v"], h["ks"], h["vs"])
        ref, tol = plain.attention("q8", K, V, q.cpu().numpy(), want[0], want[2], bs, np.float64(np.float32(sm)))
        assert (np.abs(out.cpu().numpy() - ref).max(-1) <= tol).all()

    feed([20, 7, 0])
    torch.cuda.synchronize()
    step(s)
    s.synchronize()
    verify()
    feed([1, 1, 18])
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        step()
    for new in ([1, 1, 18], [1, 20, 1], [-1, 1, 1], [15, 1, 1]):
        feed(new)
        g.replay()
        verify()
    assert planner.ctx_lens.tolist() == [15, 30, 21]


def test_offsets_past_32_bits():
    # a pool whose keys lie beyond 4 GB: sequences at its far end
    rng = np.random.default_rng(40)
    bs, n_kv, hd, G, n_blocks = 1024, 8, 256, 2, 2600       # 5.5 GB of K codes, 5.5 of V
    p = PagedPool(kvq.KVQ_Q8, n_kv, hd, bs, n_blocks)
    assert p.k.numel() > 1 << 32
    lens = np.array([1500, 700])
    table = np.array([[n_blocks - 1, n_blocks - 3], [n_blocks - 2, -1]], np.int32)
    k = rng.standard_normal((2200, n_kv, hd)).astype(np.float32)
    seq = np.repeat([0, 1], lens)
    pos = np.concatenate([np.arange(n) for n in lens])
    p.append(dev(k), dev(k[::-1].copy()), i32(seq), i32(pos), i32(table))
    bb = BlockBounds(p)
    p.bound(bb, i32(table), i32(lens), 1500)
    q = queries(rng, 2, 1, n_kv * G, hd)
    blocks, index, cells = p.select(bb, dev(q), i32(lens), 1500, i32(table), 1, 0, 1)
    out = p.decode_selected(dev(q), blocks, cells, 1 / 16)
    torch.cuda.synchronize()
    assert (blocks[0] == n_blocks - 3).all() and (blocks[1] == n_blocks - 2).all()
    assert cells[:, 0, 0].tolist() == [476, 700]
    tail = slice(n_blocks - 3, n_blocks)
    h = {m: getattr(p, m)[tail].cpu().numpy() for m in ("k", "v", "ks", "vs")}
    want = plain_bounds("q8", h, np.zeros((3, n_kv, 2, hd), np.int8), np.zeros((3, n_kv, hd // 64), np.float32),
                        np.where(table < 0, -1, table - (n_blocks - 3)), [0, 0], lens, bs)
    assert np.array_equal(bb.codes[tail].cpu().numpy(), want[0])
    assert np.array_equal(bb.scales[tail].cpu().numpy(), want[1])
    assert not bb.codes[:-3].any()
    K, V = plain.pool_rows("q8", h["k"], h["v"], h["ks"], h["vs"])
    ref, tol = plain.attention("q8", K, V, q, blocks.cpu().numpy() - (n_blocks - 3), cells.cpu().numpy(), bs,
                               1 / 16)
    assert (np.abs(out.cpu().numpy() - ref).max(-1) <= tol).all()


def test_two_streams_at_once():
    # the same calls on two streams, each with its own outputs and workspace,
    # many times over: nothing is shared between calls
    rng = np.random.default_rng(41)
    bs, n_kv, hd, G, n_sel = 16, 2, 128, 4, 12
    lens = np.array([900, 333, 1600])
    table, n_blocks = tables(rng, lens, bs)
    p, h = fill_pool(rng, "q8", n_blocks, n_kv, bs, hd)
    bb = BlockBounds(p)
    p.bound(bb, i32(table), i32(lens), 1600)
    t, L = i32(table), i32(lens)
    qs = [dev(queries(rng, 3, 1, n_kv * G, hd)) for _ in range(2)]
    want = []
    for q in qs:
        sel = p.select(bb, q, L, 1600, t, n_sel)
        want.append((sel, p.decode_selected(q, sel[0], sel[2], 0.1)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(30):
        for i, s in enumerate(streams):
            sel = p.select(bb, qs[i], L, 1600, t, n_sel, stream=s)
            got[i].append((sel, p.decode_selected(qs[i], sel[0], sel[2], 0.1, stream=s)))
    torch.cuda.synchronize()
    for i in range(2):
        for sel, out in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(sel, want[i][0]))
            assert torch.equal(out, want[i][1])
