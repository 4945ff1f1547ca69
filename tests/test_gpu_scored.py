"""GPU: kvq_decode_attn_scored against the definition in 64 bits
(tests/plain_scores.py), masked cells, empty rows, splits, streams, graphs and
the failure path."""
import numpy as np
import pytest
import torch

import quantized_kv_cache_append_gb300 as kvq
from quantized_kv_cache_append_gb300.pool import PagedPool
from tests import plain_blocks, plain_scores

pytestmark = pytest.mark.gpu

FORMATS = {"f16": kvq.KVQ_F16, "q8": kvq.KVQ_Q8, "k8v4": kvq.KVQ_K8V4}


@pytest.fixture(scope="module", autouse=True)
def _library():
    if not torch.cuda.is_available():
        pytest.fail("the GPU suite needs a CUDA device")
    kvq.build()
    kvq.load_library()


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def ints(a):
    return dev(np.asarray(a, np.int32))


class Case:
    def __init__(self, rng, fmt, n_kv, G, hd, W, bs, lens, q_scale=1.0, max_ctx=None):
        self.fmt, self.n_kv, self.hd, self.bs, self.W = fmt, n_kv, hd, bs, W
        self.lens = np.asarray(lens)
        nb = -(-self.lens // bs)
        self.max_ctx = max_ctx or max(int(self.lens.max()), W)
        width = -(-self.max_ctx // bs) + 1
        self.n_blocks = int(nb.sum()) + 1
        perm = rng.permutation(self.n_blocks)
        self.table = np.full((len(lens), width), -1)
        at = 0
        for b, n in enumerate(nb):
            self.table[b, :n] = perm[at:at + n]
            at += n
        self.pool = PagedPool(FORMATS[fmt], n_kv, hd, bs, self.n_blocks)
        n_tok = int(self.lens.sum())
        if n_tok:
            k, v = rng.standard_normal((2, n_tok, n_kv, hd)).astype(np.float32)
            k[..., rng.integers(0, hd, 3)] *= 5
            seq = np.repeat(np.arange(len(lens)), self.lens)
            pos = np.concatenate([np.arange(n) for n in self.lens])
            self.pool.append(dev(k), dev(v), ints(seq), ints(pos), ints(self.table))
        self.q = (rng.standard_normal((len(lens), W, n_kv * G, hd)) * q_scale).astype(np.float32)
        self.sm_scale = hd ** -0.5

    def run(self, scores, pool=None, **kw):
        out = (pool or self.pool).decode_scored(dev(self.q), ints(self.lens), self.max_ctx, ints(self.table),
                                                self.sm_scale, scores, **kw)
        torch.cuda.synchronize()
        return out

    def check(self, cap=0.0, window=0, slopes=None, first=None, top=2.0 ** 8, **kw):
        scores = kvq.make_scores(cap, window, None if slopes is None else dev(slopes),
                                 None if first is None else ints(first))
        got = self.run(scores, **kw)
        host = lambda t: None if t is None else t.cpu().numpy()
        p = self.pool
        K, V = plain_blocks.pool_rows(self.fmt, host(p.k), host(p.v), host(p.ks), host(p.vs))
        want, tol = plain_scores.decode(K, V, self.q, self.lens, self.table, self.bs, self.sm_scale, float(np.float32(cap)),
                                        window, slopes, first,
                                        plain_blocks.hadamard(self.hd) if self.fmt == "k8v4" else None,
                                        {"f16": None, "q8": 127, "k8v4": 8}[self.fmt], top)
        err = np.abs(got.cpu().numpy() - want)
        assert (err <= tol).all(), f"{float((err / np.maximum(tol, 1e-300)).max()):.3g} of the tolerance"
        return got, want


def slopes_of(n_q):
    return (2.0 ** (-8.0 * (np.arange(n_q) + 1) / n_q)).astype(np.float32)


SHAPES = [  # n_kv, G, hd, W, bs, lens
    (1, 1, 64, 1, 16, [1]), (2, 4, 128, 1, 64, [777]), (1, 8, 256, 4, 16, [130, 4, 3, 65]),
    (3, 7, 64, 2, 32, [64, 63, 65, 1, 0]), (8, 4, 128, 1, 256, [1000, 17, 300]), (1, 32, 128, 1, 128, [515, 128]),
    (2, 2, 64, 16, 64, [200, 16, 7]), (1, 3, 128, 5, 1024, [2000]), (2, 1, 256, 2, 64, [6000, 100]),
    (1, 4, 64, 8, 16, [900]),
]
SCORES = [dict(cap=30.0), dict(slopes=True), dict(window=100), dict(cap=2.0, window=64, slopes=True, first=True),
          dict(first=True), dict(cap=50.0, window=1), dict()]


@pytest.mark.parametrize("fmt", ["f16", "q8", "k8v4"])
@pytest.mark.parametrize("score", range(len(SCORES)))
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_shapes_and_scores(shape, score, fmt):
    rng = np.random.default_rng([shape, score])
    c = Case(rng, fmt, *SHAPES[shape], q_scale=3.0 if score == 0 else 1.0)
    s = dict(SCORES[score])
    if s.get("slopes"):
        s["slopes"] = slopes_of(c.q.shape[2])
    if s.get("first"):
        s["first"] = rng.integers(-2, np.maximum(c.lens, 1) + 2)
    c.check(**s)


@pytest.mark.parametrize("fmt", ["f16", "q8", "k8v4"])
@pytest.mark.parametrize("window", [1, 15, 63, 64, 65, 500, 4096, 9999, 10000, 2 ** 31 - 1])
def test_windows_of_one_long_sequence(window, fmt):
    rng = np.random.default_rng(window)
    Case(rng, fmt, 2, 4, 128, 1 + window % 3, 64, [10000]).check(cap=20.0, window=window)


@pytest.mark.parametrize("cap,q_scale", [(1e-3, 1.0), (0.5, 4.0), (5.0, 30.0), (50.0, 100.0), (1e6, 1.0)])
def test_caps(cap, q_scale):
    # from scores far below the cap to all of them at it
    rng = np.random.default_rng(int(q_scale))
    for fmt in ("f16", "q8"):
        Case(rng, fmt, 2, 4, 128, 1, 32, [700, 40], q_scale=q_scale).check(cap=cap)


def test_steep_and_negative_slopes():
    # a steep slope leaves the newest cells alone, a negative one favours the oldest
    rng = np.random.default_rng(1)
    c = Case(rng, "f16", 2, 4, 64, 2, 16, [3000, 333])
    c.check(slopes=np.array([8, 100, 0, 1e-3, -1e-3, -0.05, 2, 0.3], np.float32))


def test_bad_blocks_are_hidden():
    rng = np.random.default_rng(2)
    c = Case(rng, "q8", 2, 2, 128, 1, 32, [500, 90])
    c.table[0, 3], c.table[0, 9], c.table[1, 0] = -1, c.n_blocks, 2 ** 31 - 1
    c.check(cap=10.0, window=300)


@pytest.mark.parametrize("fmt", ["f16", "q8", "k8v4"])
def test_hidden_cells_may_hold_anything(fmt):
    # NaN and infinity in every cell no token sees: before `first` or the
    # window, behind the context's end, in the unused block
    rng = np.random.default_rng(3)
    for kw, W, lens in ((dict(window=100), 1, [1000, 333, 64]), (dict(first=[500, 0, 63]), 4, [1000, 333, 70]),
                        (dict(window=70, first=[0, 300, 5]), 2, [1000, 333, 7]), (dict(window=33), 1, [2000])):
        c = Case(rng, fmt, 2, 4, 128, W, 16, lens)
        first = kw.get("first", [0] * len(lens))
        scores = kvq.make_scores(15.0, kw.get("window", 0), None, ints(first) if "first" in kw else None)
        want = c.run(scores)
        clean = torch.ones(c.n_blocks, c.bs, dtype=torch.bool)
        for b, L in enumerate(lens):
            low = max(first[b], L - W - kw["window"] + 1 if "window" in kw else 0, 0)
            for j in range(low, L):
                clean[c.table[b, j // c.bs], j % c.bs] = False
        hidden = clean.cuda()[:, None, :, None]
        for name, t in (("k", c.pool.k), ("v", c.pool.v), ("ks", c.pool.ks), ("vs", c.pool.vs)):
            if t is not None and t.dtype == torch.float16:
                t.masked_fill_(hidden, float("nan"))
                t[..., ::2].masked_fill_(hidden, float("inf"))
            elif t is not None:
                t.masked_fill_(hidden, -128 if t.dtype == torch.int8 else 255)
        got = c.run(scores)
        assert torch.equal(got, want) and bool(got.isfinite().all())


def test_rows_without_cells_and_rows_behind():
    # every token hidden: 0, also where other sequences have thousands of cells
    rng = np.random.default_rng(4)
    c = Case(rng, "f16", 2, 4, 128, 2, 64, [3000, 0, 1, 64, 128])
    got, want = c.check(first=[3000, 0, 1, 64, 2 ** 31 - 1])
    assert not got.any() and not want.any()
    got, _ = c.check(first=[2999, 0, 0, 63, 127])      # the last token alone
    assert not got[0, 0].any() and got[0, 1].any()
    # one sequence alone
    c = Case(rng, "q8", 2, 4, 128, 2, 64, [3000])
    got, _ = c.check(first=[3000])
    assert not got.any()
    got, _ = c.check(first=[3000], window=10)
    assert not got.any()


def test_nan_and_infinity_in_seen_cells_reach_their_rows():
    rng = np.random.default_rng(5)
    c = Case(rng, "f16", 2, 2, 64, 1, 16, [300, 300])
    scores = kvq.make_scores(10.0, 100, dev(slopes_of(4)))
    want = c.run(scores)
    c.pool.k[c.table[0, 250 // 16], 1, 250 % 16, 5] = float("nan")
    got = c.run(scores)
    assert got[0, 0, 2:].isnan().all() and torch.equal(got[1], want[1]) and torch.equal(got[0, 0, :2], want[0, 0, :2])


def test_large_value_scales():
    # V scales above 128: p times the scale must not leave fp16's range under rising logits
    rng = np.random.default_rng(6)
    for fmt in ("q8", "k8v4"):
        c = Case(rng, fmt, 1, 4, 128, 1, 64, [2000])
        c.pool.vs.fill_(3000.0)
        got, _ = c.check(slopes=np.array([0.05, 0.2, 0.5, 0.01], np.float32), top=1.0)
        assert bool(got.isfinite().all())


def test_matches_the_dense_decode():
    # no cap, no bias, no window: the dense decode's answer within both roundings
    rng = np.random.default_rng(7)
    for fmt in ("f16", "q8", "k8v4"):
        c = Case(rng, fmt, 2, 4, 128, 2, 64, [1500, 90])
        a = c.run(kvq.make_scores())
        b = c.pool.decode(dev(c.q), ints(c.lens), c.max_ctx, ints(c.table), c.sm_scale)
        assert float((a - b).abs().max()) < 2e-4


def test_window_bounds_the_workspace():
    c = kvq.make_cache(kvq.KVQ_F16, 8, 128, 64, 4096, 1 << 20, 1 << 21)
    full = kvq.kvq_scored_workspace_bytes(c, kvq.make_scores(), 1, 1, 32, 262144)
    small = kvq.kvq_scored_workspace_bytes(c, kvq.make_scores(window=64), 1, 1, 32, 262144)
    assert 0 < small < full
    assert kvq.kvq_scored_workspace_bytes(c, kvq.make_scores(window=1 << 30), 1, 1, 32, 262144) == full


def test_long_max_ctx_short_sequences():
    # max_ctx far above every length, and a batch whose lengths differ by 1000 times
    rng = np.random.default_rng(8)
    c = Case(rng, "f16", 2, 4, 64, 1, 64, [20, 9000, 1, 640], max_ctx=65536)
    c.check(window=700, cap=30.0)
    c.check(first=[5, 8000, 0, 600])


@pytest.mark.parametrize("n_seq,hi,n_kv,G,W,fmt", [
    (2, 9000, 1, 1, 1, "f16"), (7, 3000, 2, 2, 2, "q8"), (31, 500, 1, 4, 1, "k8v4"), (33, 700, 1, 1, 1, "f16"),
    (100, 300, 2, 1, 1, "q8"), (128, 200, 1, 2, 1, "f16"), (129, 200, 1, 2, 1, "f16"), (90, 150, 7, 1, 1, "f16"),
    (300, 70, 1, 1, 1, "q8"),
])
def test_ragged_batches(n_seq, hi, n_kv, G, W, fmt):
    # lengths of one cell to hi, some empty, one many times the others'
    rng = np.random.default_rng(n_seq)
    lens = np.exp(rng.uniform(0, np.log(hi), n_seq)).astype(int)
    lens[rng.random(n_seq) < 0.1] = 0
    lens[n_seq // 2] = hi
    c = Case(rng, fmt, n_kv, G, 64, W, 16, lens, max_ctx=hi + 40)
    c.check(cap=20.0)
    c.check(window=90, first=rng.integers(0, np.maximum(lens, 1)))
    lens[:] = 0
    c.lens = lens
    got, _ = c.check(cap=20.0)
    assert not got.any()


def test_streams_and_two_graphs():
    rng = np.random.default_rng(9)
    c = Case(rng, "q8", 2, 4, 128, 1, 64, [3000, 700])
    scores = kvq.make_scores(20.0, 512)
    want = c.run(scores)
    assert torch.equal(c.run(scores, stream=torch.cuda.Stream()), want)
    q, lens, table = dev(c.q), ints(c.lens), ints(c.table)
    graphs = []
    for _ in range(2):     # each with a workspace of its own
        out = torch.zeros_like(want)
        c.pool.decode_scored(q, lens, c.max_ctx, table, c.sm_scale, scores, out=out)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.pool.decode_scored(q, lens, c.max_ctx, table, c.sm_scale, scores, out=out)
        graphs.append((g, out))
    for _ in range(2):
        for g, out in graphs:
            out.zero_()
            g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(out, want) for _, out in graphs)


def test_lost_waits_give_nan_and_leave_the_context_usable():
    rng = np.random.default_rng(10)
    for fmt in ("f16", "q8", "k8v4"):
        c = Case(rng, fmt, 2, 4, 128, 1, 64, [700, 0, 300])
        scores = kvq.make_scores(20.0, 256)
        want = c.run(scores)
        q, out = dev(c.q), torch.zeros_like(want)
        ws = torch.empty(kvq.kvq_scored_workspace_bytes(c.pool.cache, scores, 3, 1, 8, c.max_ctx), dtype=torch.uint8,
                         device="cuda")
        st = kvq.kvq_decode_attn_scored_lost_wait_test(
            c.pool.cache, scores, q, 3, 1, 8, ints(c.lens), c.max_ctx, ints(c.table), c.table.shape[1], c.sm_scale, out,
            ws, ws.numel(), 3000, 16)
        assert st == kvq.KVQ_OK
        torch.cuda.synchronize()
        assert out[[0, 2]].isnan().all() and not out[1].any()
        assert torch.equal(c.run(scores), want)


def test_methods_refuse():
    rng = np.random.default_rng(11)
    c = Case(rng, "f16", 2, 4, 128, 1, 64, [100, 50])
    for scores in (kvq.make_scores(slopes=dev(np.ones(7, np.float32))), kvq.make_scores(first=ints([1])),
                   kvq.make_scores(first=ints([1, 2]), last=ints([1, 2])), kvq.make_scores(softcap=-1.0),
                   kvq.make_scores(window=-1), kvq.make_scores(slopes=torch.ones(8))):
        with pytest.raises(kvq.KvqError):
            c.run(scores)
    with pytest.raises(kvq.KvqError):
        c.run(kvq.make_scores(), workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
