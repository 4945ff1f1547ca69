"""GPU: kvq_chunk_attn_scored against the definition in 64 bits
(tests/plain_scores.py): caps, biases, windows, documents, prefixes, empty
rows, key splits, output types, streams, graphs and the failure path."""
import numpy as np
import pytest
import torch

import quantized_kv_cache_append_gb300 as kvq
from tests import plain_scores

pytestmark = pytest.mark.gpu

TYPES = {torch.float32: (kvq.KVQ_T_F32, 0.0), torch.float16: (kvq.KVQ_T_F16, 2.0 ** -11),
         torch.bfloat16: (kvq.KVQ_T_BF16, 2.0 ** -8)}


@pytest.fixture(scope="module", autouse=True)
def _library():
    if not torch.cuda.is_available():
        pytest.fail("the GPU suite needs a CUDA device")
    kvq.build()
    kvq.load_library()


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def ints(a):
    return None if a is None else dev(np.asarray(a, np.int32))


def slopes_of(n_q):
    return (2.0 ** (-8.0 * (np.arange(n_q) + 1) / n_q)).astype(np.float32)


class Case:
    def __init__(self, rng, n_kv, G, hd, P, T, q_scale=1.0):
        self.k, self.v = rng.standard_normal((2, n_kv, P, hd)).astype(np.float16)
        self.k[..., rng.integers(0, hd, 2)] *= 5
        self.q = (rng.standard_normal((T, n_kv * G, hd)) * q_scale).astype(np.float32)
        self.sm = hd ** -0.5
        self.dk, self.dv, self.dq = dev(self.k), dev(self.v), dev(self.q)

    def run(self, scores, dtype=torch.float32, out=None, stream=None, lost=None):
        n_kv, P, hd = self.k.shape
        T, n_q, _ = self.q.shape
        if out is None:
            out = torch.full((T, n_q, hd), 7.0, dtype=dtype, device="cuda")
            torch.cuda.synchronize()
        a = (self.dk, self.dv, n_kv, P, hd, scores, self.dq, T, n_q, self.sm, out, TYPES[dtype][0])
        st = (kvq.kvq_chunk_attn_scored(*a, stream) if lost is None
              else kvq.kvq_chunk_attn_scored_lost_wait_test(*a, *lost))
        assert st == kvq.KVQ_OK, kvq.kvq_status_string(st)
        torch.cuda.synchronize()
        return out

    def check(self, dtype=torch.float32, cap=0.0, window=0, slopes=None, first=None, last=None):
        got = self.run(kvq.make_scores(cap, window, None if slopes is None else dev(slopes), ints(first), ints(last)),
                       dtype)
        want, tol = plain_scores.chunk(self.k, self.v, self.q, self.sm, float(np.float32(cap)), window, slopes, first, last,
                                       TYPES[dtype][1])
        err = np.abs(got.float().cpu().numpy() - want)
        assert (err <= tol).all(), f"{float((err / tol).max()):.3g} of the tolerance"
        return got, want


def documents(rng, P, T, n):
    """First cells of n documents' tokens, the first one begun before the chunk."""
    cut = np.sort(rng.choice(np.arange(1, T), min(n, T) - 1, replace=False)) + P - T
    starts = np.concatenate([[(P - T) // 3], cut])
    return starts[np.searchsorted(cut, np.arange(P - T, P), side="right")]


SHAPES = [(1, 1, 64, 1, 1), (2, 4, 128, 300, 300), (2, 3, 64, 777, 130), (1, 8, 256, 400, 70), (3, 1, 128, 1500, 64),
          (1, 4, 64, 5000, 33), (2, 2, 256, 3001, 40), (1, 5, 128, 129, 128), (2, 4, 128, 4096, 1)]
SCORES = [dict(cap=30.0), dict(slopes=True), dict(window=100), dict(docs=4), dict(prefix=0.6),
          dict(cap=2.0, window=64, slopes=True, docs=3), dict(window=1), dict(prefix=0.3, slopes=True, window=50), dict()]


@pytest.mark.parametrize("score", range(len(SCORES)))
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_shapes_and_scores(shape, score):
    rng = np.random.default_rng([shape, score])
    n_kv, G, hd, P, T = SHAPES[shape]
    c = Case(rng, n_kv, G, hd, P, T, q_scale=3.0 if score == 0 else 1.0)
    s = dict(SCORES[score])
    if s.get("slopes"):
        s["slopes"] = slopes_of(n_kv * G)
    if "docs" in s:
        s["first"] = documents(rng, P, T, s.pop("docs"))
    if "prefix" in s:
        end = P - T + int(T * s.pop("prefix"))
        pos = np.arange(P - T, P)
        s["last"] = np.where(pos <= end, end, rng.integers(-5, P, T) % (pos + 1))
    c.check(list(TYPES)[(shape + score) % 3], **s)


@pytest.mark.parametrize("cap,q_scale", [(1e-3, 1.0), (0.5, 4.0), (5.0, 30.0), (50.0, 100.0), (1e6, 1.0)])
def test_caps(cap, q_scale):
    rng = np.random.default_rng(int(q_scale))
    Case(rng, 2, 4, 128, 600, 90, q_scale).check(cap=cap)


def test_rows_without_keys():
    # some rows, whole row tiles and whole chunks that see nothing, split and unsplit
    rng = np.random.default_rng(1)
    for P, T in ((700, 300), (6000, 50)):
        c = Case(rng, 2, 4, 64, P, T)
        pos = np.arange(P - T, P)
        first = np.where(np.arange(T) % 3 == 0, pos + 1, 0)
        first[T // 2:T // 2 + 40] = 2 ** 31 - 1
        for dtype in TYPES:
            got, want = c.check(dtype, first=first, cap=20.0)
            assert not got[torch.from_numpy(first > pos).cuda()].any()
            got, _ = c.check(dtype, first=pos + 1)
            assert not got.any()
    c = Case(rng, 1, 2, 256, 2000, 100)
    got, _ = c.check(first=np.full(100, 2000), window=10)
    assert not got.any()


def test_first_and_last_out_of_range():
    rng = np.random.default_rng(2)
    P, T = 500, 200
    c = Case(rng, 2, 2, 128, P, T)
    c.check(first=rng.integers(-2 ** 31, 300, T))
    c.check(last=np.full(T, 2 ** 31 - 1))          # the whole staging, both ways
    c.check(last=np.full(T, -2 ** 31), window=33)
    c.check(first=np.full(T, 450), last=np.full(T, 460))


def test_steep_and_negative_slopes_under_a_prefix():
    rng = np.random.default_rng(3)
    c = Case(rng, 2, 4, 64, 900, 400)
    c.check(slopes=np.array([8, 100, 0, 1e-3, -1e-3, -0.05, 2, 0.3], np.float32), last=np.full(400, 700))


def test_rising_scores_rescale():
    # a bias that lifts the running maximum past the lazy threshold tile after tile
    rng = np.random.default_rng(4)
    for hd in (64, 128, 256):
        c = Case(rng, 1, 2, hd, 2500, 300)
        c.check(slopes=np.array([0.12, 0.4], np.float32))
        c.check(slopes=np.array([-0.12, -0.4], np.float32))


def test_matches_the_plain_chunk():
    rng = np.random.default_rng(5)
    c = Case(rng, 2, 4, 128, 1000, 200)
    want = torch.empty(200, 8, 128, device="cuda")
    assert kvq.kvq_chunk_attn(c.dk, c.dv, 2, 1000, 128, c.dq, 200, 8, c.sm, want) == kvq.KVQ_OK
    # (the tiles run the other way, so a row's reference maximum may be another one
    # and each weight rounds to fp16 from another multiple: 2^-11 of it in either,
    # of weights that sum to 1)
    err = (c.run(kvq.make_scores()) - want).abs()
    assert float(err.max()) <= 2 * 2.0 ** -11 * float(c.dv.abs().max())


def test_documents_do_not_mix():
    # other documents' keys and values change nothing of a document's rows
    rng = np.random.default_rng(6)
    c = Case(rng, 2, 4, 128, 1000, 600)
    first = documents(rng, 1000, 600, 5)
    scores = kvq.make_scores(10.0, 0, dev(slopes_of(8)), ints(first))
    want = c.run(scores)
    mid = int(np.unique(first)[2])
    c.dk[:, mid:int(np.unique(first)[3])] += 1
    c.dv[:, mid:int(np.unique(first)[3])] *= -3
    same = torch.from_numpy(first != mid).cuda()
    got = c.run(scores)
    assert torch.equal(got[same], want[same]) and not torch.equal(got, want)


def test_streams_and_graphs():
    rng = np.random.default_rng(7)
    c = Case(rng, 2, 4, 128, 3000, 64)
    scores = kvq.make_scores(20.0, 700, dev(slopes_of(8)))
    want = c.run(scores, torch.bfloat16)
    assert torch.equal(c.run(scores, torch.bfloat16, stream=torch.cuda.Stream()), want)
    out = torch.zeros_like(want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kvq.kvq_chunk_attn_scored(c.dk, c.dv, 2, 3000, 128, scores, c.dq, 64, 8, c.sm, out, kvq.KVQ_T_BF16)
    for _ in range(2):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


@pytest.mark.parametrize("n_kv,G,hd,P,T", [(2, 4, 128, 1000, 200), (1, 4, 64, 6000, 30), (1, 4, 256, 3000, 100)])
def test_lost_waits_give_nan_and_leave_the_context_usable(n_kv, G, hd, P, T):
    rng = np.random.default_rng(8)
    c = Case(rng, n_kv, G, hd, P, T)
    scores = kvq.make_scores(20.0)
    want = c.run(scores)
    for dtype in TYPES:
        assert c.run(scores, dtype, lost=(3000, 16)).isnan().all()
    assert torch.equal(c.run(scores), want)


@pytest.mark.parametrize("hd,tile", [(64, 128), (128, 128), (256, 64)])
@pytest.mark.parametrize("splits", range(2, 9))
def test_key_splits_merge(hd, tile, splits):
    # as many key tiles as up to `splits` splits take; rows that see the keys of
    # one split or of none beside rows that see them all; two heads of a key head
    # whose scores lie far apart
    rng = np.random.default_rng([hd, splits])
    P, T = (4 * splits + 1) * tile - 5, 37
    c = Case(rng, 1, 3, hd, P, T)
    c.dq[:, 1] *= 6
    c.q[:, 1] *= 6
    pos = np.arange(P - T, P)
    first = np.where(np.arange(T) % 4 == 1, pos - 20, np.where(np.arange(T) % 4 == 2, pos + 1, 0))
    first[3] = pos[3]
    for dtype in TYPES:
        c.check(dtype, first=first)
    c.check(cap=8.0, slopes=np.array([0.5, -0.01, 0.0], np.float32))


def test_a_chunk_that_reads_the_one_before():
    # each call's q is the output of the last: launched while it ends, it must not
    # read before; the same one by one, in a row and captured
    rng = np.random.default_rng(9)
    for hd, P, T in ((64, 4000, 60), (128, 1000, 300), (256, 2000, 50)):
        c = Case(rng, 2, 2, hd, P, T)
        scores = kvq.make_scores(20.0, 600)
        bufs = [c.dq] + [torch.zeros(T, 4, hd, device="cuda") for _ in range(6)]

        def row(wait):
            for a, b in zip(bufs, bufs[1:]):
                assert kvq.kvq_chunk_attn_scored(c.dk, c.dv, 2, P, hd, scores, a, T, 4, c.sm * 8, b) == kvq.KVQ_OK
                if wait:
                    torch.cuda.synchronize()

        row(True)
        want = [b.clone() for b in bufs[1:]]
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            row(False)
        for f in (lambda: row(False), g.replay, g.replay):
            for b in bufs[1:]:
                b.zero_()
            f()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(bufs[1:], want))
