"""GPU: kvq_plan_step against the plain form (tests/plain_blocks.py), every
output equal, untouched entries unchanged."""
import numpy as np
import pytest
import torch

import quantized_kv_cache_append_gb300 as kvq
from quantized_kv_cache_append_gb300.steps import StepPlanner
from tests import plain_blocks as plain

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _library():
    if not torch.cuda.is_available():
        pytest.fail("the GPU suite needs a CUDA device")
    kvq.build()
    kvq.load_library()


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(np.asarray(a, np.int32))).cuda()


def state(rng, ctx, bs, width, extra):
    """Table rows of shuffled blocks for ctx, and a stack of `extra` free ones."""
    nb = [-(-max(int(c), 0) // bs) for c in ctx]
    n_blocks = sum(nb) + extra
    perm = rng.permutation(max(n_blocks, 1)).astype(np.int32)
    table = np.full((len(ctx), width), -1, np.int32)
    at = 0
    for b, n in enumerate(nb):
        n = min(n, width)
        table[b, :n] = perm[at:at + n]
        at += nb[b]
    free = np.full(max(n_blocks, 1), -7, np.int32)
    free[:extra] = perm[at:at + extra]
    return table, free, extra, max(n_blocks, 1)


def run(ctx, n_new, table, free, count, bs, n_blocks, max_tok, slots=True):
    n, width = table.shape
    d = dict(block_table=dev(table), free_list=dev(free))
    mk = lambda m: torch.full((m,), 12345, dtype=torch.int32, device="cuda")
    d.update(ctx_out=mk(n), tok_start=mk(n + 1), tok_seq=mk(max_tok), tok_pos=mk(max_tok),
             slots=mk(max_tok), free_count_out=mk(1), info=mk(4))
    st = kvq.kvq_plan_step(dev(ctx), dev(n_new), n, bs, n_blocks, d["block_table"], width,
                           d["free_list"], dev([count]), max_tok, d["ctx_out"], d["tok_start"],
                           d["tok_seq"], d["tok_pos"], d["slots"] if slots else None,
                           d["free_count_out"], d["info"])
    assert st == kvq.KVQ_OK, kvq.kvq_status_string(st)
    torch.cuda.synchronize()
    got = {k: v.cpu().numpy() for k, v in d.items()}
    got["free_count_out"] = int(got["free_count_out"][0])
    return got


def check(ctx, n_new, table, free, count, bs, n_blocks, max_tok, slots=True):
    want = plain.plan(ctx, n_new, table, free, count, bs, n_blocks, max_tok)
    got = run(ctx, n_new, table, free, count, bs, n_blocks, max_tok, slots)
    for k, v in want.items():
        if k == "slots" and not slots:
            assert (got[k] == 12345).all()
        else:
            assert np.array_equal(got[k], v), k
    return want


@pytest.mark.parametrize("n_seq,bs,hi,new,seed", [
    (1, 16, 1, 1, 0), (1, 1024, 3000, 1, 1), (3, 16, 50, 40, 2), (64, 256, 16383, 1, 3),
    (257, 32, 900, 70, 4), (513, 16, 100, 9, 5), (1000, 64, 4000, 300, 6), (2, 16, 40, 5001, 7),
])
def test_random_steps(n_seq, bs, hi, new, seed):
    rng = np.random.default_rng(seed)
    ctx = rng.integers(0, hi + 1, n_seq)
    kind = rng.random(n_seq)
    n_new = np.where(kind < 0.5, rng.integers(0, new + 1, n_seq), np.where(kind < 0.75, 1, -1))
    width = (hi + new) // bs + 1
    table, free, count, n_blocks = state(rng, ctx, bs, width, n_seq * (new // bs + 2))
    total = int(np.maximum(n_new, 0).sum())
    for max_tok in {max(total, 1), total + 1, total + 4099}:
        want = check(ctx, n_new, table, free, count, bs, n_blocks, max_tok, slots=max_tok != total + 1)
        assert want["info"][3] == 0


@pytest.mark.parametrize("released,grown", [(3, 1), (1, 3), (2, 2), (4, 0), (0, 4)])
def test_blocks_given_back_are_handed_out_again(released, grown):
    # more, fewer and as many blocks come back as are needed, with 0, 1 or
    # plenty on the free list before
    rng = np.random.default_rng(released * 10 + grown)
    bs = 16
    ctx = np.array([48, 17, 33, 16, 0, 64])
    n_new = np.zeros(6, np.int64)
    n_new[:released] = -1
    n_new[released:released + grown] = [40, 3, 100, 1][:grown]
    for extra in (0, 1, 50):
        table, free, count, n_blocks = state(rng, ctx, bs, 12, extra)
        check(ctx, n_new, table, free, count, bs, n_blocks, 200)


@pytest.mark.parametrize("why", ["tokens", "row", "negative", "blocks", "list", "count", "several"])
def test_a_step_that_cannot_be_placed_changes_nothing(why):
    rng = np.random.default_rng(1)
    bs, ctx, n_new = 16, np.array([30, 5, 0, 100]), np.array([3, -1, 20, 1])
    table, free, count, n_blocks = state(rng, ctx, bs, 8, 4)
    max_tok = 24
    if why == "tokens":
        max_tok = 23
    if why == "row":
        n_new = np.array([3, -1, 20, 29])
        max_tok = 100
    if why == "negative":
        ctx = np.array([30, -1, 0, 100])
    if why == "blocks":
        count = 0
        n_new = np.array([3, 0, 20, 1])
    if why == "list":
        n_blocks = count
        free = free[:count]
    if why == "count":
        count = -1
    if why == "several":
        max_tok, count, n_new = 3, 0, np.array([3, 4, 20, 29])
    want = check(ctx, n_new, table, free, count, bs, n_blocks, max_tok)
    assert want["info"][3] != 0
    assert np.array_equal(want["block_table"], table) and np.array_equal(want["free_list"], free)


def test_token_totals_past_32_bits_are_refused_not_wrapped():
    # 4096 requests of 2^20 tokens: 2^32 in all, 0 in 32 bits
    n, bs = 4096, 1024
    table = np.full((n, 1024), 0, np.int32)
    got = run(np.zeros(n), np.full(n, 1 << 20), table, np.arange(64), 64, bs, 64, 8)
    assert got["info"].tolist() == [0, 0, 0, plain.TOKENS + plain.BLOCKS]
    assert (got["ctx_out"] == 0).all() and (got["block_table"] == 0).all() and (got["tok_seq"] == -1).all()


def test_the_most_sequences_and_no_tokens():
    rng = np.random.default_rng(3)
    n = 16384
    ctx = rng.integers(0, 40, n)
    table, free, count, n_blocks = state(rng, ctx, 16, 3, 5)
    check(ctx, np.zeros(n, np.int64), table, free, count, 16, n_blocks, 1)
    n_new = np.where(rng.random(n) < 0.3, -1, 0)
    check(ctx, n_new, table, free, count, 16, n_blocks, 1)
    n_new[rng.random(n) < 0.5] = 1
    check(ctx, n_new, table, free, count, 16, n_blocks, n)


def test_a_step_without_token_arrays():
    rng = np.random.default_rng(4)
    ctx, n_new = np.array([20, 5, 0]), np.array([-1, 0, 0])
    table, free, count, n_blocks = state(rng, ctx, 16, 3, 2)
    bt, fl = dev(table), dev(free)
    mk = lambda m: torch.full((m,), 12345, dtype=torch.int32, device="cuda")
    ctx_out, start, cnt, info = mk(3), mk(4), mk(1), mk(4)
    st = kvq.kvq_plan_step(dev(ctx), dev(n_new), 3, 16, n_blocks, bt, 3, fl, dev([count]), 0, ctx_out, start,
                           None, None, None, cnt, info)
    assert st == kvq.KVQ_OK
    torch.cuda.synchronize()
    assert ctx_out.tolist() == [0, 5, 0] and info.tolist() == [0, 0, 2, 0] and cnt.tolist() == [4]
    assert fl.tolist()[2:4] == table[0, :2].tolist() and start.tolist() == [0, 0, 0, 0]


@pytest.mark.parametrize("n_seq", [1024, 1025, 2047, 5000])
def test_many_sequences(n_seq):
    # up to and past the lengths that go through shared memory
    rng = np.random.default_rng(n_seq)
    ctx = rng.integers(0, 200, n_seq)
    n_new = np.where(rng.random(n_seq) < 0.2, -1, rng.integers(0, 40, n_seq))
    table, free, count, n_blocks = state(rng, ctx, 16, 16, n_seq * 3)
    check(ctx, n_new, table, free, count, 16, n_blocks, int(np.maximum(n_new, 0).sum()) + 3)


def test_planner_runs_requests_to_their_end():
    # 40 steps of arrivals, decoding and endings, replayed on the host; the
    # blocks in use are never handed out twice, and all come back at the end
    rng = np.random.default_rng(9)
    n, bs, n_blocks, max_tok = 12, 16, 90, 128
    p = StepPlanner(n, 12, bs, n_blocks, max_tok)
    ctx = np.zeros(n, np.int64)
    table, free = p.block_table.cpu().numpy(), p.free_list.cpu().numpy()
    count = n_blocks
    refused = 0
    for step in range(40):
        n_new = np.where(ctx == 0, np.where(rng.random(n) < 0.4, rng.integers(1, 60, n), 0),
                         np.where(rng.random(n) < 0.15, -1, 1))
        if step == 39:
            n_new = np.full(n, -1)
        want = plain.plan(ctx, n_new, table, free, count, bs, n_blocks, max_tok)
        p.plan(dev(n_new))
        for k, t in dict(ctx_out=p.ctx_lens, tok_start=p.tok_start, tok_seq=p.tok_seq, tok_pos=p.tok_pos,
                         slots=p.slots, block_table=p.block_table, free_list=p.free_list,
                         info=p.info).items():
            assert np.array_equal(t.cpu().numpy(), want[k]), (step, k)
        assert int(p.free_count) == want["free_count_out"]
        assert np.array_equal(p.ctx_start.cpu().numpy(), ctx)
        ctx, table, free, count = want["ctx_out"].astype(np.int64), want["block_table"], want["free_list"], \
            want["free_count_out"]
        refused += want["info"][3] != 0
        used = [int(x) for b in range(n) for x in table[b, :-(-ctx[b] // bs)]]
        assert sorted(used + [int(x) for x in free[:count]]) == list(range(n_blocks))
    assert count == n_blocks and 0 < refused < 39


def test_planner_in_a_captured_graph():
    p = StepPlanner(4, 8, 16, 32, 16)
    n_new = dev([3, 0, 5, 1])
    p.plan(n_new)                                 # (warm-up outside the capture)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    with torch.cuda.graph(g, stream=s):
        p.plan(n_new)
    for k in range(3):
        g.replay()
    torch.cuda.synchronize()
    assert p.ctx_lens.tolist() == [12, 0, 20, 4] and p.ctx_start.tolist() == [9, 0, 15, 3]
    n_new.copy_(dev([-1, 2, 0, -1]))
    g.replay()
    torch.cuda.synchronize()
    assert p.ctx_lens.tolist() == [0, 2, 20, 0] and p.info.tolist() == [2, 1, 2, 0]
