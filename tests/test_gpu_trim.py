"""GPU: kvq_trim_step against the plain form (tests/plain_draft.py), every
output equal, and plan and trim in turn."""
import numpy as np
import pytest
import torch

import quantized_kv_cache_append_gb300 as kvq
from quantized_kv_cache_append_gb300.steps import StepPlanner
from tests import plain_draft as plain
from tests.test_gpu_plan_step import dev, state

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _library():
    if not torch.cuda.is_available():
        pytest.fail("the GPU suite needs a CUDA device")
    kvq.build()
    kvq.load_library()


def check(ctx, drop, table, free, count, bs, n_blocks):
    n, width = table.shape
    want = plain.trim(ctx, drop, table, free, count, bs, n_blocks)
    mk = lambda m: torch.full((m,), 12345, dtype=torch.int32, device="cuda")
    got = dict(ctx_out=mk(n), free_count_out=mk(1), free_list=dev(free), info=mk(4))
    t = dev(table)
    st = kvq.kvq_trim_step(dev(ctx), dev(drop), n, bs, n_blocks, t, width, got["free_list"], dev([count]),
                           got["ctx_out"], got["free_count_out"], got["info"])
    assert st == kvq.KVQ_OK, kvq.kvq_status_string(st)
    torch.cuda.synchronize()
    assert torch.equal(t, dev(table))
    for k, v in want.items():
        assert np.array_equal(got[k].cpu().numpy().reshape(np.shape(v)), v), k
    return want


@pytest.mark.parametrize("n_seq,bs,hi,drop,seed", [
    (1, 16, 1, 1, 0), (1, 1024, 3000, 3000, 1), (3, 16, 50, 40, 2), (64, 256, 16383, 5, 3), (257, 32, 900, 70, 4),
    (1025, 16, 100, 9, 5), (5000, 64, 700, 700, 6), (16384, 16, 33, 33, 7), (2, 16, 40, 0, 8),
])
def test_random_trims(n_seq, bs, hi, drop, seed):
    rng = np.random.default_rng(seed)
    ctx = rng.integers(0, hi + 1, n_seq)
    table, free, count, n_blocks = state(rng, ctx, bs, hi // bs + 1, n_seq // 2 + 3)
    back = int((-(-ctx // bs)).sum())
    free = np.concatenate([free, np.full(max(0, count + back - len(free)), -7, np.int32)])
    want = check(ctx, np.minimum(rng.integers(0, drop + 1, n_seq), ctx), table, free, count, bs, n_blocks)
    assert want["info"][3] == 0
    check(ctx, ctx, table, free, count, bs, n_blocks)          # everything taken back


@pytest.mark.parametrize("why", ["below", "more", "negative", "row", "list", "count", "several", "both"])
def test_a_broken_trim_changes_nothing(why):
    rng = np.random.default_rng(1)
    bs, ctx, drop = 16, np.array([30, 5, 0, 100]), np.array([3, 5, 0, 90])
    table, free, count, n_blocks = state(rng, ctx, bs, 8, 4)
    if why in ("below", "several"):
        drop = np.array([3, 5, 0, -1])
    if why == "more":
        drop = np.array([31, 5, 0, 90])
    if why == "negative":
        ctx, drop = np.array([30, -5, 0, 100]), np.array([3, -5, 0, 90])
    if why == "row":
        ctx = np.array([30, 5, 0, 129])
    if why in ("list", "several"):
        n_blocks, free = count + 1, free[:count + 1]
    if why == "count":
        count = -1
    if why == "both":
        drop, n_blocks, free = np.array([30, 6, 0, 90]), count + 1, free[:count + 1]
    want = check(ctx, drop, table, free, count, bs, n_blocks)
    # (several: the broken sequence gives nothing back, the other one block, which the list holds)
    assert want["info"][3] == {"list": 8, "count": 8, "both": 10}.get(why, 2)


@pytest.mark.parametrize("ctx,drop", [([2 ** 31 - 1, 7], [2 ** 31 - 1, 7]), ([64, 7], [2 ** 31 - 1, 7]),
                                      ([-2 ** 31, 7], [-2 ** 31, 0]), ([64, 7], [-2 ** 31, 0])])
def test_extreme_numbers_are_refused(ctx, drop):
    table, free = np.arange(8, dtype=np.int32).reshape(2, 4), np.arange(8, dtype=np.int32)
    assert check(np.array(ctx), np.array(drop), table, free, 0, 16, 8)["info"][3] == 2


def test_plan_and_trim_in_turn():
    # a planner's blocks: every one is in the table or on the list, never twice
    rng = np.random.default_rng(2)
    n, width, bs, n_blocks = 40, 12, 16, 300
    p = StepPlanner(n, width, bs, n_blocks, 4000)
    ctx = np.zeros(n, np.int64)
    for step in range(25):
        new = np.where(rng.random(n) < 0.1, -1, rng.integers(0, 9, n))
        new = np.where(ctx + np.maximum(new, 0) > width * bs, -1, new)
        p.plan(dev(new))
        ctx = np.where(new < 0, 0, ctx + new)
        drop = np.minimum(np.where(rng.random(n) < 0.1, ctx, rng.integers(0, 6, n)), ctx)
        p.trim(dev(drop))
        torch.cuda.synchronize()
        assert p.info[3] == 0 and p.info[0] == drop.sum()
        assert np.array_equal(p.ctx_start.cpu().numpy(), ctx)
        ctx = ctx - drop
        assert np.array_equal(p.ctx_lens.cpu().numpy(), ctx)
        table, count = p.block_table.cpu().numpy(), int(p.free_count[0])
        held = [x for b in range(n) for x in table[b, :-(-ctx[b] // bs)]] + list(p.free_list[:count].cpu().numpy())
        assert sorted(held) == list(range(n_blocks))


def test_method_refuses():
    p = StepPlanner(3, 4, 16, 12, 30)
    for bad in (torch.zeros(2, dtype=torch.int32, device="cuda"), torch.zeros(3, device="cuda"),
                torch.zeros(3, dtype=torch.int32)):
        with pytest.raises(kvq.KvqError):
            p.trim(bad)
