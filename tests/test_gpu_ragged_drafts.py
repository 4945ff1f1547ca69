"""GPU: a speculative decoding step whose sequences have different numbers of
drafts, some none, some no token at all, some ending, and steps the pool has no
blocks for: the planner's packed tokens, the attention's windows and the
verification's rows meet through StepPlanner.window_rows and n_draft."""
import numpy as np
import pytest
import torch

import quantized_kv_cache_append_gb300 as kvq
from quantized_kv_cache_append_gb300.draft import verify_draft
from quantized_kv_cache_append_gb300.pool import PagedPool
from quantized_kv_cache_append_gb300.steps import StepPlanner
from tests import plain_blocks, plain_draft, plain_scores
from tests.test_gpu_plan_step import dev

pytestmark = pytest.mark.gpu

FORMATS = {"f16": kvq.KVQ_F16, "q8": kvq.KVQ_Q8}
N, W, N_KV, G, HD, V, BS, WIDTH, BLOCKS = 6, 4, 2, 2, 64, 40, 16, 6, 8
N_Q = N_KV * G


@pytest.fixture(scope="module", autouse=True)
def _library():
    if not torch.cuda.is_available():
        pytest.fail("the GPU suite needs a CUDA device")
    kvq.build()
    kvq.load_library()


def f32(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.float32)).cuda()


def host(t):
    return t.cpu().numpy()


class Loop:
    """Steps as README shows them, every array in a place of its own."""

    def __init__(self, fmt, certain):
        self.fmt, self.certain = fmt, certain
        self.pl = StepPlanner(N, WIDTH, BS, BLOCKS, N * W)
        self.pool = PagedPool(FORMATS[fmt], N_KV, HD, BS, BLOCKS)
        inv = f32(100.0 ** (-np.arange(HD // 2) / (HD // 2)))
        self.rotary = kvq.make_rotary(kvq.KVQ_T_F32, HD, False, inv)
        self.scores = kvq.make_scores(softcap=20.0)
        zeros = lambda *s: torch.zeros(s, device="cuda")
        self.new = torch.zeros(N, dtype=torch.int32, device="cuda")
        self.qkv, self.target = zeros(N * W, N_Q + 2 * N_KV, HD), zeros(N * W, V)   # (packed, as the planner's tokens)
        self.draft, self.drafts = zeros(N, W - 1, V), torch.zeros(N, W - 1, dtype=torch.int32, device="cuda")
        self.u, self.us = zeros(N, W - 1), zeros(N)
        self.q, self.windows, self.out = zeros(N * W, N_Q, HD), zeros(N * W + 1, N_Q, HD), zeros(N, W, N_Q, HD)
        self.rows, self.packed = zeros(N * W + 1, V), zeros(N * W, N_Q, HD)
        self.ws = torch.zeros(max(256, kvq.kvq_scored_workspace_bytes(self.pool.cache, self.scores, N, W, N_Q, WIDTH * BS)),
                              dtype=torch.uint8, device="cuda")
        ints = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")
        self.verdict, self.n_draft = (ints(N), ints(N, W), ints(N)), ints(N)

    def fill(self, new, rng):
        self.new.copy_(dev(new))
        self.qkv.copy_(f32(rng.standard_normal(tuple(self.qkv.shape))))
        p = rng.random((N * W, V)).astype(np.float32) ** 4
        q = rng.random((N, W - 1, V)).astype(np.float32) ** 4
        self.target.copy_(f32(p / p.sum(-1, keepdims=True)))
        self.draft.copy_(f32(q / q.sum(-1, keepdims=True)))
        self.drafts.copy_(dev(rng.integers(0, V, (N, W - 1))))
        self.u.copy_(f32(rng.random((N, W - 1)) * 0.7))
        self.us.copy_(f32(rng.random(N)))

    def step(self):
        n, pl = N * W, self.pl
        pl.plan(self.new)
        pl.n_draft(out=self.n_draft)
        attend, verify = pl.window_rows(W, n)
        k, v = self.qkv[:, N_Q:N_Q + N_KV], self.qkv[:, N_Q + N_KV:]
        self.pool.append_rotary(self.rotary, self.qkv[:, :N_Q], k, v, pl.tok_seq[:n], pl.tok_pos[:n], pl.block_table,
                                q_out=self.q)
        self.windows.zero_().index_copy_(0, attend, self.q)
        self.pool.decode_scored(self.windows[:n].view(N, W, N_Q, HD), pl.ctx_lens, WIDTH * BS, pl.block_table, HD ** -0.5,
                                self.scores, out=self.out, workspace=self.ws)
        self.packed.copy_(self.out.view(n, N_Q, HD)[attend.clamp(max=n - 1)])
        self.rows.zero_().index_copy_(0, verify, self.target)
        verify_draft(self.rows[:n].view(N, W, V), None if self.certain else self.draft, self.drafts, self.u, self.us,
                     self.n_draft, out=self.verdict)
        pl.trim(self.verdict[2])


def plans(rng, steps):
    """n_new of each step; every tenth asks for more than a row holds."""
    for i in range(steps):
        new = rng.integers(1, W + 1, N)
        new[rng.random(N) < 0.25] = 0
        new[rng.random(N) < 0.12] = -1
        if i % 10 == 9:
            new[i % N] = WIDTH * BS + 1
        yield np.full(N, W) if i in (0, 7) else new


def blocks(x):
    return -(-x // BS)


@pytest.mark.parametrize("fmt,certain,seed", [("f16", False, 0), ("q8", True, 1), ("f16", True, 2)])
def test_ragged_steps_against_the_definitions(fmt, certain, seed):
    rng = np.random.default_rng(seed)
    s = Loop(fmt, certain)
    lens = np.zeros(N, np.int64)
    refused = idle = part = 0
    for new in plans(rng, 45):
        s.fill(new, rng)
        s.step()
        torch.cuda.synchronize()
        ctx = np.where(new < 0, 0, lens + np.maximum(new, 0))
        ok = blocks(ctx).sum() <= BLOCKS and (ctx <= WIDTH * BS).all()
        if not ok:
            ctx, new = lens.copy(), np.zeros(N, np.int64)
        refused, idle, part = refused + (not ok), idle + int((new == 0).sum()), part + int(((new > 0) & (new < W)).sum())
        assert bool(s.pl.plan_info[3] == 0) == ok
        placed = np.where(new < 0, -lens, new)
        assert np.array_equal(host(s.n_draft), placed - 1)
        # the packed tokens' attention
        table, q = host(s.pl.block_table), host(s.q)
        seq = np.repeat(np.arange(N), np.maximum(new, 0))
        pos = np.concatenate([np.arange(c - max(m, 0), c) for c, m in zip(ctx, new)])
        at = seq * W + W + pos - ctx[seq]
        K, V_ = plain_blocks.pool_rows(fmt, *(None if t is None else host(t) for t in (s.pool.k, s.pool.v, s.pool.ks, s.pool.vs)))
        windows = np.zeros((N * W, N_Q, HD), np.float32)
        windows[at] = q[:len(seq)]
        want, tol = plain_scores.decode(K, V_, windows.reshape(N, W, N_Q, HD), ctx, table, BS, HD ** -0.5, 20.0,
                                        code=None if fmt == "f16" else 127)
        assert (np.abs(host(s.packed)[:len(seq)] - want.reshape(N * W, N_Q, HD)[at])
                <= tol.reshape(N * W, N_Q, HD)[at]).all()
        # the verdict: target row i of a sequence is its packed token i's
        rows = np.zeros((N, W, V), np.float32)
        rows.reshape(N * W, V)[seq * W + pos - (ctx - np.maximum(new, 0))[seq]] = host(s.target)[:len(seq)]
        want = plain_draft.verify(rows, None if certain else host(s.draft), host(s.drafts), placed - 1, host(s.u), host(s.us))
        assert all(np.array_equal(host(a), b) for a, b in zip(s.verdict, want))
        assert (want[2] <= np.maximum(new, 0)).all() and (want[1][new <= 0] == -1).all()
        lens = ctx - want[2]
        assert np.array_equal(host(s.pl.ctx_lens), lens)
        assert int(s.pl.free_count[0]) == BLOCKS - blocks(lens).sum()
    assert refused and idle and part      # (every kind of row was there)


def test_a_captured_ragged_step_is_the_eager_one():
    a, b = Loop("q8", False), Loop("q8", False)
    for s in (a, b):
        s.fill([W] * N, np.random.default_rng(0))
        s.step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        b.step()
    rng, refused = np.random.default_rng(3), 0
    for new in plans(rng, 30):
        seed = int(rng.integers(1 << 30))
        for s in (a, b):
            s.fill(new, np.random.default_rng(seed))
        a.step()
        g.replay()
        torch.cuda.synchronize()
        refused += int(a.pl.plan_info[3] != 0)
        for x, y in ((a.packed, b.packed), *zip(a.verdict, b.verdict), (a.pl.ctx_lens, b.pl.ctx_lens), (a.pool.k, b.pool.k),
                     (a.pl.plan_info, b.pl.plan_info), (a.pl.free_count, b.pl.free_count), (a.n_draft, b.n_draft)):
            n = int(a.pl.plan_info[0]) if x is a.packed else len(x)
            assert torch.equal(x[:n], y[:n])
    assert refused


def test_rows_of_tokens_outside_the_window():
    # 9 tokens for a window of 4: the last 4 are its rows, the first 4 the target's; padding has none
    p = StepPlanner(3, 4, 16, 12, 16)
    p.plan(dev([9, 0, 2]))
    attend, verify = p.window_rows(4, 16)
    torch.cuda.synchronize()
    assert attend.dtype == verify.dtype == torch.int64
    assert attend.tolist() == [12] * 5 + [0, 1, 2, 3, 10, 11] + [12] * 5
    assert verify.tolist() == [0, 1, 2, 3] + [12] * 5 + [8, 9] + [12] * 5
    assert p.n_draft().tolist() == [8, -1, 1]
    p.plan(dev([100, 0, 0]))                       # refused
    assert p.n_draft().tolist() == [-1, -1, -1] and p.window_rows(4, 16)[0].tolist() == [12] * 16
    p.plan(dev([1, 1, -1]))
    assert p.n_draft().tolist() == [0, 0, -3]
    with pytest.raises(kvq.KvqError):
        p.window_rows(4, 17)
    with pytest.raises(kvq.KvqError):
        p.window_rows(0, 16)
    with pytest.raises(kvq.KvqError):
        p.n_draft(out=torch.zeros(3, device="cuda"))
