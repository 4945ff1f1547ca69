"""GPU: a speculative decoding step as a serving loop runs it (plan, rotary
append, scored attention, verification, trim), eagerly and captured, and the
prompt before it (rotary append, compaction, scored chunk attention)."""
import numpy as np
import pytest
import torch

import quantized_kv_cache_append_gb300 as kvq
from quantized_kv_cache_append_gb300.draft import verify_draft
from quantized_kv_cache_append_gb300.pool import PagedPool
from quantized_kv_cache_append_gb300.steps import StepPlanner
from tests import plain_blocks, plain_draft, plain_scores

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


class Loop:
    """n sequences, W tokens each a step, everything in buffers that stay where they are."""

    def __init__(self, fmt, n, W, n_kv, G, hd, V, bs=16, width=40, window=0):
        self.fmt, self.n, self.W, self.n_kv, self.G, self.hd, self.V, self.bs = fmt, n, W, n_kv, G, hd, V, bs
        self.planner = StepPlanner(n, width, bs, n * width, n * 300)
        self.pool = PagedPool(FORMATS[fmt], n_kv, hd, bs, n * width)
        self.sm = hd ** -0.5
        self.max_ctx = width * bs
        inv = (10000.0 ** (-np.arange(hd // 2) / (hd // 2))).astype(np.float32)
        self.w = dev(np.random.default_rng(0).uniform(0.5, 1.5, (2, hd)).astype(np.float32))
        self.rotary = kvq.make_rotary(kvq.KVQ_T_BF16, hd, False, dev(inv), q_norm=self.w[0], k_norm=self.w[1], eps=1e-6)
        self.slopes = dev((2.0 ** -np.arange(1.0, n_kv * G + 1)).astype(np.float32))
        self.scores = kvq.make_scores(20.0, window, self.slopes)
        z = lambda *s, dt=torch.float32: torch.zeros(s, dtype=dt, device="cuda")
        i32 = torch.int32
        self.n_new = torch.full((n,), W, dtype=i32, device="cuda")
        self.qkv = z(n * W, (G + 2) * n_kv, hd, dt=torch.bfloat16)
        self.q = z(n * W, n_kv * G, hd)
        self.out = z(n, W, n_kv * G, hd)
        self.ws = z(max(kvq.kvq_scored_workspace_bytes(self.pool.cache, self.scores, n, W, n_kv * G, self.max_ctx), 256),
                    dt=torch.uint8)
        self.target, self.draft = z(n, W, V), z(n, W - 1, V)
        self.tokens, self.u, self.us = z(n, W - 1, dt=i32), z(n, W - 1), z(n)
        self.verdict = (z(n, dt=i32), z(n, W, dt=i32), z(n, dt=i32))

    def fill(self, rng):
        self.qkv.copy_(dev(rng.standard_normal(tuple(self.qkv.shape)).astype(np.float32)))
        p = rng.random((self.n, self.W, self.V)).astype(np.float32) ** 6
        q = p[:, :self.W - 1] * rng.uniform(0.5, 2, (self.n, self.W - 1, self.V)).astype(np.float32)
        p, q = p / p.sum(-1, keepdims=True), q / q.sum(-1, keepdims=True)
        self.target.copy_(dev(p))
        self.draft.copy_(dev(q))
        self.tokens.copy_(dev(((np.cumsum(q, -1) < rng.random(q.shape[:2])[..., None]).sum(-1)).clip(0, self.V - 1).astype(np.int32)))
        self.u.copy_(dev(rng.random((self.n, self.W - 1)).astype(np.float32)))
        self.us.copy_(dev(rng.random(self.n).astype(np.float32)))

    def step(self):
        n, W, n_q, pl = self.n, self.W, self.n_kv * self.G, self.planner
        pl.plan(self.n_new)
        k, v = self.qkv[:, n_q:n_q + self.n_kv], self.qkv[:, n_q + self.n_kv:]
        self.pool.append_rotary(self.rotary, self.qkv[:, :n_q], k, v, pl.tok_seq[:n * W], pl.tok_pos[:n * W],
                                pl.block_table, q_out=self.q)
        self.pool.decode_scored(self.q.view(n, W, n_q, self.hd), pl.ctx_lens, self.max_ctx, pl.block_table, self.sm,
                                self.scores, out=self.out, workspace=self.ws)
        verify_draft(self.target, self.draft, self.tokens, self.u, self.us, out=self.verdict)
        pl.trim(self.verdict[2])


@pytest.mark.parametrize("fmt,W,n_kv,G,hd,window", [("f16", 4, 2, 2, 64, 0), ("q8", 3, 1, 4, 128, 40),
                                                     ("k8v4", 2, 2, 3, 256, 0), ("q8", 8, 2, 2, 64, 25)])
def test_steps_against_the_definitions(fmt, W, n_kv, G, hd, window):
    rng = np.random.default_rng(W)
    s = Loop(fmt, 5, W, n_kv, G, hd, 300, window=window)
    host = lambda t: None if t is None else t.cpu().numpy()
    lens = np.zeros(5, np.int64)
    for i in range(12):
        s.fill(rng)
        before = [None if t is None else t.clone() for t in (s.pool.k, s.pool.v, s.pool.ks, s.pool.vs)]
        s.step()
        torch.cuda.synchronize()
        ctx = lens + W
        assert np.array_equal(host(s.planner.ctx_start), ctx) and int(s.planner.info[3]) == 0
        table = host(s.planner.block_table)
        # q: the definition; the cells of earlier steps are as they were
        pos = np.concatenate([np.arange(c - W, c) for c in ctx])
        want, size = plain_draft.rotated(host(s.qkv[:, :n_kv * G].float()), pos[None], host(s.rotary.held[0]), hd, False,
                                         host(s.w[0]), 1e-6)
        assert (np.abs(host(s.q) - want) <= 2.0 ** -19 * size + 1e-30).all()
        for old, new in zip(before, (s.pool.k, s.pool.v, s.pool.ks, s.pool.vs)):
            if old is not None:
                for b in range(5):
                    cell = np.arange(lens[b])
                    assert torch.equal(old[table[b, cell // s.bs], :, cell % s.bs], new[table[b, cell // s.bs], :, cell % s.bs])
        # attention over the pool as it is now
        K, V = plain_blocks.pool_rows(fmt, host(s.pool.k), host(s.pool.v), host(s.pool.ks), host(s.pool.vs))
        want, tol = plain_scores.decode(K, V, host(s.q).reshape(s.out.shape), ctx, table, s.bs, s.sm, 20.0, window,
                                        host(s.slopes), None, plain_blocks.hadamard(hd) if fmt == "k8v4" else None,
                                        {"f16": None, "q8": 127, "k8v4": 8}[fmt])
        assert (np.abs(host(s.out) - want) <= tol).all()
        # drafts, and the cells that stay
        want = plain_draft.verify(host(s.target), host(s.draft), host(s.tokens), None, host(s.u), host(s.us))
        assert all(np.array_equal(host(a), b) for a, b in zip(s.verdict, want))
        lens = ctx - want[2]
        assert np.array_equal(host(s.planner.ctx_lens), lens)
        held = sum(-(-int(x) // s.bs) for x in lens)
        assert int(s.planner.free_count[0]) == s.planner.n_blocks - held


def test_a_captured_step_is_the_eager_one():
    a, b = (Loop("q8", 4, 4, 2, 4, 128, 1000) for _ in range(2))
    rng = np.random.default_rng(1)
    for s in (a, b):
        s.fill(np.random.default_rng(0))
        s.step()                      # (kernels' one-time setup outside the capture)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        b.step()
    for i in range(10):
        seed = int(rng.integers(1 << 30))
        for s in (a, b):
            s.fill(np.random.default_rng(seed))
        a.step()
        g.replay()
        torch.cuda.synchronize()
        for x, y in ((a.out, b.out), (a.q, b.q), (a.pool.k, b.pool.k), (a.pool.v, b.pool.v), *zip(a.verdict, b.verdict),
                     (a.planner.ctx_lens, b.planner.ctx_lens), (a.planner.block_table, b.planner.block_table),
                     (a.planner.free_list, b.planner.free_list), (a.planner.free_count, b.planner.free_count)):
            assert torch.equal(x, y)


@pytest.mark.parametrize("fmt,hd,axes,interleaved", [("f16", 128, 1, False), ("q8", 64, 3, True), ("k8v4", 256, 2, False)])
def test_a_prompt(fmt, hd, axes, interleaved):
    # rotary append of a prompt (image positions for several axes), compaction, the chunk's last
    # tokens with a bidirectional prefix and capped scores
    rng = np.random.default_rng(axes)
    n, n_kv, G, bs, T = 500, 2, 3, 32, 77
    qkv = dev(rng.standard_normal((n, (G + 2) * n_kv, hd)).astype(np.float32)).to(torch.float16)
    pos = np.arange(n)
    grid = np.stack([pos // 64, pos // 8 % 8, pos % 8][:axes]) if axes > 1 else None
    pair_axis = (np.arange(hd // 2) % axes).astype(np.int32)
    inv = (100.0 ** (-np.arange(hd // 2) / (hd // 2))).astype(np.float32)
    r = kvq.make_rotary(kvq.KVQ_T_F16, hd, interleaved, dev(inv), dev(pair_axis) if axes > 1 else None, axes)
    pool = PagedPool(FORMATS[fmt], n_kv, hd, bs, 16)
    table = dev(rng.permutation(16).astype(np.int32)[None])
    seq = torch.zeros(n, dtype=torch.int32, device="cuda")
    q = pool.append_rotary(r, qkv[:, :n_kv * G], qkv[:, n_kv * G:n_kv * (G + 1)], qkv[:, n_kv * (G + 1):], seq,
                           dev(pos.astype(np.int32)), table, None if grid is None else dev(grid.astype(np.int32)))
    k16, v16 = pool.compact(table[0], n)
    last = np.where(np.arange(n - T, n) < n - 30, n - 31, 0).astype(np.int32)
    out = torch.empty(T, n_kv * G, hd, dtype=torch.bfloat16, device="cuda")
    kvq.check(kvq.kvq_chunk_attn_scored(k16, v16, n_kv, n, hd, kvq.make_scores(30.0, last=dev(last)), q[n - T:].contiguous(),
                                        T, n_kv * G, hd ** -0.5, out, kvq.KVQ_T_BF16))
    torch.cuda.synchronize()
    host = lambda t: t.cpu().numpy()
    want, size = plain_draft.rotated(host(qkv[:, :n_kv * G].float()), grid if axes > 1 else pos[None], inv, hd, interleaved,
                                     pair_axis=pair_axis if axes > 1 else None)
    assert (np.abs(host(q) - want) <= 2.0 ** -19 * size + 1e-30).all()
    want, tol = plain_scores.chunk(host(k16), host(v16), host(q)[n - T:], hd ** -0.5, 30.0, last=last, out_step=2.0 ** -8)
    assert (np.abs(host(out.float()) - want) <= tol).all()
