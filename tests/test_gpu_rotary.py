"""GPU: kvq_append_rotary.  q against the definition in 64 bits; the cache's
bytes against kvq_append's of the same fp32 rows (bit for bit)."""
import numpy as np
import pytest
import torch

import quantized_kv_cache_append_gb300 as kvq
from quantized_kv_cache_append_gb300.pool import ELEMENT_TYPES, PagedPool
from tests import plain_draft as plain

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


def tolerance(size, angle):
    """size: |a| + |b| of each value's pair.  The norm: a sum of squares over 8
    values and up to 5 shuffles (13 half steps, halved by the root), rsqrtf
    and two products, together below 15 * 2^-24; the angle within 2^-22 of
    the definition's (beyond 2^22 radians: three fp64 roundings of it) plus
    its fp32 rounding and sincospif's 2 ulp, below 3 * 2^-22; gain, two
    products and a sum: 4 half steps."""
    return size * (15 * 2.0 ** -24 + 3 * 2.0 ** -22 + 4 * 2.0 ** -24 + 3 * 2.0 ** -53 * angle) + 1e-37


class Call:
    """One call's inputs; strided views of one [n_tok][n_q + 2 n_kv heads + pad] array."""

    def __init__(self, rng, fmt, dtype, n_tok, n_q, n_kv, hd, rot, interleaved, axes=1, norm=True, bs=16, top=1000,
                 pad=0, gain=1.0, base=10000.0):
        width = (n_q + 2 * n_kv) * hd + pad
        x = rng.standard_normal((n_tok, width)).astype(np.float32)
        x[:, ::37] *= 20
        self.qkv = dev(x).to(dtype)
        cut = [0, n_q * hd, (n_q + n_kv) * hd, (n_q + 2 * n_kv) * hd]
        self.q, self.k, self.v = (self.qkv[:, a:b].unflatten(1, ((b - a) // hd, hd)) if b > a
                                  else self.qkv[:, :0].reshape(n_tok, 0, hd) for a, b in zip(cut, cut[1:]))
        n_seq = min(3, n_tok)
        self.seq = np.sort(rng.integers(0, n_seq, n_tok))
        self.pos = np.concatenate([top - c + np.arange(c) for c in np.bincount(self.seq, minlength=n_seq)])
        width_b = top // bs + 1
        self.n_blocks = n_seq * width_b
        self.table = rng.permutation(self.n_blocks).reshape(n_seq, width_b)
        self.inv_freq = (base ** (-2.0 * np.arange(rot // 2) / max(rot, 1))).astype(np.float32)
        self.pair_axis = rng.integers(0, axes, rot // 2) if axes > 1 else None
        self.positions = rng.integers(-500, 500, (axes, n_tok)) if axes > 1 else None
        self.q_w, self.k_w = (rng.standard_normal((2, hd)) + 1).astype(np.float32) if norm else (None, None)
        self.fmt, self.bs, self.n_kv, self.hd, self.n_q, self.rot = fmt, bs, n_kv, hd, n_q, rot
        self.interleaved, self.gain, self.axes, self.eps = interleaved, gain, axes, 1e-5

    def rotary(self, q_norm, k_norm):
        opt = lambda x, f: None if x is None else f(x)
        return kvq.make_rotary(ELEMENT_TYPES[self.qkv.dtype], self.rot, self.interleaved, dev(self.inv_freq),
                               opt(self.pair_axis, ints), self.axes, opt(q_norm, dev), opt(k_norm, dev), self.eps,
                               self.gain)

    def pool(self):
        return PagedPool(FORMATS[self.fmt], self.n_kv, self.hd, self.bs, self.n_blocks, fill=3)

    def run(self, q=None, q_norm=0, pool=None, stream=None, q_out=None, seq=None, pos=None, table=None):
        pool = self.pool() if pool is None else pool
        out = pool.append_rotary(self.rotary(self.q_w if isinstance(q_norm, int) else q_norm, self.k_w),
                                 self.q if q is None else q, self.k, self.v,
                                 ints(self.seq if seq is None else seq), ints(self.pos if pos is None else pos),
                                 ints(self.table if table is None else table),
                                 None if self.positions is None else ints(self.positions), q_out, stream)
        torch.cuda.synchronize()
        return pool, out

    def check_q(self, out):
        pos = self.pos[None] if self.positions is None else self.positions
        want, size = plain.rotated(self.q.float().cpu().numpy(), pos, self.inv_freq, self.rot, self.interleaved,
                                   self.q_w, self.eps, self.gain, self.pair_axis)
        angle = np.abs(pos).max() * np.abs(self.inv_freq).max() if self.rot else 0.0
        err = np.abs(out.cpu().numpy() - want)
        assert (err <= tolerance(size, angle)).all(), float((err / size).max())

    def check_cache(self, pool, seq=None, pos=None, table=None):
        """The rotated keys come out as q (k's rows and weights given as q's); kvq_append stores them."""
        _, k = self.run(q=self.k, q_norm=self.k_w, seq=seq, pos=pos, table=table)
        want = self.pool()
        want.append(k, self.v.float().contiguous(), ints(self.seq if seq is None else seq),
                    ints(self.pos if pos is None else pos), ints(self.table if table is None else table))
        torch.cuda.synchronize()
        for a, b in ((pool.k, want.k), (pool.v, want.v), (pool.ks, want.ks), (pool.vs, want.vs)):
            if a is not None:
                bits = (lambda t: t.view(torch.int16)) if a.dtype == torch.float16 else (lambda t: t)
                assert torch.equal(bits(a), bits(b))


SHAPES = [  # n_tok, n_q, n_kv, hd, rot, interleaved, axes
    (1, 32, 8, 128, 128, False, 1), (5, 21, 3, 64, 64, False, 1), (67, 16, 1, 256, 256, False, 1),
    (3, 1, 1, 64, 32, True, 1), (33, 7, 7, 128, 32, False, 1), (64, 16, 2, 256, 64, True, 3),
    (129, 5, 5, 64, 16, False, 2), (40, 12, 4, 128, 96, True, 1), (17, 8, 8, 128, 0, False, 1),
    (1025, 4, 2, 128, 128, False, 4), (7, 0, 3, 128, 128, False, 1), (700, 3, 3, 256, 240, False, 1),
]


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("fmt", ["f16", "q8", "k8v4"])
@pytest.mark.parametrize("shape", SHAPES)
def test_shapes(shape, fmt, dtype):
    rng = np.random.default_rng([SHAPES.index(shape), FORMATS[fmt]])
    c = Call(rng, fmt, dtype, *shape, norm=shape[0] % 2 == 1, pad=8 * (shape[0] % 3), gain=1.25 if shape[2] == 2 else 1.0,
             top=2000)
    pool, out = c.run()
    c.check_q(out)
    c.check_cache(pool)


@pytest.mark.parametrize("top", [15, 131071, (1 << 22) + 5, (1 << 24) + 3, (1 << 26) + 12345])
def test_far_positions(top):
    # (blocks of 1024: a long row of the table, a pool of three blocks)
    rng = np.random.default_rng(top)
    c = Call(rng, "f16", torch.float32, 12, 4, 2, 128, 128, False, bs=1024, top=2000)
    c.pos = top - np.arange(12)[::-1]
    c.seq = np.zeros(12, np.int64)
    c.n_blocks = 3
    c.table = np.full((1, top // 1024 + 1), -1)
    c.table[0, max(0, top // 1024 - 1):] = [2, 0][:c.table.shape[1]]
    pool, out = c.run()
    c.check_q(out)
    c.check_cache(pool)


def test_padding_and_broken_places():
    # padding tokens leave q_out and the pool alone; a token without a block
    # gets its q and no cell
    rng = np.random.default_rng(3)
    c = Call(rng, "q8", torch.bfloat16, 9, 4, 2, 128, 128, False, top=100)
    seq, pos, table = c.seq.copy(), c.pos.copy(), c.table.copy()
    seq[1], seq[4], pos[6] = -1, 3, -1
    pos[7] = table.shape[1] * c.bs          # behind the row
    table[seq[2], pos[2] // c.bs] = c.n_blocks
    q_out = torch.full((9, 4, 128), 7.0, device="cuda")
    pool, out = c.run(q_out=q_out, seq=seq, pos=pos, table=table)
    assert out is q_out and (out[[1, 4, 6]] == 7).all()
    c.pos = pos
    keep = torch.tensor([0, 2, 3, 5, 7, 8], device="cuda")
    full, size = plain.rotated(c.q.float().cpu().numpy(), pos[None], c.inv_freq, c.rot, False, c.q_w, c.eps)
    err = np.abs(out.cpu().numpy() - full)[keep.cpu().numpy()]
    assert (err <= tolerance(size, 1e4)[keep.cpu().numpy()]).all()
    c.check_cache(pool, seq, pos, table)


def test_non_finite_heads_stay_alone():
    # NaN or infinity in one head or dim reaches no other head, nor the dims
    # that do not rotate
    rng = np.random.default_rng(4)
    c = Call(rng, "f16", torch.float32, 4, 4, 2, 128, 64, False, norm=False, top=50)
    ref, out0 = c.run()
    c.q[1, 2, 100] = float("inf")
    c.q[2, 3, 5] = float("nan")
    c.k[0, 1, 127] = float("-inf")
    pool, out = c.run()
    changed = ~((out == out0) | (out.isnan() & out0.isnan()))
    assert changed.nonzero().tolist() == [[1, 2, 100], [2, 3, 5], [2, 3, 37]]
    bits = pool.k.view(torch.int16) != ref.k.view(torch.int16)
    assert int(bits.sum()) == 1 and torch.equal(pool.v.view(torch.int16), ref.v.view(torch.int16))


def test_side_stream_and_graph():
    rng = np.random.default_rng(5)
    c = Call(rng, "k8v4", torch.bfloat16, 65, 8, 2, 256, 256, False, top=300)
    pool, want = c.run()
    side = torch.cuda.Stream()
    pool2, got = c.run(stream=side)
    assert torch.equal(got, want) and torch.equal(pool.v, pool2.v)
    # captured: the arrays' later contents count
    pool3, args = c.pool(), (c.rotary(c.q_w, c.k_w), ints(c.seq), ints(c.pos), ints(c.table))
    out = torch.zeros_like(want)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        pool3.append_rotary(args[0], c.q, c.k, c.v, *args[1:], q_out=out)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            pool3.append_rotary(args[0], c.q, c.k, c.v, *args[1:], q_out=out)
    out.zero_()
    for t in (pool3.k, pool3.v):     # (as the other pools began)
        t.fill_(3)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(pool3.v, pool.v) and torch.equal(pool3.k, pool.k)


def test_more_than_2_31_elements_apart():
    # token rows 2^30 elements apart: offsets pass 32 bits (2 GB bf16 rows of one buffer)
    n_tok, n_q, n_kv, hd = 4, 2, 1, 128
    big = torch.zeros(3 * (1 << 30) + 1024, dtype=torch.bfloat16, device="cuda")
    rows = big.as_strided((n_tok, n_q + 2 * n_kv, hd), (1 << 30, hd, 1))
    rows.copy_(torch.randn(n_tok, n_q + 2 * n_kv, hd, device="cuda"))
    r = kvq.make_rotary(kvq.KVQ_T_BF16, hd, False, dev((10.0 ** -np.arange(64.0)).astype(np.float32)))
    outs = []
    for x in (rows, rows.contiguous()):
        pool = PagedPool(kvq.KVQ_F16, n_kv, hd, 16, 2)
        out = pool.append_rotary(r, x[:, :2], x[:, 2:3], x[:, 3:], ints([0] * 4), ints(range(4)), ints([[1, 0]]))
        torch.cuda.synchronize()
        outs.append((out, pool.k.view(torch.int16), pool.v.view(torch.int16)))
    assert all(torch.equal(a, b) for a, b in zip(*outs)) and bool(outs[0][0].any())


def test_methods_refuse():
    rng = np.random.default_rng(6)
    c = Call(rng, "f16", torch.float32, 3, 4, 2, 128, 128, False, top=50)
    pool, r = c.pool(), c.rotary(None, None)
    seq, pos, table = ints(c.seq), ints(c.pos), ints(c.table)
    good = (r, c.q, c.k, c.v, seq, pos, table)
    pool.append_rotary(*good)
    for i, bad in ((1, c.q.half()), (2, c.k[:2]), (2, c.k.transpose(1, 2).contiguous().transpose(1, 2)),
                   (3, c.v.cpu()), (4, seq.long()), (5, pos[:2]), (6, table[0]), (1, c.q[..., :64])):
        with pytest.raises(kvq.KvqError):
            pool.append_rotary(*good[:i], bad, *good[i + 1:])
    with pytest.raises(kvq.KvqError):
        pool.append_rotary(*good, positions=ints(np.zeros((2, 3))))
    with pytest.raises(kvq.KvqError):
        pool.append_rotary(*good, q_out=c.q)     # the input itself
