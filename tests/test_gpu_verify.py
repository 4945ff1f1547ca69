"""GPU: kvq_verify_draft against the definition (tests/plain_draft.py), every
output equal."""
import numpy as np
import pytest
import torch

import quantized_kv_cache_append_gb300 as kvq
from quantized_kv_cache_append_gb300.draft import verify_draft
from tests import plain_draft as plain

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _library():
    if not torch.cuda.is_available():
        pytest.fail("the GPU suite needs a CUDA device")
    kvq.build()
    kvq.load_library()


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def draws(rng, n, W, V, dtype, spread=2.0, pad=0):
    """Probabilities, drafts sampled from theirs, random numbers; rows V + pad apart."""
    lt = rng.standard_normal((n, W, V)) * spread
    ld = lt[:, :W - 1] + rng.standard_normal((n, W - 1, V)) * 0.5
    soft = lambda x: np.exp(x - x.max(-1, keepdims=True)) / np.exp(x - x.max(-1, keepdims=True)).sum(-1, keepdims=True)
    pt, pd = soft(lt), soft(ld) if W > 1 else ld
    tok = (np.cumsum(pd, -1) < rng.random((n, W - 1, 1))).sum(-1).clip(0, V - 1) if W > 1 else np.zeros((n, 0))

    def rows(x):
        wide = np.full((*x.shape[:2], V + pad), np.nan, np.float32)
        wide[..., :V] = x
        return dev(wide).to(dtype)[..., :V]
    return dict(target=rows(pt), draft=rows(pd), tok=tok.astype(np.int32), u=rng.random((n, W - 1)).astype(np.float32),
                us=rng.random(n).astype(np.float32), nd=rng.integers(-1, W + 1, n).astype(np.int32))


def check(d, certain=False, nd=True, stream=None):
    out = verify_draft(d["target"], None if certain else d["draft"], dev(d["tok"]), dev(d["u"]), dev(d["us"]),
                       dev(d["nd"]) if nd else None, stream=stream)
    torch.cuda.synchronize()
    want = plain.verify(d["target"].float().cpu().numpy(), None if certain else d["draft"].float().cpu().numpy(),
                        d["tok"], d["nd"] if nd else None, d["u"], d["us"])
    for name, a, b in zip(("accepted", "tokens", "dropped"), out, want):
        assert np.array_equal(a.cpu().numpy(), b), name
    return want


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("n,W,V,pad", [
    (1, 1, 1, 0), (1, 2, 2, 0), (3, 4, 31, 0), (5, 2, 1023, 0), (2, 8, 1024, 0), (7, 3, 1025, 7), (16, 4, 32000, 0),
    (40, 3, 4096, 8), (200, 5, 2050, 6), (3, 32, 3000, 0), (2, 3, 131075, 0), (1, 6, 1 << 20, 0), (700, 2, 40, 0),
])
def test_sizes(n, W, V, pad, dtype):
    rng = np.random.default_rng([n, W, V])
    d = draws(rng, n, W, V, dtype, pad=pad)
    check(d)
    check(d, certain=True)
    check(d, nd=False)


def test_every_place_of_a_row():
    # u_sample just below, at and above each boundary of known weights, in every tile
    V = 2500
    w = np.zeros(V, np.float32)
    at = np.array([0, 1, 31, 32, 1023, 1024, 1055, 2047, 2048, 2499])
    w[at] = 2.0 ** -np.array([3, 3, 3, 3, 3, 4, 4, 4, 4, 3])
    total = w.sum(dtype=np.float64)
    edges = np.cumsum(w[at].astype(np.float64)) / total
    us = np.clip(np.concatenate([edges, edges - 2.0 ** -24, edges + 2.0 ** -24, [0, 1 - 2.0 ** -24]]), 0, 1 - 2.0 ** -24)
    n = len(us)
    d = dict(target=dev(np.tile(w, (n, 1, 1))), tok=np.zeros((n, 0), np.int32), u=np.zeros((n, 0), np.float32),
             us=us.astype(np.float32), nd=None)
    got = check(d, certain=True, nd=False)
    assert set(got[1][:, 0]) == set(at)


@pytest.mark.parametrize("case", ["equal", "zero", "nan", "above_one", "tiny", "outside", "one_token", "u_edges"])
def test_corners(case):
    rng = np.random.default_rng(9)
    d = draws(rng, 24, 4, 1500, torch.float32)
    d["nd"][:] = 3
    t, q = d["target"], d["draft"]
    if case == "equal":        # nothing above 0 in the difference: the target itself
        q.copy_(t[:, :3])
        d["u"][:] = 1 - 2.0 ** -24
        q[:, 0] = torch.maximum(q[:, 0] * 2, torch.tensor(1e-30))
        d["u"][:, 0] = 0.75
    if case == "zero":         # a target row that leaves nothing: token -1
        t[::2] = 0
    if case == "nan":
        t[:, :, ::5] = float("nan")
        q[:, :, ::7] = float("nan")
        t[:, :, 3] = -1.0
    if case == "above_one":
        t[:, :, 100:200] = 3.0
        t[:, :, 300] = float("inf")
    if case == "tiny":         # below one unit, and around it
        t.fill_(2.0 ** -41)
        t[:, :, 700] = 2.0 ** -40
        t[:, :, 900] = 2.0 ** -39 - 2.0 ** -63
    if case == "outside":
        d["tok"][:, 1] = [-1, 1500, 2 ** 31 - 1] * 8
    if case == "one_token":    # the whole row on the rejected token
        t.zero_()
        t[:, :, 77] = 1.0
        d["tok"][:] = 77
        d["u"][:] = 1.0        # (outside [0, 1): 1 < 1 is false)
    if case == "u_edges":
        d["us"][:6] = [0, 1, 2, -1, np.nan, 1 - 2.0 ** -24]
        d["u"][:6] = [[0, 0, 0], [1, 1, 1], [np.nan, 0, 0], [-1, 0, 0], [0, np.nan, 0], [0, 0, 1]]
    for certain in (False, True):
        got = check(d, certain)
        if case == "zero":
            assert (got[1][::2, 0] == -1).all()
        if case == "one_token" and certain:
            assert (got[1][:, 0] == 77).all()


def test_distribution():
    # accepted or resampled, the first token is distributed as the target's: 40000 trials over
    # 6 tokens, each count within 6 standard deviations
    rng = np.random.default_rng(11)
    n, V = 40000, 6
    p, q = np.array([.3, .05, .25, .2, .15, .05]), np.array([.1, .3, .2, .05, .05, .3])
    d = dict(target=dev(np.tile(p.astype(np.float32), (n, 2, 1))), draft=dev(np.tile(q.astype(np.float32), (n, 1, 1))),
             tok=rng.choice(V, (n, 1), p=q).astype(np.int32), u=rng.random((n, 1)).astype(np.float32),
             us=rng.random(n).astype(np.float32), nd=None)
    got = check(d, nd=False)
    counts = np.bincount(got[1][:, 0], minlength=V)
    assert (np.abs(counts - n * p) <= 6 * np.sqrt(n * p * (1 - p))).all(), counts


def test_streams_graphs_and_repeats():
    rng = np.random.default_rng(12)
    d = draws(rng, 30, 4, 50000, torch.bfloat16)
    want = check(d)
    check(d, stream=torch.cuda.Stream())
    a = (d["target"], d["draft"], dev(d["tok"]), dev(d["u"]), dev(d["us"]), dev(d["nd"]))
    out = verify_draft(*a)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        verify_draft(*a, out=out)
    for _ in range(3):
        for t in out:
            t.fill_(99)
        g.replay()
        torch.cuda.synchronize()
        assert all(np.array_equal(x.cpu().numpy(), y) for x, y in zip(out, want))


def test_method_refuses():
    rng = np.random.default_rng(13)
    d = draws(rng, 4, 3, 100, torch.float32)
    good = dict(target=d["target"], draft=d["draft"], draft_tokens=dev(d["tok"]), u=dev(d["u"]), u_sample=dev(d["us"]),
                n_draft=dev(d["nd"]))
    verify_draft(**good)
    for bad in (dict(target=d["target"].double()), dict(draft=d["draft"].half()), dict(draft=d["draft"][:, :1]),
                dict(draft_tokens=dev(d["tok"]).long()), dict(u=dev(d["u"])[:, :1]), dict(u_sample=dev(d["us"])[:2]),
                dict(n_draft=dev(d["nd"]).cpu()), dict(target=d["target"].transpose(1, 2).contiguous().transpose(1, 2)),
                dict(target=d["target"][:1].expand(4, 3, 100))):
        with pytest.raises(kvq.KvqError):
            verify_draft(**dict(good, **bad))
