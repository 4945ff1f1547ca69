"""CPU: how the score that kvq_select_blocks ranks blocks by relates to the
bound of q . k it stands for.  The bounds' part is exact; q enters as 8-bit
codes, so a score lies beside the bound of the unrounded q, above or below, by
at most half a code step of every dim times the larger bound."""
import numpy as np
import pytest

from tests import plain_blocks as plain


def pool_bounds(rng, n, bs, hd):
    gain = np.ones(hd)
    gain[rng.choice(hd, 4, replace=False)] = 6.0             # a few channels far larger, as keys have
    K = ((rng.standard_normal((n, bs, hd)) + 0.5 * rng.standard_normal((n, 1, hd))) * gain).astype(np.float16)
    codes, scales = np.zeros((n, 2, hd), np.int8), np.zeros((n, hd // 64), np.float32)
    for j in range(n):
        codes[j], scales[j] = plain.bounds_of(K[j].astype(np.float64))
    return K, codes, scales


def exact_bounds(codes, scales, q):
    """The bounds with the unrounded q, and how far a score may lie from them:
    [blocks][rows] each."""
    step = np.repeat(scales.astype(np.float64), 64, -1)
    lo, hi = codes[:, 0] * step, codes[:, 1] * step
    q = q.astype(np.float64)
    f = np.array([[plain.scale_of(np.abs(r[g:g + 64]).max(), -60, 60) for g in range(0, len(r), 64)] for r in q])
    most = np.maximum(np.abs(lo), np.abs(hi))
    off = most @ (0.5 * np.repeat(f, 64, -1)).T
    sums = most @ (np.abs(q) + 0.5 * np.repeat(f, 64, -1)).T   # two fp32 additions at most
    return np.maximum(q, 0) @ hi.T + np.minimum(q, 0) @ lo.T, (off + 2 * 2.0 ** -24 * sums).T


def queries(rng, G, hd, large):
    gain = np.ones(hd)
    gain[rng.choice(hd, 2, replace=False)] = large
    return (rng.standard_normal((G, hd)) * gain).astype(np.float32)


@pytest.mark.parametrize("hd,G,n,bs", [(64, 1, 200, 16), (128, 4, 300, 64), (256, 8, 150, 32)])
@pytest.mark.parametrize("large", [1.0, 30.0])
def test_a_score_is_the_bound_of_the_rounded_query(hd, G, n, bs, large):
    rng = np.random.default_rng(hd + n)
    K, codes, scales = pool_bounds(rng, n, bs, hd)
    q = queries(rng, G, hd, large)
    got = plain.scores(codes, scales, q)
    assert np.array_equal(got, [max(plain.score(codes[j], scales[j], r) for r in q) for j in range(n)])
    # the bound with the unrounded q is one
    exact, off = exact_bounds(codes, scales, q)
    logits = np.einsum("gd,ncd->gnc", q.astype(np.float64), K.astype(np.float64)).max(2)
    assert (logits <= exact * (1 + 1e-12) + 1e-12).all()
    # the score lies within the rounding of q of it
    exact = exact.max(0)
    assert (np.abs(got - exact) <= off.max(0)).all()
    # so a block that the rounding moves in or out of a list lies that close to
    # the list's border
    k = n // 8
    border = np.sort(exact)[-k]
    ours, theirs = (set(np.lexsort((np.arange(n), -s))[:k]) for s in (got, exact))
    for j in ours ^ theirs:
        assert abs(exact[j] - border) <= 2 * off.max()


def test_a_score_may_lie_below_a_logit():
    # one large dim and 63 below half a code step: those are lost
    q = np.full((1, 64), 0.49, np.float32)
    q[0, 0] = 127
    k = np.ones((1, 64))
    codes, scales = plain.bounds_of(k)
    score = plain.scores(codes[None], scales[None], q)[0]
    assert score == 127 and (q.astype(np.float64) @ k[0])[0] > 157
