"""CPU: what the scored attention calls refuse before any launch (made-up
addresses, as in test_abi.py; skipped on a machine with a GPU)."""
import pytest
import torch

import quantized_kv_cache_append_gb300 as kvq

ARG, UNSUPPORTED, WORKSPACE = kvq.KVQ_ERR_ARG, kvq.KVQ_ERR_UNSUPPORTED, kvq.KVQ_ERR_WORKSPACE
A = 1 << 32


@pytest.fixture(scope="module", autouse=True)
def _library():
    kvq.build()
    kvq.load_library()


no_gpu_only = pytest.mark.skipif(torch.cuda.is_available(), reason="made-up addresses")


def cache(**kw):
    a = dict(fmt=kvq.KVQ_Q8, n_kv=8, hd=128, bs=64, nb=100, k=A, v=2 * A, ks=3 * A, vs=4 * A)
    a.update(kw)
    return kvq.make_cache(a["fmt"], a["n_kv"], a["hd"], a["bs"], a["nb"], a["k"], a["v"], a["ks"], a["vs"])


BAD_SCORES = [dict(softcap=-1.0), dict(softcap=float("nan")), dict(softcap=float("inf")), dict(softcap=1e-4),
              dict(softcap=2e6), dict(window=-1), dict(slopes=A + 2), dict(first=A + 1), dict(last=A + 3)]


def decode(scores, **bad):
    a = dict(cache=cache(), q=A, n_seq=2, W=2, n_q=32, lens=2 * A, max_ctx=1000, bt=3 * A, mbps=16, sm=0.1, out=4 * A,
             ws=5 * A, ws_bytes=1 << 30)
    a.update(bad)
    return kvq.kvq_decode_attn_scored(a["cache"], scores, a["q"], a["n_seq"], a["W"], a["n_q"], a["lens"], a["max_ctx"],
                                      a["bt"], a["mbps"], a["sm"], a["out"], a["ws"], a["ws_bytes"], 0)


@no_gpu_only
@pytest.mark.parametrize("bad", BAD_SCORES + [dict(last=A)])
def test_decode_refuses_scores(bad):
    assert decode(kvq.make_scores(**bad)) == ARG
    assert kvq.kvq_scored_workspace_bytes(cache(), kvq.make_scores(**bad), 2, 2, 32, 1000) == 0


@no_gpu_only
@pytest.mark.parametrize("bad,status", [
    (dict(cache=cache(vs=None)), ARG), (dict(n_seq=0), ARG), (dict(W=0), ARG), (dict(W=17), ARG), (dict(n_q=20), ARG),
    (dict(max_ctx=1), ARG), (dict(max_ctx=16 * 64 + 1), ARG), (dict(sm=float("nan")), ARG),
    *[(dict([(k, None)]), ARG) for k in ("q", "lens", "bt", "out")], (dict(q=A + 4), ARG), (dict(out=A + 8), ARG),
    (dict(ws=None), WORKSPACE), (dict(ws=A + 16), WORKSPACE), (dict(ws_bytes=64), WORKSPACE),
    (dict(n_q=8 * 17), UNSUPPORTED),
])
def test_decode_refuses(bad, status):
    assert decode(kvq.make_scores(softcap=30.0, window=100, slopes=A, first=A), **bad) == status


def test_workspace_sizes():
    whole = kvq.kvq_scored_workspace_bytes(cache(), kvq.make_scores(), 1, 1, 32, 6400)
    window = kvq.kvq_scored_workspace_bytes(cache(), kvq.make_scores(window=64), 1, 1, 32, 6400)
    assert 0 < window < whole
    assert kvq.kvq_scored_workspace_bytes(cache(), kvq.make_scores(window=6400), 1, 1, 32, 6400) == whole
    for bad in ((0, 1, 32, 100), (1, 0, 32, 100), (1, 1, 30, 100), (1, 1, 32, 0), (1, 1, 8 * 33, 100)):
        assert kvq.kvq_scored_workspace_bytes(cache(), kvq.make_scores(), *bad) == 0


def chunk(scores, **bad):
    a = dict(k=A, v=2 * A, n_kv=8, P=1000, hd=128, q=3 * A, T=100, n_q=32, sm=0.1, out=4 * A, type=kvq.KVQ_T_BF16)
    a.update(bad)
    return kvq.kvq_chunk_attn_scored(a["k"], a["v"], a["n_kv"], a["P"], a["hd"], scores, a["q"], a["T"], a["n_q"],
                                     a["sm"], a["out"], a["type"], 0)


@no_gpu_only
@pytest.mark.parametrize("bad", BAD_SCORES)
def test_chunk_refuses_scores(bad):
    assert chunk(kvq.make_scores(**bad)) == ARG


@no_gpu_only
@pytest.mark.parametrize("bad,status", [
    *[(dict([(k, None)]), ARG) for k in ("k", "v", "q", "out")], (dict(k=A + 8), ARG), (dict(out=4 * A + 8), ARG),
    (dict(type=3), ARG), (dict(type=-1), ARG), (dict(P=0), ARG), (dict(T=0), ARG), (dict(T=1001), ARG),
    (dict(n_q=30), ARG), (dict(n_kv=0), ARG), (dict(sm=float("inf")), ARG), (dict(hd=96), UNSUPPORTED),
    (dict(P=1 << 28), UNSUPPORTED),
])
def test_chunk_refuses(bad, status):
    assert chunk(kvq.make_scores(softcap=30.0, window=100, slopes=A, first=A, last=A), **bad) == status
