"""PagedPool.chunk_scored: what it refuses before any launch (CPU, the call
itself replaced by one that counts), and that it is the call (GPU)."""
import contextlib

import pytest
import torch

import quantized_kv_cache_append_gb300 as kvq
from quantized_kv_cache_append_gb300 import pool as pool_module
from quantized_kv_cache_append_gb300.pool import PagedPool

N_KV, HD, P, T, N_Q = 2, 64, 40, 9, 4
I32 = torch.int32


def arrays(device="cpu"):
    g = torch.Generator().manual_seed(1)
    mk = lambda *s: torch.randn(s, generator=g)
    return dict(k16=mk(N_KV, P, HD).half().to(device), v16=mk(N_KV, P, HD).half().to(device), q=mk(T, N_Q, HD).to(device))


def settings(device="cpu"):
    return dict(softcap=20.0, window=30, slopes=torch.full((N_Q,), 0.1, device=device),
                first=torch.full((T,), 3, dtype=I32, device=device), last=torch.full((T,), 36, dtype=I32, device=device))


@pytest.fixture
def call(monkeypatch):
    launched = []
    monkeypatch.setattr(pool_module, "kvq_chunk_attn_scored", lambda *a, **k: launched.append(a) or 0)
    monkeypatch.setattr(PagedPool, "_on", lambda self, stream: contextlib.nullcontext())
    pool = PagedPool(kvq.KVQ_Q8, N_KV, HD, 16, 4, device="cpu")

    def run(scores=None, **kw):
        a = dict(arrays(), out=None)
        a.update(kw)
        before = len(launched)
        try:
            return pool.chunk_scored(a["k16"], a["v16"], a["q"], 0.1, kvq.make_scores(**dict(settings(), **(scores or {}))),
                                     out=a["out"], out_dtype=a.get("out_dtype", torch.float32))
        finally:
            run.launches = len(launched) - before
    return run


def test_good_calls(call):
    assert call().dtype == torch.float32 and call.launches == 1
    assert call(out_dtype=torch.bfloat16).shape == (T, N_Q, HD)
    out = torch.zeros(T, N_Q, HD, dtype=torch.float16)
    assert call(out=out) is out and call.launches == 1
    call(scores=dict(slopes=None, first=1 << 32, last=None))
    assert call.launches == 1


@pytest.mark.parametrize("bad", [
    dict(k16=torch.zeros(N_KV, P, HD)), dict(v16=torch.zeros(N_KV, P - 1, HD).half()),
    dict(v16=torch.zeros(P, N_KV, HD).half().transpose(0, 1)), dict(k16=torch.zeros(1, P, HD).half()),
    dict(q=torch.zeros(T, N_Q, HD).half()), dict(q=torch.zeros(T, N_Q, 128)), dict(q=torch.zeros(T, N_Q, HD, device="meta")),
    dict(out=torch.zeros(T, N_Q, HD, dtype=torch.float64)), dict(out=torch.zeros(T + 1, N_Q, HD)),
    dict(out=torch.zeros(N_Q, T, HD).transpose(0, 1)), dict(out_dtype=torch.int8),
    dict(scores=dict(slopes=torch.zeros(N_Q, dtype=torch.float16))), dict(scores=dict(slopes=torch.zeros(N_KV))),
    dict(scores=dict(first=torch.zeros(T, dtype=torch.int64))), dict(scores=dict(first=torch.zeros(1, dtype=I32))),
    dict(scores=dict(last=torch.zeros(T, device="meta", dtype=I32))), dict(scores=dict(last=torch.zeros(2 * T, dtype=I32)[::2])),
])
def test_refused(call, bad):
    with pytest.raises(kvq.KvqError):
        call(**bad)
    assert call.launches == 0


def test_host_pool_refused():
    pool = PagedPool(kvq.KVQ_Q8, N_KV, HD, 16, 4, device="cpu")
    with pytest.raises(kvq.KvqError):
        pool.chunk_scored(*arrays().values(), 0.1, kvq.make_scores())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,code", [(torch.float32, kvq.KVQ_T_F32), (torch.float16, kvq.KVQ_T_F16),
                                        (torch.bfloat16, kvq.KVQ_T_BF16)])
def test_it_is_the_call(dtype, code):
    kvq.build()
    kvq.load_library()
    a, pool = arrays("cuda"), PagedPool(kvq.KVQ_F16, N_KV, HD, 16, 4)
    scores = kvq.make_scores(**settings("cuda"))
    want = torch.empty(T, N_Q, HD, dtype=dtype, device="cuda")
    kvq.check(kvq.kvq_chunk_attn_scored(a["k16"], a["v16"], N_KV, P, HD, scores, a["q"], T, N_Q, 0.1, want, code))
    got = pool.chunk_scored(a["k16"], a["v16"], a["q"], 0.1, scores, out_dtype=dtype)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = torch.zeros_like(want)
    torch.cuda.synchronize()
    assert pool.chunk_scored(a["k16"], a["v16"], a["q"], 0.1, scores, out=out, stream=side) is out
    torch.cuda.synchronize()
    assert torch.equal(got, want) and torch.equal(out, want) and bool(want.any())
