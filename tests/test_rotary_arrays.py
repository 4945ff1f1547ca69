"""CPU: PagedPool.append_rotary looks at the arrays inside its `rotary` before
any launch (the call itself is replaced by one that counts)."""
import contextlib

import pytest
import torch

import quantized_kv_cache_append_gb300 as kvq
from quantized_kv_cache_append_gb300 import pool as pool_module
from quantized_kv_cache_append_gb300.pool import PagedPool

HD = 64


@pytest.fixture
def call(monkeypatch):
    launched = []
    monkeypatch.setattr(pool_module, "kvq_append_rotary", lambda *a, **k: launched.append(a) or 0)
    monkeypatch.setattr(PagedPool, "_on", lambda self, stream: contextlib.nullcontext())
    p = PagedPool(kvq.KVQ_Q8, 1, HD, 16, 4, device="cpu")
    x, one = torch.zeros(2, 1, HD), torch.zeros(2, dtype=torch.int32)

    def run(rot_dim=32, n_axes=2, **arrays):
        a = dict(inv_freq=torch.zeros(rot_dim // 2), pair_axis=torch.zeros(rot_dim // 2, dtype=torch.int32),
                 q_norm=torch.ones(HD), k_norm=torch.ones(HD))
        a.update(arrays)
        r = kvq.make_rotary(kvq.KVQ_T_F32, rot_dim, False, n_axes=n_axes, **a)
        before = len(launched)
        try:
            p.append_rotary(r, x, x, x, one, one, torch.zeros(1, 4, dtype=torch.int32),
                            positions=torch.zeros(n_axes, 2, dtype=torch.int32))
        finally:
            run.launches = len(launched) - before
    return run


def test_good_arrays(call):
    call()
    assert call.launches == 1
    call(pair_axis=None, q_norm=None, k_norm=None)
    assert call.launches == 1
    call(rot_dim=0, inv_freq=None, pair_axis=None)
    assert call.launches == 1
    call(inv_freq=1 << 32, pair_axis=1 << 33, q_norm=1 << 34, k_norm=None)     # raw addresses: the caller's word
    assert call.launches == 1


@pytest.mark.parametrize("bad", [
    dict(q_norm=torch.ones(HD, dtype=torch.bfloat16)), dict(k_norm=torch.ones(HD, dtype=torch.float16)),
    dict(q_norm=torch.ones(HD // 2)), dict(k_norm=torch.ones(1, HD)), dict(k_norm=torch.ones(2 * HD)[::2]),
    dict(inv_freq=torch.zeros(16, dtype=torch.float64)), dict(inv_freq=torch.zeros(15)), dict(inv_freq=torch.zeros(32)),
    dict(inv_freq=torch.zeros(16, device="meta")), dict(pair_axis=torch.zeros(16, dtype=torch.int64)),
    dict(pair_axis=torch.zeros(8, dtype=torch.int32)), dict(q_norm=torch.ones(HD, device="meta")),
])
def test_bad_arrays_are_refused(call, bad):
    with pytest.raises(kvq.KvqError, match=next(iter(bad))):
        call(**bad)
    assert call.launches == 0
