"""CPU: what kvq_append_rotary, kvq_verify_draft and kvq_trim_step refuse
before any launch.  As in test_abi.py each call carries one invalid argument
and made-up addresses that nothing dereferences; skipped on a machine with a
GPU.  The Python methods refuse host memory with the binding's own error."""
import pytest
import torch

import quantized_kv_cache_append_gb300 as kvq
from quantized_kv_cache_append_gb300.draft import verify_draft
from quantized_kv_cache_append_gb300.pool import PagedPool
from quantized_kv_cache_append_gb300.steps import StepPlanner

ARG, UNSUPPORTED = kvq.KVQ_ERR_ARG, kvq.KVQ_ERR_UNSUPPORTED
A = 1 << 32          # aligned stand-in addresses, far apart


@pytest.fixture(scope="module", autouse=True)
def _library():
    kvq.build()
    kvq.load_library()


no_gpu_only = pytest.mark.skipif(torch.cuda.is_available(), reason="made-up addresses")


def cache(**kw):
    a = dict(fmt=kvq.KVQ_Q8, n_kv=8, hd=128, bs=64, nb=100, k=A, v=2 * A, ks=3 * A, vs=4 * A)
    a.update(kw)
    return kvq.make_cache(a["fmt"], a["n_kv"], a["hd"], a["bs"], a["nb"], a["k"], a["v"], a["ks"], a["vs"])


ROTARY = dict(type=kvq.KVQ_T_BF16, rot_dim=128, interleaved=0, inv_freq=20 * A, pair_axis=21 * A, n_axes=1,
              q_norm=22 * A, k_norm=23 * A, eps=1e-6, gain=1.0)
CALL = dict(cache=cache(), q=5 * A, k=6 * A, v=7 * A, qs=6144, ks=6144, vs=6144, n_tok=10, n_q=32, seq=8 * A,
            pos=9 * A, positions=None, bt=10 * A, n_seq=4, mbps=8, out=11 * A)


def append(rotary, a):
    return kvq.kvq_append_rotary(a["cache"], rotary, a["q"], a["k"], a["v"], a["qs"], a["ks"], a["vs"], a["n_tok"],
                                 a["n_q"], a["seq"], a["pos"], a["positions"], a["bt"], a["n_seq"], a["mbps"],
                                 a["out"], 0)


@no_gpu_only
@pytest.mark.parametrize("bad", [
    dict(type=3), dict(type=-1), dict(rot_dim=-16), dict(rot_dim=144), dict(rot_dim=24), dict(interleaved=2),
    dict(n_axes=0), dict(n_axes=9), dict(n_axes=2), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")),
    dict(gain=float("nan")), dict(gain=float("inf")), dict(inv_freq=None), dict(inv_freq=A + 4),
    dict(pair_axis=A + 2), dict(q_norm=A + 8), dict(k_norm=A + 4),
])
def test_rotary_settings_refused(bad):
    assert append(kvq.make_rotary(**dict(ROTARY, **bad)), CALL) == ARG


@no_gpu_only
@pytest.mark.parametrize("bad,status", [
    (dict(cache=cache(ks=None)), ARG), (dict(cache=cache(hd=96)), ARG), (dict(n_tok=-1), ARG), (dict(n_q=-1), ARG),
    *[(dict([(k, None)]), ARG) for k in ("q", "k", "v", "seq", "pos", "bt", "out")],
    (dict(q=5 * A + 8), ARG), (dict(k=6 * A + 2), ARG), (dict(v=7 * A + 4), ARG), (dict(out=11 * A + 4), ARG),
    (dict(seq=8 * A + 2), ARG), (dict(positions=A + 1), ARG), (dict(qs=4095), ARG), (dict(qs=6148), ARG),
    (dict(ks=1016), ARG), (dict(ks=6145), ARG), (dict(vs=0), ARG), (dict(n_seq=0), ARG), (dict(mbps=0), ARG),
    (dict(out=5 * A), ARG), (dict(out=6 * A + 1024), ARG), (dict(out=7 * A - 4096), ARG),
    (dict(ks=(1 << 31) + 8), UNSUPPORTED), (dict(n_tok=1 << 26), UNSUPPORTED),
])
def test_append_rotary_refuses(bad, status):
    assert append(kvq.make_rotary(**ROTARY), dict(CALL, **bad)) == status


@no_gpu_only
def test_no_tokens_is_a_no_op():
    a = dict(CALL, n_tok=0, q=None, k=None, v=None, seq=None, pos=None, bt=None, out=None)
    assert append(kvq.make_rotary(**ROTARY), a) == kvq.KVQ_OK


VERIFY = dict(target=A, draft=2 * A, type=kvq.KVQ_T_F32, target_stride=1000, draft_stride=1000, n_seq=4, W=3,
              vocab=1000, draft_tokens=3 * A, n_draft=4 * A, u=5 * A, u_sample=6 * A, n_accepted=7 * A,
              tokens=8 * A, n_dropped=9 * A)


@no_gpu_only
@pytest.mark.parametrize("bad,status", [
    (dict(type=5), ARG), (dict(n_seq=0), ARG), (dict(W=0), ARG), (dict(vocab=0), ARG),
    *[(dict([(k, None)]), ARG) for k in ("target", "draft_tokens", "u", "u_sample", "n_accepted", "tokens")],
    (dict(target=A + 2), ARG), (dict(draft=A + 1), ARG), (dict(u=A + 2), ARG), (dict(tokens=A + 2), ARG),
    (dict(target_stride=999), ARG), (dict(draft_stride=10), ARG),
    (dict(tokens=A + 4000), ARG), (dict(n_accepted=2 * A + 8), ARG), (dict(n_dropped=3 * A), ARG),
    (dict(n_dropped=8 * A + 44), ARG), (dict(tokens=6 * A - 44), ARG),
    (dict(W=33), UNSUPPORTED), (dict(n_seq=65535 * 8 + 1), UNSUPPORTED),
    (dict(vocab=(1 << 20) + 1, target_stride=1 << 21, draft_stride=1 << 21), UNSUPPORTED),
    (dict(target_stride=1 << 32), UNSUPPORTED),
])
def test_verify_draft_refuses(bad, status):
    assert kvq.kvq_verify_draft(**dict(VERIFY, **bad), stream=0) == status


TRIM = dict(ctx_in=A, n_drop=2 * A, n_seq=4, block_size=16, n_blocks=100, block_table=3 * A, max_blocks_per_seq=8,
            free_list=4 * A, free_count_in=5 * A, ctx_out=6 * A, free_count_out=7 * A, info=8 * A)


@no_gpu_only
@pytest.mark.parametrize("bad,status", [
    (dict(n_seq=0), ARG), (dict(n_blocks=0), ARG), (dict(max_blocks_per_seq=0), ARG), (dict(block_size=8), ARG),
    (dict(block_size=100), ARG), (dict(n_blocks=1 << 27), ARG), (dict(max_blocks_per_seq=1 << 27), ARG),
    *[(dict([(k, None)]), ARG) for k in TRIM if TRIM[k] >= A],
    (dict(info=8 * A + 4), ARG), (dict(ctx_in=A + 1), ARG), (dict(ctx_out=A), ARG), (dict(ctx_out=2 * A + 12), ARG),
    (dict(free_count_out=5 * A), ARG), (dict(free_list=3 * A), ARG), (dict(info=6 * A), ARG),
    (dict(n_seq=16385), UNSUPPORTED),
])
def test_trim_step_refuses(bad, status):
    assert kvq.kvq_trim_step(**dict(TRIM, **bad), stream=0) == status


def test_methods_refuse_host_memory():
    i32, f32 = torch.int32, torch.float32
    p = PagedPool(kvq.KVQ_Q8, 1, 64, 16, 4, device="cpu")
    r = kvq.make_rotary(kvq.KVQ_T_F32, 64, False, torch.zeros(32))
    x, one = torch.zeros(2, 1, 64), torch.zeros(2, dtype=i32)
    for call in (lambda: p.append_rotary(r, x, x, x, one, one, torch.zeros(1, 4, dtype=i32)),
                 lambda: p.append_rotary(r, x.half(), x.half(), x.half(), one, one, torch.zeros(1, 4, dtype=i32)),
                 lambda: verify_draft(torch.zeros(2, 2, 5), None, torch.zeros(2, 1, dtype=i32), torch.zeros(2, 1),
                                      torch.zeros(2, dtype=f32)),
                 lambda: StepPlanner(2, 4, 16, 8, 16, device="cpu").trim(one)):
        with pytest.raises(kvq.KvqError):
            call()
