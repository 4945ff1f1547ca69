"""CPU: what kvq_plan_step, kvq_bound_blocks, kvq_select_blocks and
kvq_sparse_decode_attn refuse before any launch, and their sizes.  As in
test_abi.py each call carries one invalid argument and made-up addresses
that nothing dereferences; skipped on a machine with a GPU."""
import pytest
import torch

import quantized_kv_cache_append_gb300 as kvq

ARG, UNSUPPORTED, WORKSPACE = kvq.KVQ_ERR_ARG, kvq.KVQ_ERR_UNSUPPORTED, kvq.KVQ_ERR_WORKSPACE
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


PLAN = dict(ctx_in=A, n_new=2 * A, n_seq=4, block_size=16, n_blocks=100, block_table=3 * A,
            max_blocks_per_seq=8, free_list=4 * A, free_count_in=5 * A, max_tok=64, ctx_out=6 * A,
            tok_start=7 * A, tok_seq=8 * A, tok_pos=9 * A, slots=10 * A, free_count_out=11 * A, info=12 * A)


@no_gpu_only
@pytest.mark.parametrize("bad,status", [
    (dict(n_seq=0), ARG), (dict(n_blocks=0), ARG), (dict(max_blocks_per_seq=0), ARG), (dict(max_tok=-1), ARG),
    (dict(block_size=48), ARG), (dict(block_size=8), ARG), (dict(block_size=2048), ARG),
    (dict(n_blocks=1 << 27), ARG), (dict(max_blocks_per_seq=1 << 27), ARG),
    *[(dict([(k, None)]), ARG) for k in PLAN if PLAN[k] >= A and k != "slots"],
    (dict(tok_seq=8 * A + 4), ARG), (dict(tok_pos=9 * A + 8), ARG), (dict(slots=10 * A + 4), ARG),
    (dict(info=12 * A + 4), ARG), (dict(ctx_in=A + 2), ARG),
    (dict(ctx_out=A), ARG), (dict(ctx_out=A + 12), ARG), (dict(free_count_out=5 * A), ARG),   # in place
    (dict(tok_pos=8 * A), ARG), (dict(slots=9 * A + 240), ARG), (dict(tok_start=3 * A + 124), ARG),
    (dict(free_list=3 * A), ARG), (dict(n_new=6 * A), ARG), (dict(free_count_in=4 * A + 396), ARG),
    (dict(n_seq=16385), UNSUPPORTED), (dict(max_tok=(1 << 30) + 4, tok_seq=20 * A, tok_pos=40 * A, slots=None),
                                       UNSUPPORTED),
])
def test_plan_step_refuses(bad, status):
    a = dict(PLAN, **bad)
    assert kvq.kvq_plan_step(**a, stream=0) == status


@no_gpu_only
@pytest.mark.parametrize("bad,status", [
    (dict(cache=cache(ks=None)), ARG), (dict(cache=cache(hd=96)), ARG), (dict(n_seq=0), ARG),
    (dict(mbps=0), ARG), (dict(max_new=-1), ARG), (dict(max_new=8 * 64 + 1), ARG), (dict(bt=None), ARG),
    (dict(lens=None), ARG), (dict(bounds=None), ARG), (dict(scales=None), ARG), (dict(bounds=A + 128), ARG),
    (dict(scales=A + 4), ARG), (dict(start=A + 1), ARG), (dict(n_seq=1 << 28), UNSUPPORTED),
])
def test_bound_blocks_refuses(bad, status):
    a = dict(cache=cache(), bt=A, n_seq=4, mbps=8, start=2 * A, lens=3 * A, max_new=100, bounds=4 * A,
             scales=5 * A)
    a.update(bad)
    assert kvq.kvq_bound_blocks(a["cache"], a["bt"], a["n_seq"], a["mbps"], a["start"], a["lens"], a["max_new"],
                                a["bounds"], a["scales"], 0) == status


@no_gpu_only
def test_bound_blocks_without_new_cells_is_a_no_op():
    assert kvq.kvq_bound_blocks(cache(), None, 4, 8, None, None, 0, None, None, 0) == kvq.KVQ_OK


@no_gpu_only
@pytest.mark.parametrize("bad,status", [
    (dict(cache=cache(bs=8)), ARG), (dict(n_seq=0), ARG), (dict(W=0), ARG), (dict(n_q=30), ARG),
    (dict(max_ctx=0), ARG), (dict(max_ctx=16 * 64 + 1), ARG), (dict(n_sel=0), ARG), (dict(n_first=-1), ARG),
    (dict(n_last=-1), ARG), (dict(n_first=5, n_last=4), ARG), (dict(n_first=(1 << 31) - 1, n_last=(1 << 31) - 1), ARG),
    *[(dict([(k, None)]), ARG) for k in ("bounds", "scales", "q", "lens", "bt", "blocks", "out_lens")],
    (dict(bounds=A + 64), ARG), (dict(q=A + 8), ARG), (dict(blocks=A + 2), ARG), (dict(index=A + 2), ARG),
    (dict(n_q=8 * 33), UNSUPPORTED), (dict(n_sel=1 << 25), UNSUPPORTED), (dict(n_seq=1 << 22), UNSUPPORTED),
    (dict(cache=cache(bs=16), mbps=40000, max_ctx=32769 * 16), UNSUPPORTED),
])
def test_select_blocks_refuses(bad, status):
    a = dict(cache=cache(), bounds=A, scales=2 * A, q=3 * A, n_seq=2, W=1, n_q=32, lens=4 * A, max_ctx=1000,
             bt=5 * A, mbps=16, n_sel=8, n_first=1, n_last=2, blocks=6 * A, index=7 * A, out_lens=8 * A)
    a.update(bad)
    assert kvq.kvq_select_blocks(a["cache"], a["bounds"], a["scales"], a["q"], a["n_seq"], a["W"], a["n_q"],
                                 a["lens"], a["max_ctx"], a["bt"], a["mbps"], a["n_sel"], a["n_first"],
                                 a["n_last"], a["blocks"], a["index"], a["out_lens"], 0) == status


@no_gpu_only
@pytest.mark.parametrize("bad,status", [
    (dict(cache=cache(vs=None)), ARG), (dict(n_seq=0), ARG), (dict(W=0), ARG), (dict(n_q=20), ARG),
    (dict(n_sel=0), ARG), (dict(sm=float("nan")), ARG), (dict(sm=float("inf")), ARG),
    *[(dict([(k, None)]), ARG) for k in ("q", "blocks", "lens", "out")],
    (dict(q=A + 4), ARG), (dict(out=A + 8), ARG), (dict(lens=A + 2), ARG), (dict(ws=None), WORKSPACE),
    (dict(ws=A + 16), WORKSPACE), (dict(ws_bytes=64), WORKSPACE), (dict(n_q=8 * 33), UNSUPPORTED),
    (dict(n_seq=1 << 22), UNSUPPORTED), (dict(n_sel=1 << 25), UNSUPPORTED),
])
def test_sparse_decode_refuses(bad, status):
    a = dict(cache=cache(), q=A, n_seq=2, W=1, n_q=32, blocks=2 * A, lens=3 * A, n_sel=8, sm=0.1, out=4 * A,
             ws=5 * A, ws_bytes=1 << 30)
    a.update(bad)
    assert kvq.kvq_sparse_decode_attn(a["cache"], a["q"], a["n_seq"], a["W"], a["n_q"], a["blocks"], a["lens"],
                                      a["n_sel"], a["sm"], a["out"], a["ws"], a["ws_bytes"], 0) == status


def test_sparse_workspace_size():
    c = cache()
    one = kvq.kvq_sparse_workspace_bytes(c, 1, 1, 32, 8)
    assert 0 < one <= kvq.kvq_sparse_workspace_bytes(c, 1, 1, 32, 64)
    # enough lists to fill the SMs meet in clusters and need no partials
    assert kvq.kvq_sparse_workspace_bytes(c, 64, 4, 32, 64) == 256
    for bad in ((0, 1, 32, 8), (1, 0, 32, 8), (1, 1, 30, 8), (1, 1, 32, 0), (1, 1, 8 * 33, 8)):
        assert kvq.kvq_sparse_workspace_bytes(c, *bad) == 0
    assert kvq.kvq_sparse_workspace_bytes(cache(ks=None), 1, 1, 32, 8) == 0
