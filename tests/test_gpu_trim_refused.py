"""GPU: a trim behind a plan that was refused takes nothing back, and the plan's
status stays to be seen."""
import numpy as np
import pytest
import torch

import quantized_kv_cache_append_gb300 as kvq
from quantized_kv_cache_append_gb300.steps import StepPlanner
from tests.test_gpu_plan_step import dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _library():
    if not torch.cuda.is_available():
        pytest.fail("the GPU suite needs a CUDA device")
    kvq.build()
    kvq.load_library()


def full():
    """Lengths 30 and 32 on 4 blocks of 16 cells: no block is free."""
    p = StepPlanner(2, 8, 16, 4, 100)
    p.plan(dev([30, 32]))
    torch.cuda.synchronize()
    assert p.ctx_lens.tolist() == [30, 32] and p.free_count.tolist() == [0] and p.info.tolist() == [62, 4, 0, 0]
    return p


def held(p):
    table, lens = p.block_table.cpu().numpy(), p.ctx_lens.cpu().numpy()
    ids = [x for b in range(p.n_seq) for x in table[b, :-(-lens[b] // p.block_size)]]
    return sorted(ids + list(p.free_list[:int(p.free_count[0])].cpu().numpy()))


def test_a_refused_plan_loses_no_cells():
    p = full()
    for _ in range(2):
        p.plan(dev([3, 3]))
        for drop in ([3, 3], [1, 0], [30, 32]):
            p.trim(dev(drop))
            torch.cuda.synchronize()
            assert p.ctx_lens.tolist() == [30, 32] and p.free_count.tolist() == [0] and held(p) == [0, 1, 2, 3]
            assert p.plan_info[3] != 0 and p.info.tolist() == [0, 0, 0, 0]
    # (a broken trim says so, whatever the plan was)
    p.trim(dev([-1, 0]))
    torch.cuda.synchronize()
    assert p.ctx_lens.tolist() == [30, 32] and p.plan_info[3] != 0


@pytest.mark.parametrize("why,new", [("blocks", [3, 3]), ("tokens", [50, 51]), ("row", [99, 0])])
def test_whatever_refused_it_and_a_placed_plan_ends_it(why, new):
    p = full()
    p.plan(dev(new))
    p.trim(dev([2, 2]))
    torch.cuda.synchronize()
    assert p.ctx_lens.tolist() == [30, 32] and p.plan_info[3] != 0
    p.plan(dev([0, -1]))
    torch.cuda.synchronize()
    assert p.info.data_ptr() == p.plan_info.data_ptr() and p.info.tolist() == [0, 0, 2, 0]
    p.trim(dev([15, 0]))
    torch.cuda.synchronize()
    assert p.ctx_start.tolist() == [30, 0] and p.ctx_lens.tolist() == [15, 0] and p.free_count.tolist() == [3]
    assert p.info.tolist() == [15, 0, 1, 0] and p.plan_info.tolist() == [0, 0, 2, 0] and held(p) == [0, 1, 2, 3]


def test_a_captured_step_whose_plan_is_refused():
    p = full()
    new, drop = dev([0, 0]), dev([0, 0])
    p.plan(new)
    p.trim(drop)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        p.plan(new)
        p.trim(drop)
    lens = np.array([30, 32])
    # refused, placed (a sequence's cells within its last block), refused, one ends, placed
    for n, d, after in (([3, 3], [2, 2], [30, 32]), ([2, 0], [1, 0], [31, 32]), ([1, 1], [1, 1], [31, 32]),
                        ([1, -1], [0, 0], [32, 0]), ([4, 4], [3, 4], [33, 0])):
        new.copy_(dev(n))
        drop.copy_(dev(d))
        g.replay()
        torch.cuda.synchronize()
        refused = list(after) == list(lens)
        assert p.ctx_lens.tolist() == after and bool(p.plan_info[3] != 0) == refused
        assert p.info[0] == (0 if refused else sum(d))
        assert held(p) == [0, 1, 2, 3]
        lens = np.array(after)


def test_other_streams():
    p = full()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    new, drop = dev([3, 3]), dev([3, 3])
    torch.cuda.synchronize()
    p.plan(new, stream=side)
    p.trim(drop, stream=side)
    side.synchronize()
    assert p.ctx_lens.tolist() == [30, 32]
