"""CPU: the block-selecting methods refuse pools and planners that no GPU holds,
with the binding's own error."""
import pytest
import torch

import quantized_kv_cache_append_gb300 as kvq
from quantized_kv_cache_append_gb300.pool import BlockBounds, PagedPool
from quantized_kv_cache_append_gb300.steps import StepPlanner


def ints(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def test_pools_and_planners_in_host_memory_are_refused():
    kvq.build()
    p = PagedPool(kvq.KVQ_Q8, 1, 64, 16, 4, device="cpu")
    bounds, q = BlockBounds(p), torch.zeros(1, 1, 4, 64)
    for call in (lambda: p.bound(bounds, ints(1, 3), ints(1), 16),
                 lambda: p.select(bounds, q, ints(1), 16, ints(1, 3), 2),
                 lambda: p.decode_selected(q, ints(1, 1, 1, 2), ints(1, 1, 1), 0.1),
                 lambda: StepPlanner(2, 4, 16, 8, 16, device="cpu").plan(ints(2))):
        with pytest.raises(kvq.KvqError):
            call()
