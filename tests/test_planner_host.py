"""CPU: a planner on host memory refuses every call with the binding's own error."""
import pytest
import torch

import quantized_kv_cache_append_gb300 as kvq
from quantized_kv_cache_append_gb300.steps import StepPlanner


@pytest.mark.parametrize("call", [lambda p, x: p.plan(x), lambda p, x: p.trim(x), lambda p, x: p.n_draft(),
                                  lambda p, x: p.n_draft(out=x), lambda p, x: p.window_rows(2, 4)])
def test_refused(call):
    with pytest.raises(kvq.KvqError):
        call(StepPlanner(2, 4, 16, 8, 16, device="cpu"), torch.zeros(2, dtype=torch.int32))
