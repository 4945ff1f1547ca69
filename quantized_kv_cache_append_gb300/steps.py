"""A serving loop's sequences held on the device: their lengths, block tables
and free list, advanced step by step by kvq_plan_step (include/kvq.h).

This module is argument marshalling: the plan itself runs in the library's
kernel, and nothing is read back to the host unless the caller does so.
"""
from __future__ import annotations

import torch

from . import KvqError, KVQ_ERR_ARG, check, kvq_plan_step
from .pool import on_stream


class StepPlanner:
    """n_seq sequence rows over a pool of n_blocks blocks.

    plan(n_new) leaves the step's arrays in tok_seq, tok_pos, slots
    [max_tok], tok_start [n_seq + 1], ctx_start (the lengths before),
    ctx_lens (the lengths after), block_table and info (tokens, blocks handed
    out, blocks given back, status); the next plan overwrites them.  The
    addresses stay the same, so a captured graph may hold whole steps."""

    def __init__(self, n_seq: int, max_blocks: int, block_size: int, n_blocks: int, max_tok: int,
                 device="cuda"):
        self.n_seq, self.max_blocks, self.block_size = n_seq, max_blocks, block_size
        self.n_blocks, self.max_tok = n_blocks, max_tok

        def ints(*shape, fill=0):
            return torch.full(shape, fill, dtype=torch.int32, device=device)

        # lengths and free count: what a step reads, and what it writes
        before, after = ints(n_seq + 1), ints(n_seq + 1)
        before[n_seq] = after[n_seq] = n_blocks
        self._before, self._after = before, after
        self.ctx_start, self._count_in = before[:n_seq], before[n_seq:]
        self.ctx_lens, self.free_count = after[:n_seq], after[n_seq:]
        self.block_table = ints(n_seq, max_blocks, fill=-1)
        self.free_list = torch.arange(n_blocks - 1, -1, -1, dtype=torch.int32, device=device)
        self.tok_start = ints(n_seq + 1)
        self.tok_seq, self.tok_pos, self.slots = (ints(max_tok, fill=-1) for _ in range(3))
        self.info = ints(4)

    def plan(self, n_new, stream=None) -> None:
        """n_new int32 [n_seq] on the device: tokens each sequence gets;
        negative: it ends and gives its blocks back.  A step that cannot be
        placed changes nothing and says why in info[3]."""
        if (n_new.shape != (self.n_seq,) or n_new.dtype != torch.int32 or not n_new.is_contiguous()
                or n_new.device != self.info.device):
            raise KvqError(KVQ_ERR_ARG, "StepPlanner.plan: n_new must be a contiguous int32 [n_seq] on "
                                        f"{self.info.device}")
        if self.info.device.type != "cuda":
            raise KvqError(KVQ_ERR_ARG, f"StepPlanner.plan: the planner is on {self.info.device}, not a GPU")
        with torch.cuda.device(self.info.device), on_stream(stream):
            self._before.copy_(self._after)
            check(kvq_plan_step(self.ctx_start, n_new, self.n_seq, self.block_size, self.n_blocks,
                                self.block_table, self.max_blocks, self.free_list, self._count_in,
                                self.max_tok, self.ctx_lens, self.tok_start, self.tok_seq,
                                self.tok_pos, self.slots, self.free_count, self.info, stream),
                  "kvq_plan_step")
