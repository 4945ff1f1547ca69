"""A serving loop's sequences held on the device: their lengths, block tables
and free list, advanced step by step by kvq_plan_step (include/kvq.h).

This module is argument marshalling: the plan itself runs in the library's
kernel, and nothing is read back to the host unless the caller does so.
"""
from __future__ import annotations

import torch

from . import KvqError, KVQ_ERR_ARG, check, kvq_plan_step, kvq_trim_step
from .pool import on_stream


class StepPlanner:
    """n_seq sequence rows over a pool of n_blocks blocks.

    plan(n_new) leaves the step's arrays in tok_seq, tok_pos, slots
    [max_tok], tok_start [n_seq + 1], ctx_start (the lengths before),
    ctx_lens (the lengths after), block_table and plan_info (tokens, blocks
    handed out, blocks given back, status); the next plan overwrites them.  trim
    writes trim_info; info is that of the last call, plan_info or trim_info.
    The addresses stay the same, so a captured graph may hold whole steps."""

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
        self.plan_info, self.trim_info = ints(4), ints(4)
        self.info = self.plan_info
        self._placed = torch.ones(1, dtype=torch.bool, device=device)   # whether the last plan was
        self._drop = ints(n_seq)

    def _check(self, call: str, **tensors) -> None:
        """Each tensor (None: left out) is a contiguous int32 [n_seq] on the
        planner's device, which is a GPU."""
        dev = self.plan_info.device
        for name, t in tensors.items():
            if t is not None and (t.shape != (self.n_seq,) or t.dtype != torch.int32 or not t.is_contiguous()
                                  or t.device != dev):
                raise KvqError(KVQ_ERR_ARG, f"StepPlanner.{call}: {name} must be a contiguous int32 [n_seq] on {dev}")
        if dev.type != "cuda":
            raise KvqError(KVQ_ERR_ARG, f"StepPlanner.{call}: the planner is on {dev}, not a GPU")

    def plan(self, n_new, stream=None) -> None:
        """n_new int32 [n_seq] on the device: tokens each sequence gets;
        negative: it ends and gives its blocks back.  A step that cannot be
        placed changes nothing and says why in plan_info[3]."""
        self._check("plan", n_new=n_new)
        self.info = self.plan_info
        with torch.cuda.device(self.info.device), on_stream(stream):
            self._before.copy_(self._after)
            check(kvq_plan_step(self.ctx_start, n_new, self.n_seq, self.block_size, self.n_blocks,
                                self.block_table, self.max_blocks, self.free_list, self._count_in,
                                self.max_tok, self.ctx_lens, self.tok_start, self.tok_seq,
                                self.tok_pos, self.slots, self.free_count, self.info, stream),
                  "kvq_plan_step")

    def n_draft(self, out=None, stream=None):
        """verify_draft's n_draft behind a plan whose tokens were each sequence's
        last sampled one and its drafts: int32 [n_seq], the tokens placed less
        one; negative, so that verify_draft passes the sequence over, where it got
        none, ended, or the plan was not placed.  To be read before trim."""
        self._check("n_draft", out=out)
        with torch.cuda.device(self.plan_info.device), on_stream(stream):
            return torch.sub(self.ctx_lens, self.ctx_start, out=out).sub_(1)

    def window_rows(self, W: int, n_tok: int, stream=None):
        """Where the plan's first n_tok tokens, which are packed, stand in arrays
        of W rows a sequence: (attend, verify), int64 [n_tok].  The attention has a
        sequence's tokens in the last rows of its window (row W - 1 is its last
        cell), verify_draft its first in row 0; the two are the same where every
        sequence got W tokens.  Row n_seq * W, behind the arrays, stands for
        padding and for tokens that the window does not reach.  To be read before
        trim."""
        self._check("window_rows")
        if W < 1 or not 0 <= n_tok <= self.max_tok:
            raise KvqError(KVQ_ERR_ARG, f"StepPlanner.window_rows: W = {W}, n_tok = {n_tok} of {self.max_tok}")
        with torch.cuda.device(self.plan_info.device), on_stream(stream):
            seq, pos = self.tok_seq[:n_tok].long(), self.tok_pos[:n_tok]
            none = self.n_seq * W

            def rows(at):
                return torch.where((seq >= 0) & (at >= 0) & (at < W), seq * W + at, none)

            return rows(W + pos - self.ctx_lens[seq]), rows(pos - self.ctx_start[seq])

    def trim(self, n_drop, stream=None) -> None:
        """n_drop int32 [n_seq] on the device: cells taken back from the end of
        each sequence (verify_draft's n_dropped, or more: a rollback).  ctx_lens
        shrink (ctx_start are the lengths before), blocks go back; trim_info:
        cells taken back, 0, blocks given back, status.  The plan's token arrays
        stay as they are.  Behind a plan that could not be placed, whose tokens
        are in no cell, nothing is taken back until another plan is placed."""
        self._check("trim", n_drop=n_drop)
        self.info = self.trim_info
        with torch.cuda.device(self.info.device), on_stream(stream):
            self._before.copy_(self._after)
            torch.eq(self.plan_info[3:], 0, out=self._placed)
            torch.mul(n_drop, self._placed, out=self._drop)
            check(kvq_trim_step(self.ctx_start, self._drop, self.n_seq, self.block_size, self.n_blocks,
                                self.block_table, self.max_blocks, self.free_list, self._count_in,
                                self.ctx_lens, self.free_count, self.info, stream), "kvq_trim_step")
