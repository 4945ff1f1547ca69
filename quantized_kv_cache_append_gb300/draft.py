"""Drafted tokens of a verify window: which of them stand, and the token behind
them (kvq_verify_draft, include/kvq.h).  Argument marshalling only."""
from __future__ import annotations

import torch

from . import KVQ_ERR_ARG, KvqError, check, kvq_verify_draft
from .pool import ELEMENT_TYPES, on_stream


def verify_draft(target, draft, draft_tokens, u, u_sample, n_draft=None, out=None, stream=None):
    """target [n_seq][W][vocab], draft [n_seq][W - 1][vocab] (None: certain
    drafts) probabilities, draft_tokens int32 and u fp32 [n_seq][W - 1],
    u_sample fp32 [n_seq], n_draft int32 [n_seq] -> (n_accepted [n_seq], tokens
    [n_seq][W], n_dropped [n_seq]), int32; out: such a tuple to write.  Rows may
    be wider than vocab (a padded array's view).

    n_draft None says that every sequence of the batch has W - 1 drafts in its
    cache.  Where some have fewer, or take no part in the step (negative), it has
    to be given (StepPlanner.n_draft): n_dropped counts drafts, and a trim by it
    takes that many cells."""
    n_seq, W, vocab = target.shape
    dev = target.device

    def need(ok, what):
        if not ok:
            raise KvqError(KVQ_ERR_ARG, f"verify_draft: {what}")

    def row_stride(t):   # (torch leaves the stride of a dimension of one row open)
        return t.stride(1) if t.shape[1] > 1 else t.stride(0) if n_seq > 1 else vocab

    def whole(name, t, dtype, shape):
        need(t is None or (t.dtype == dtype and tuple(t.shape) == shape and t.is_contiguous() and t.device == dev),
             f"{name} must be a contiguous {dtype} tensor of shape {shape} on {dev}")

    need(dev.type == "cuda", f"the probabilities are on {dev}, not a GPU")
    need(target.dtype in ELEMENT_TYPES, f"probabilities of {target.dtype}")
    for name, t, rows in (("target", target, W), ("draft", draft, W - 1)):
        if t is None or t.numel() == 0:
            continue
        need(t.dtype == target.dtype and tuple(t.shape) == (n_seq, rows, vocab) and t.device == dev
             and (vocab == 1 or t.stride(2) == 1) and (n_seq == 1 or t.stride(0) == rows * row_stride(t)),
             f"{name} must be [{n_seq}][{rows}][{vocab}] of {target.dtype} on {dev}, rows evenly apart")
    whole("draft_tokens", draft_tokens, torch.int32, (n_seq, W - 1))
    whole("u", u, torch.float32, (n_seq, W - 1))
    whole("u_sample", u_sample, torch.float32, (n_seq,))
    whole("n_draft", n_draft, torch.int32, (n_seq,))
    with torch.cuda.device(dev), on_stream(stream):
        if out is None:
            new = lambda *s: torch.empty(s, dtype=torch.int32, device=dev)
            out = (new(n_seq), new(n_seq, W), new(n_seq))
        for name, t, shape in zip(("n_accepted", "tokens", "n_dropped"), out, ((n_seq,), (n_seq, W), (n_seq,))):
            whole(name, t, torch.int32, shape)
        has_draft = draft is not None and draft.numel() > 0
        check(kvq_verify_draft(target, draft if has_draft else None, ELEMENT_TYPES[target.dtype],
                               row_stride(target), row_stride(draft) if has_draft else vocab, n_seq, W, vocab,
                               draft_tokens, n_draft, u, u_sample, *out, stream), "kvq_verify_draft")
    return out
