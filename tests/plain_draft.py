"""Plain numpy forms of a speculative decoding step's calls, in whole numbers
and 64-bit floats, written from the definitions in include/kvq.h: norm and
rotation, draft verification, trimming."""
from __future__ import annotations

import math

import numpy as np

ROW, LIST = 2, 8


def rotated(x, pos, inv_freq, rot_dim, interleaved, weight=None, eps=0.0, gain=1.0, pair_axis=None):
    """x [n][heads][hd], pos [axes][n] -> (values, their pair's |a| + |b| before the rotation)."""
    x = x.astype(np.float64)
    if weight is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + float(np.float32(eps))) * weight.astype(np.float64)
    out, size = x.copy(), np.abs(x)
    for i in range(rot_dim // 2):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot_dim // 2)
        axis = 0 if pair_axis is None else min(max(int(pair_axis[i]), 0), len(pos) - 1)
        t = pos[axis].astype(np.float64) * float(inv_freq[i])
        c, s = (np.cos(t) * gain)[:, None], (np.sin(t) * gain)[:, None]
        out[..., a], out[..., b] = x[..., a] * c - x[..., b] * s, x[..., b] * c + x[..., a] * s
        size[..., a] = size[..., b] = (np.abs(x[..., a]) + np.abs(x[..., b])) * abs(gain)
    return out, size


def units(r):
    """floor(r * 2^40), r in fp32 held in [0, 1], NaN as 0."""
    r = np.asarray(r, np.float32).astype(np.float64)
    return np.floor(np.clip(np.where(np.isnan(r), 0, r), 0, 1) * 2.0 ** 40).astype(np.int64)


def verify(target, draft, draft_tokens, n_draft, u, u_sample):
    """float32 arrays (16-bit types widened) -> (accepted, tokens, dropped)."""
    n, W, V = target.shape
    accepted, tokens, dropped = np.zeros(n, np.int32), np.full((n, W), -1, np.int32), np.zeros(n, np.int32)
    for b in range(n):
        nd = W - 1 if n_draft is None else min(int(n_draft[b]), W - 1)
        if nd < 0:
            continue
        a = 0
        while a < nd:
            x = int(draft_tokens[b, a])
            if not 0 <= x < V:
                break
            q = 1.0 if draft is None else float(draft[b, a, x])
            if not float(u[b, a]) * q < float(target[b, a, x]):
                break
            tokens[b, a] = x
            a += 1
        p = target[b, a]
        w = units(p)
        if a < nd:
            if draft is None:
                w = w.copy()
                if 0 <= int(draft_tokens[b, a]) < V:
                    w[int(draft_tokens[b, a])] = 0
            else:
                with np.errstate(invalid="ignore"):
                    w = units(p - draft[b, a])
            if not w.any():
                w = units(p)
        S = int(w.sum())
        us = float(u_sample[b])
        U = 0 if math.isnan(us) else int(min(max(math.floor(us * 2 ** 24), 0), 2 ** 24 - 1))
        if S:
            tokens[b, a] = int(np.searchsorted(np.cumsum(w), S * U >> 24, side="right"))
        accepted[b], dropped[b] = a, nd - a
    return accepted, tokens, dropped


def trim(ctx, drop, table, free, count, bs, n_blocks):
    """One trim; returns a dict of every output (inputs unchanged)."""
    width = table.shape[1]
    ctx, drop, free = [int(x) for x in ctx], [int(x) for x in drop], free.copy()
    ceil = lambda x: -(-x // bs)
    bad = [c < 0 or d < 0 or d > c or c > width * bs for c, d in zip(ctx, drop)]
    back = [int(x) for b, (c, d) in enumerate(zip(ctx, drop)) if not bad[b] for x in table[b, ceil(c - d):ceil(c)]]
    status = (ROW if any(bad) else 0) + (LIST if count < 0 or count + len(back) > n_blocks else 0)
    if status:
        return dict(ctx_out=np.array(ctx, np.int32), free_count_out=count, free_list=free,
                    info=np.array([0, 0, 0, status], np.int32))
    free[count:count + len(back)] = back
    return dict(ctx_out=np.array(ctx, np.int32) - np.array(drop, np.int32), free_count_out=count + len(back),
                free_list=free, info=np.array([sum(drop), 0, len(back), 0], np.int32))
