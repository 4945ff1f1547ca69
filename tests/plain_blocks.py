"""Plain numpy forms of the block-selecting decode step, in whole numbers and
64-bit floats, written from the definitions in include/kvq.h: step planning,
key bounds, block selection, attention over block lists."""
from __future__ import annotations

import math

import numpy as np

TOKENS, ROW, BLOCKS, LIST = 1, 2, 4, 8


def plan(ctx, n_new, table, free, count, bs, n_blocks, max_tok):
    """One step; returns a dict of every output (inputs unchanged)."""
    n, width = table.shape
    ctx, n_new = [int(x) for x in ctx], [int(x) for x in n_new]
    table, free = table.copy(), free.copy()
    ceil = lambda x: -(-x // bs)
    tokens = sum(max(x, 0) for c, x in zip(ctx, n_new) if c >= 0)
    back = sum(ceil(c) for c, x in zip(ctx, n_new) if x < 0 and c >= 0)
    grow = sum(ceil(c + x) - ceil(c) for c, x in zip(ctx, n_new) if x >= 0 and c >= 0)
    status = 0
    if tokens > max_tok:
        status += TOKENS
    if any(c < 0 or c + max(x, 0) > width * bs for c, x in zip(ctx, n_new)):
        status += ROW
    if grow > count + back:
        status += BLOCKS
    if count < 0 or count + back > n_blocks:
        status += LIST
    none = np.full(max_tok, -1, np.int32)
    out = dict(ctx_out=np.array(ctx, np.int32), tok_start=np.zeros(n + 1, np.int32),
               tok_seq=none.copy(), tok_pos=none.copy(), slots=none.copy(), block_table=table,
               free_list=free, free_count_out=count, info=np.array([0, 0, 0, status], np.int32))
    if status:
        return out
    stack = [int(x) for x in free[:count]]
    for b in range(n):
        if n_new[b] < 0:
            stack += [int(x) for x in table[b, :ceil(ctx[b])]]
    top = stack[count:]
    at = 0
    for b in range(n):
        out["tok_start"][b] = at
        if n_new[b] < 0:
            out["ctx_out"][b] = 0
            continue
        end = ctx[b] + n_new[b]
        for c in range(ceil(ctx[b]), ceil(end)):
            table[b, c] = stack.pop()
        for p in range(ctx[b], end):
            out["tok_seq"][at], out["tok_pos"][at] = b, p
            out["slots"][at] = table[b, p // bs] * bs + p % bs
            at += 1
        out["ctx_out"][b] = end
    out["tok_start"][n] = at
    if len(stack) > count:
        free[count:len(stack)] = top[:len(stack) - count]
    out["free_count_out"] = len(stack)
    out["info"] = np.array([tokens, grow, back, 0], np.int32)
    return out


def scale_of(m, lowest, highest):
    """2^e, the smallest e in [lowest, highest] with 127 * 2^e >= m."""
    e = lowest
    while e < highest and 127 * 2.0 ** e < m:
        e += 1
    return 2.0 ** e


def bounds_of(rows):
    """rows [cells][hd] float64 (one block, one KV head) -> codes [2][hd], scales."""
    hd = rows.shape[1]
    codes, scales = np.zeros((2, hd), np.int8), np.zeros(hd // 64, np.float32)
    for g in range(hd // 64):
        x = rows[:, 64 * g:64 * g + 64]
        lo = np.where(np.isnan(x), np.inf, x).min(0)
        hi = np.where(np.isnan(x), -np.inf, x).max(0)
        empty = np.isnan(x).all(0)
        lo[empty] = hi[empty] = 0
        s = scale_of(max(np.abs(lo).max(), np.abs(hi).max()), -24, 16)
        codes[0, 64 * g:64 * g + 64] = np.clip(np.floor(lo / s), -127, 127)
        codes[1, 64 * g:64 * g + 64] = np.clip(np.ceil(hi / s), -127, 127)
        scales[g] = s
    return codes, scales


def score(codes, scales, q):
    """Score of one block for one query row q [hd] (fp32 where the definition says so)."""
    t = []
    for g in range(len(q) // 64):
        x = np.nan_to_num(q[64 * g:64 * g + 64].astype(np.float64), nan=0.0, posinf=np.inf, neginf=-np.inf)
        f = scale_of(np.abs(x).max(), -60, 60)
        c = np.clip(np.rint(x / f), -127, 127).astype(np.int64)
        lo, hi = (codes[k, 64 * g:64 * g + 64].astype(np.int64) for k in (0, 1))
        S = int((np.maximum(c, 0) * hi + np.minimum(c, 0) * lo).sum())
        t.append(np.float32(S * f * float(scales[g])))
    if len(t) == 4:
        t = [np.float32(t[0] + t[1]), np.float32(t[2] + t[3])]
    return t[0] if len(t) == 1 else np.float32(t[0] + t[1])


def scores(codes, scales, q):
    """codes [n][2][hd], scales [n][hd/64], q [G][hd] -> [n], the largest over q's rows."""
    G, hd = q.shape
    total = None
    parts = []
    for g in range(hd // 64):
        x = np.where(np.isnan(q[:, 64 * g:64 * g + 64]), 0.0, q[:, 64 * g:64 * g + 64].astype(np.float64))
        f = np.array([scale_of(np.abs(r).max(), -60, 60) for r in x])
        c = np.clip(np.rint(x / f[:, None]), -127, 127).astype(np.int64)
        lo, hi = (codes[:, k, 64 * g:64 * g + 64].astype(np.int64) for k in (0, 1))
        S = hi @ np.maximum(c, 0).T + lo @ np.minimum(c, 0).T           # [n][G]
        parts.append((S * f * scales[:, g].astype(np.float64)[:, None]).astype(np.float32))
    if len(parts) == 4:
        parts = [parts[0] + parts[1], parts[2] + parts[3]]
    total = parts[0] if len(parts) == 1 else parts[0] + parts[1]
    return total.max(1)


def select(codes, scales, q, ctx, table, bs, n_blocks, n_sel, n_first, n_last):
    """Lists of every (sequence, token, KV head): blocks, indexes, cells."""
    n_seq, W, n_q, hd = q.shape
    n_kv = codes.shape[1]
    G = n_q // n_kv
    blocks = np.full((n_seq, W, n_kv, n_sel), -1, np.int32)
    index, lens = blocks.copy(), np.zeros((n_seq, W, n_kv), np.int32)
    for b in range(n_seq):
        for w in range(W):
            cells = max(0, min(int(ctx[b]), table.shape[1] * bs) - W + w + 1)
            nb = -(-cells // bs)
            ids = table[b, :nb]
            ok = np.nonzero((ids >= 0) & (ids < n_blocks))[0]
            for h in range(n_kv):
                if not len(ok):
                    continue
                s = scores(codes[ids[ok], h], scales[ids[ok], h], q[b, w, h * G:(h + 1) * G]).astype(np.float64)
                s[(ok < n_first) | (ok >= nb - n_last)] = np.inf
                best = np.sort(ok[np.lexsort((ok, -s))[:n_sel]])
                index[b, w, h, :len(best)] = best
                blocks[b, w, h, :len(best)] = ids[best]
                lens[b, w, h] = len(best) * bs - ((nb * bs - cells) if len(best) and best[-1] == nb - 1 else 0)
    return blocks, index, lens


def hadamard(n):
    h = np.ones((1, 1))
    while len(h) < n:
        h = np.block([[h, h], [h, -h]])
    return h


def pool_rows(fmt, k, v, ks, vs):
    """A pool's arrays -> dequantised keys and values, float64 (k8v4's values
    in the rotated basis)."""
    if fmt == "f16":
        return k.astype(np.float64), v.astype(np.float64)
    K = k.astype(np.float64) * np.repeat(ks.astype(np.float64), 64, -1)
    if fmt == "q8":
        return K, v.astype(np.float64) * np.repeat(vs.astype(np.float64), 64, -1)
    codes = np.stack([v & 15, v >> 4], -1).reshape(*v.shape[:-1], -1).astype(np.float64) - 8
    return K, codes * np.repeat(vs.astype(np.float64), 32, -1)


def attention(fmt, K, V, q, sel_blocks, sel_lens, bs, sm_scale):
    """K, V [n_blocks][n_kv][bs][hd] of pool_rows; returns (out, tolerance),
    tolerance [n_seq][W][n_q] the largest error fp32 sums of fp16 hi + lo
    products may leave (see below)."""
    n_seq, W, n_q, hd = q.shape
    n_kv = K.shape[1]
    G = n_q // n_kv
    out = np.zeros(q.shape)
    tol = np.zeros(q.shape[:3])
    n_blocks = K.shape[0]
    for b in range(n_seq):
        for w in range(W):
            for h in range(n_kv):
                n = int(np.clip(sel_lens[b, w, h], 0, sel_blocks.shape[-1] * bs))
                ids = np.repeat(sel_blocks[b, w, h], bs)[:n]
                slot = (np.arange(n) % bs)
                live = (ids >= 0) & (ids < n_blocks)
                if not live.any():
                    continue
                k, v = K[ids[live], h, slot[live]], V[ids[live], h, slot[live]]
                Q = q[b, w, h * G:(h + 1) * G].astype(np.float64)
                z = sm_scale * (Q @ k.T)
                p = np.exp(z - z.max(1, keepdims=True))
                p /= p.sum(1, keepdims=True)
                o = p @ v
                # Logit: q enters as fp16 hi + lo (2^-22 relative, half a step
                # of lo) and is summed in fp32 in hd / 16 <= 16 steps, each
                # off by at most 2^-23 of the partial sum of |q k|: together
                # below 2^-18 of it, in natural-log units.  p carries that
                # (twice: itself and the sum it is divided by), 2^-21 of the
                # exponential, 2^-22 of its own hi + lo halves; the sum over
                # the cells runs in steps of 16 cells of one warp in fp32,
                # n / 64 steps at 2^-23 of the sum of p |v|.
                dz = 2.0 ** -18 * sm_scale * (np.abs(Q) @ np.abs(k).T).max(1)
                spread = (p @ np.abs(v)).max(1)
                err = (2 * dz + 2.0 ** -20 + (n / 64 + 32) * 2.0 ** -23) * spread
                if fmt == "k8v4":   # rotated back: a sum of hd values, / hd, in fp32
                    o = o @ hadamard(hd) / hd
                    err = err + 2.0 ** -20 * spread
                out[b, w, h * G:(h + 1) * G] = o
                tol[b, w, h * G:(h + 1) * G] = err
    return out, tol
