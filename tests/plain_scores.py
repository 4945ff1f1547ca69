"""Attention with capped, biased and masked scores in 64-bit floats, written
from the definition at kvq_scores in include/kvq.h, and the error fp32 may
leave."""
from __future__ import annotations

import numpy as np


def rows(q, k, v, places, pos, low, high, sm_scale, cap=0.0, slopes=None, p_step=2.0 ** -22,
         code=None, top=2.0 ** 8, dot=2.0 ** -18, sums=64):
    """One KV head: q [T][G][hd] at positions pos [T]; k, v [n][hd], cells
    `places` [n]; low, high [T] first and last cell seen; slopes [G] ->
    (out [T][G][hd], tolerance [T][G][hd]).

    Tolerance.  A score's error dz (natural-log units): q enters as fp16 hi +
    lo and is summed in fp32, below `dot` of sm_scale * sum |q k|
    (plain_blocks.attention: hd / 16 <= 16 steps at 2^-23); the tanh's argument, value and product with the
    cap below 2^-19 of the capped score (its approximation 2^-21, the rest half
    steps; the slope of the tanh is at most 1); slope * log2(e), distance and
    their fma below 2^-22 of the bias; the log2 domain's own roundings 2^-22 of
    the score.  The output moves by at most sum p dz |v| + |o| sum p dz.  p
    itself: 2^-21 of the exponential and p_step of its rounding; the sum over
    the cells in fp32, n / sums steps at 2^-23 of sum p |v|.

    code: the largest |v| in the units that meet p in the tensor core (int8
    and K8V4 fold the scale into p: 127 and 8; FP16: the values).  p's lo half
    is fp16, so its rounding is at least half of fp16's smallest step, 2^-25,
    whatever p is; where the row's largest p is `top` (2^8, or 1 where a scale
    is above 128) that is n * 2^-25 * code / top in the output."""
    T, G, hd = q.shape
    out, tol = np.zeros((T, G, hd)), np.zeros((T, G, hd))
    k, v = k.astype(np.float64), v.astype(np.float64)
    for t in range(T):
        seen = (places >= low[t]) & (places <= high[t])
        if not seen.any():
            continue
        ks, vs, d = k[seen], v[seen], np.abs(pos[t] - places[seen])
        Q = q[t].astype(np.float64)
        z = sm_scale * (Q @ ks.T)
        dz = dot * abs(sm_scale) * (np.abs(Q) @ np.abs(ks).T)
        if cap:
            z = cap * np.tanh(z / cap)
            dz = dz + 2.0 ** -19 * np.abs(z)
        if slopes is not None:
            bias = slopes.astype(np.float64)[:, None] * d
            z = z - bias
            dz = dz + 2.0 ** -22 * np.abs(bias)
        dz = dz + 2.0 ** -22 * np.abs(z)
        p = np.exp(z - z.max(1, keepdims=True))
        p /= p.sum(1, keepdims=True)
        o = p @ vs
        out[t] = o
        tol[t] = ((p * dz) @ np.abs(vs) + np.abs(o) * (p * dz).sum(1, keepdims=True)
                  + (2.0 ** -20 + p_step + (seen.sum() / sums + 32) * 2.0 ** -23) * (p @ np.abs(vs)) + 1e-30
                  + len(ks) * 2.0 ** -25 * (np.abs(vs).max() if code is None else code) / top)
    return out, tol


def decode(K, V, q, ctx, table, bs, sm_scale, cap=0.0, window=0, slopes=None, first=None, rotated=None, code=None,
           top=2.0 ** 8):
    """K, V [n_blocks][n_kv][bs][hd] (plain_blocks.pool_rows) -> (out, tolerance);
    rotated: the matrix that takes K8V4's values back (a mean of hd terms: the
    largest dim's tolerance, and as much again for its fp32 sums)."""
    n_seq, W, n_q, hd = q.shape
    n_kv = K.shape[1]
    G = n_q // n_kv
    out, tol = np.zeros(q.shape), np.zeros(q.shape)
    for b in range(n_seq):
        L = int(np.clip(ctx[b], 0, table.shape[1] * bs))
        cell = np.arange(L)
        ids = table[b, cell // bs]
        cell = cell[(ids >= 0) & (ids < len(K))]
        ids = table[b, cell // bs]
        pos = L - W + np.arange(W)
        low = np.zeros(W, np.int64) + (0 if first is None else int(first[b]))
        if window:
            low = np.maximum(low, pos - window + 1)
        for h in range(n_kv):
            s = slice(h * G, (h + 1) * G)
            o, e = rows(q[b, :, s], K[ids, h, cell % bs], V[ids, h, cell % bs], cell, pos, low, pos, sm_scale, cap,
                        None if slopes is None else slopes[s], code=code, top=top)
            if rotated is not None:
                o, e = o @ rotated / hd, np.broadcast_to(2 * e.max(-1, keepdims=True), e.shape)
            out[b, :, s], tol[b, :, s] = o, e
    return out, tol


def chunk(k16, v16, q, sm_scale, cap=0.0, window=0, slopes=None, first=None, last=None, out_step=0.0):
    """k16, v16 [n_kv][P][hd], q [T][n_q][hd] -> (out, tolerance).  Sums of hi and
    lo halves in turn: 2 hd / 16 <= 32 steps at 2^-23 and q's 2^-22, below
    2^-17; p is one fp16 value (2^-11; its reference maximum is at most the
    row's, so the largest p is at least 1), 16 cells a step of the fp32 sum;
    out_step: half a step of the output type."""
    n_kv, P, hd = k16.shape
    T, n_q, _ = q.shape
    G = n_q // n_kv
    pos = P - T + np.arange(T)
    low, high = np.zeros(T, np.int64), pos
    if first is not None:
        low = np.maximum(first, 0)
    if window:
        low = np.maximum(low, pos - window + 1)
    if last is not None:
        high = np.minimum(np.maximum(pos, last), P - 1)
    out, tol = np.zeros(q.shape), np.zeros(q.shape)
    for h in range(n_kv):
        s = slice(h * G, (h + 1) * G)
        out[:, s], tol[:, s] = rows(q[:, s], k16[h], v16[h], np.arange(P), pos, low, high, sm_scale, cap,
                                    None if slopes is None else slopes[s], 2.0 ** -11, top=1.0, dot=2.0 ** -17,
                                    sums=16)
    return out, tol + out_step * (np.abs(out) + tol) + (2.0 ** -25 if out_step else 0)
