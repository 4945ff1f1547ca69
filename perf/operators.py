"""The block-selecting decode step over the paged K/V cache, operator by operator:
cases, plain forms in torch, and the definitions in 64 bits.

    plan    block tables and slot maps of one step from the request lengths
    bound   bounds of each cache block's keys (int8 codes, power-of-two scales)
    select  the blocks each query token and KV head attends to, by those bounds
    attend  decode attention over each (token, KV head)'s own block list

`run` computes the plain form, or, with `own` set, calls the library.
"""
import math

import numpy as np
import torch

own = False

F16, Q8, K8V4 = 0, 1, 2          # the library's cache formats
GROUP = 64                       # dims per bound scale, and per int8 cache scale
FORMATS = {"f16": F16, "q8": Q8, "k8v4": K8V4}


def listed():
    return [
        # one decode token for each of 64 running requests: what every step pays
        dict(name="plan_step", op="plan", n_seq=64, bs=256, max_blocks=64, lo=1024, hi=16383,
             new=1, mixed=False, max_tok=64),
        # a prefill server's step: 700 requests, most of them prompts, some decoding, idle or
        # finished (their blocks go back), tokens padded to a fixed capacity
        dict(name="plan_prompts", op="plan", n_seq=700, bs=16, max_blocks=1024, lo=0, hi=8001,
             new=4096, mixed=True, max_tok=1000003),
        # after a decode step's append: the newest block of 16 ragged requests
        dict(name="bound_step_f16", op="bound", fmt="f16", n_seq=16, n_kv=8, hd=128, bs=256,
             lo=1024, hi=16384, new=1),
        # after a prompt chunk's append into an int8 cache
        dict(name="bound_chunk_q8", op="bound", fmt="q8", n_seq=1, n_kv=8, hd=128, bs=64,
             lo=131072, hi=131072, new=4096),
        # a whole long prompt, FP16, few wide heads
        dict(name="bound_prompt_f16", op="bound", fmt="f16", n_seq=1, n_kv=2, hd=256, bs=256,
             lo=262144, hi=262144, new=262144),
        # one request's decode token over 32768 cells
        dict(name="select_gqa32k", op="select", n_seq=1, W=1, n_kv=8, G=4, hd=128, bs=64,
             lo=32768, hi=32768, n_sel=64, n_first=1, n_last=2),
        # a 4-token verify window over 131072 cells, small blocks
        dict(name="select_verify", op="select", n_seq=1, W=4, n_kv=8, G=4, hd=128, bs=32,
             lo=131072, hi=131072, n_sel=256, n_first=1, n_last=4),
        # a batch of 64 ragged long requests
        dict(name="select_batch", op="select", n_seq=64, W=1, n_kv=8, G=4, hd=128, bs=32,
             lo=4099, hi=131072, n_sel=128, n_first=1, n_last=4),
        # the attention of one request's decode token over 64 chosen blocks
        dict(name="attend_gqa32k_f16", op="attend", fmt="f16", n_seq=1, W=1, n_kv=8, G=4, hd=128,
             bs=64, lo=32768, hi=32768, n_sel=64),
        # 16 ragged requests on an int8 cache, lists of up to 4096 cells
        dict(name="attend_ragged_q8", op="attend", fmt="q8", n_seq=16, W=1, n_kv=8, G=4, hd=128,
             bs=64, lo=1024, hi=16384, n_sel=64),
        # a verify window over small blocks, rotated 4-bit values, wide heads
        dict(name="attend_verify_k8v4", op="attend", fmt="k8v4", n_seq=1, W=4, n_kv=2, G=8, hd=256,
             bs=16, lo=65536, hi=65536, n_sel=509),
        # a full serving batch, FP16
        dict(name="attend_batch_f16", op="attend", fmt="f16", n_seq=64, W=1, n_kv=8, G=4, hd=128,
             bs=32, lo=4099, hi=32768, n_sel=128),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["plan", "bound", "select", "attend"])
    if op == "plan":
        bs = rng.choice([16, 32, 64, 128, 256])
        n_seq, new = _log_int(rng, 1, 1500), _log_int(rng, 1, 4000)
        hi = _log_int(rng, 1, 16000)
        mixed = rng.random() < 0.6
        tokens = n_seq * new
        if tokens > 1400000:
            new = max(1, 1400000 // n_seq)
            tokens = n_seq * new
        return dict(op=op, n_seq=n_seq, bs=bs, max_blocks=(hi + new) // bs + 1 + rng.randrange(3),
                    lo=rng.randrange(hi), hi=hi, new=new, mixed=mixed,
                    max_tok=tokens + rng.randrange(1 + tokens // 8))
    n_kv, G, hd = rng.choice([(8, 4, 128), (2, 8, 256), (1, 4, 128), (4, 1, 64), (3, 7, 64),
                              (5, 3, 128), (8, 2, 64), (1, 16, 256)])
    bs = rng.choice([16, 32, 64, 128, 256])
    if op == "bound":
        fmt = rng.choice(["f16", "q8", "k8v4"])
        n_seq = _log_int(rng, 1, 48)
        hi = _log_int(rng, 1, min(131072, 131072 * 1024 // (n_seq * n_kv * hd)))
        lo = rng.randrange(1, hi + 1)
        return dict(op=op, fmt=fmt, n_seq=n_seq, n_kv=n_kv, hd=hd, bs=bs, lo=lo, hi=hi,
                    new=1 if rng.random() < 0.3 else _log_int(rng, 1, hi))
    W = rng.choice([w for w in (1, 1, 1, 2, 3, 4) if w * G <= 32])
    n_seq = _log_int(rng, 1, 64)
    hi = max(W, bs, _log_int(rng, 1, 262144))
    if op == "select":
        hi = max(W, min(hi, 64 * 8 * 2112 * 128 * 4 // (n_seq * n_kv * hd * W * G) * bs))
        n_blocks = (hi + bs - 1) // bs
        first, last = rng.randrange(3), rng.randrange(5)
        return dict(op=op, n_seq=n_seq, W=W, n_kv=n_kv, G=G, hd=hd, bs=bs, lo=rng.randrange(W, hi + 1),
                    hi=hi, n_sel=max(1, first + last, _log_int(rng, 1, min(n_blocks, 1000))),
                    n_first=first, n_last=last)
    hi = max(W, min(hi, 64 * 32768 * 1024 // (n_seq * n_kv * hd)))
    n_blocks = (hi + bs - 1) // bs
    n_sel = _log_int(rng, 1, min(n_blocks, 64 * 8 * 4096 * 128 // (n_seq * W * n_kv * hd * bs) + 1, 1000))
    return dict(op=op, fmt=rng.choice(["f16", "q8", "k8v4"]), n_seq=n_seq, W=W, n_kv=n_kv, G=G, hd=hd,
                bs=bs, lo=rng.randrange(W, hi + 1), hi=hi, n_sel=n_sel)


# ---------------------------------------------------------------------------
# Inputs, from the seed alone
# ---------------------------------------------------------------------------
def _lengths(rng, case):
    """The case's lengths (the same ones for every seed, so that a pool holds any) in the seed's order."""
    lens = np.random.default_rng([case["n_seq"], case["lo"], case["hi"]]).integers(
        case["lo"], case["hi"] + 1, case["n_seq"])
    return rng.permutation(lens.astype(np.int64))


def _table(rng, lens, bs, n_blocks=None, max_blocks=None):
    """Every sequence's blocks at shuffled places of the pool."""
    nb = -(-lens // bs)
    total = int(nb.sum())
    perm = rng.permutation(n_blocks or max(total, 1))
    width = max_blocks or max(int(nb.max()), 1)
    col = np.arange(width)
    live = col[None, :] < nb[:, None]
    start = np.cumsum(nb) - nb
    table = np.where(live, perm[np.minimum(start[:, None] + col, len(perm) - 1)], -1)
    return table.astype(np.int32), perm, total


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _keys(gen, n_blocks, n_kv, bs, hd):
    """Rows as keys look: a few channels per head far larger than the rest."""
    x = torch.randn(n_blocks, n_kv, bs, hd, generator=gen, device="cuda", dtype=torch.float16)
    gain = torch.ones(n_kv, 1, hd, device="cuda", dtype=torch.float16)
    gain.scatter_(2, torch.rand(n_kv, 1, hd, generator=gen, device="cuda").argsort(2)[:, :, :4], 6.0)
    return x.mul_(gain)


def _int8_rows(x):
    """int8 codes with one fp16 scale per 64 dims."""
    g = x.view(*x.shape[:-1], -1, GROUP)
    s = (g.abs().amax(-1).float() / 127).half()
    codes = (g / s.unsqueeze(-1)).round_().clamp_(-127, 127).to(torch.int8)
    return codes.view(x.shape), s


def _pool(gen, fmt, n_blocks, n_kv, bs, hd, values=True):
    """One layer's pool arrays in the library's layout."""
    k = _keys(gen, n_blocks, n_kv, bs, hd)
    p = {"k": k, "v": None, "ks": None, "vs": None}
    if fmt != F16:
        p["k"], p["ks"] = _int8_rows(k)
        del k
    shape = (n_blocks, n_kv, bs)
    if not values:      # the bounds read keys alone
        return p
    if fmt == F16:
        p["v"] = torch.randn(*shape, hd, generator=gen, device="cuda", dtype=torch.float16)
    elif fmt == Q8:
        p["v"], p["vs"] = _int8_rows(torch.randn(*shape, hd, generator=gen, device="cuda",
                                                 dtype=torch.float16))
    else:               # 4-bit codes of the rotated row (about N(0, hd)), a scale per 32 dims
        p["v"] = torch.randint(0, 256, (*shape, hd // 2), generator=gen, device="cuda",
                               dtype=torch.uint8)
        p["vs"] = (torch.rand(*shape, hd // 32, generator=gen, device="cuda") * 0.1 + 0.25).mul_(
            math.sqrt(hd)).half()
    return p


def _inputs(case, seed):
    rng = np.random.default_rng([int(seed), 77])
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    bs = case["bs"]
    if case["op"] == "plan":
        n, lens = case["n_seq"], _lengths(rng, case)
        n_new = np.full(n, case["new"], np.int64)
        if case["mixed"]:
            kind = rng.random(n)
            n_new = rng.integers(1, case["new"] + 1, n)
            n_new = np.where(kind < 0.25, 1, np.where(kind < 0.35, 0, np.where(kind < 0.45, -1, n_new)))
        need = int((-(-(lens + case["new"]) // bs)).sum()) + 1
        table, perm, used = _table(rng, lens, bs, need, case["max_blocks"])
        free = np.full(need, -1)
        free[:need - used] = perm[used:]
        return dict(ctx_in=_dev(lens.astype(np.int32)), n_new=_dev(n_new.astype(np.int32)),
                    block_table=_dev(table), free_list=_dev(free.astype(np.int32)),
                    free_count=_dev(np.array([need - used], np.int32)), n_blocks=need)
    lens = _lengths(rng, case)
    table, _, n_blocks = _table(rng, lens, bs)
    s = dict(ctx_lens=_dev(lens.astype(np.int32)), block_table=_dev(table), n_blocks=n_blocks,
             max_ctx=int(lens.max()))
    n_kv, hd = case["n_kv"], case["hd"]
    if case["op"] == "bound":
        start = np.maximum(lens - case["new"], 0)
        s["start"] = _dev(start.astype(np.int32))
        s["max_new"] = int((lens - start).max())
        s.update(_pool(gen, FORMATS[case["fmt"]], n_blocks, n_kv, bs, hd, values=False))
        s["bounds"] = torch.randint(-100, 101, (n_blocks, n_kv, 2, hd), generator=gen, device="cuda",
                                    dtype=torch.int8)
        s["scales"] = torch.exp2(torch.randint(-7, 0, (n_blocks, n_kv, hd // GROUP), generator=gen,
                                               device="cuda").float())
        return s
    W, G, n_seq = case["W"], case["G"], case["n_seq"]
    s["q"] = torch.randn(n_seq, W, n_kv * G, hd, generator=gen, device="cuda")
    if case["op"] == "select":
        # extremes of a block's cells: about 2.5 deviations out, spread between blocks; -127..127
        ext = torch.randn(n_blocks, n_kv, 2, hd, generator=gen, device="cuda").mul_(12).add_(84)
        ext = ext.clamp_(0, 127).round_().to(torch.int8)
        ext[:, :, 0].neg_()
        s["bounds"] = ext
        s["scales"] = torch.exp2(torch.randint(-6, -4, (n_blocks, n_kv, hd // GROUP), generator=gen,
                                               device="cuda").float())
        return s
    s.update(_pool(gen, FORMATS[case["fmt"]], n_blocks, n_kv, bs, hd))
    # each (token, KV head) has its own ascending list: a random choice with the newest block
    n_sel = case["n_sel"]
    vis = s["ctx_lens"].long()[:, None] - W + 1 + torch.arange(W, device="cuda")      # [n_seq][W]
    nb = (vis + bs - 1) // bs
    width = table.shape[1]
    col = torch.arange(width, device="cuda")
    r = torch.rand(n_seq, W, n_kv, width, generator=gen, device="cuda")
    r = torch.where(col == nb[..., None, None] - 1, -1.0, r)
    r = torch.where(col >= nb[..., None, None], 2.0, r)
    r = torch.nn.functional.pad(r, (0, max(0, n_sel - width)), value=2.0)
    val, idx = r.sort(-1)
    idx = torch.where(val[..., :n_sel] < 1.5, idx[..., :n_sel], 1 << 30).sort(-1)[0]
    have = idx < (1 << 30)
    tab = s["block_table"].long()[:, None, None, :].expand(n_seq, W, n_kv, width)
    blocks = torch.where(have, tab.gather(-1, idx.clamp(max=width - 1)), -1)
    s["sel_blocks"] = blocks.int()
    s["sel_lens"] = (have.sum(-1) * bs - (nb * bs - vis)[..., None]).int()
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    new = lambda *shape: torch.empty(*shape, dtype=torch.int32, device="cuda")  # noqa: E731
    n_seq = case["n_seq"]
    if case["op"] == "plan":
        m = case["max_tok"]
        s["out"] = dict(ctx_out=new(n_seq), tok_start=new(n_seq + 1), tok_seq=new(m), tok_pos=new(m),
                        slots=new(m), free_count_out=new(1), info=new(4))
    if case["op"] == "select":
        shape = (n_seq, case["W"], case["n_kv"])
        s["out"] = (new(*shape, case["n_sel"]), new(*shape, case["n_sel"]), new(*shape))
    if case["op"] == "attend":
        s["out"] = torch.empty_like(s["q"])
        s["sm_scale"] = 1.0 / math.sqrt(case["hd"])
    if own and case["op"] != "plan":
        import quantized_kv_cache_append_gb300 as kvq
        fmt = FORMATS[case.get("fmt", "f16")]
        k = s.get("k", s.get("bounds"))     # the selection reads the pool's geometry only
        v = s.get("v") if case["op"] == "attend" else k
        vs = s.get("vs") if case["op"] == "attend" else s.get("ks")
        s["cache"] = kvq.make_cache(fmt, case["n_kv"], case["hd"], case["bs"], s["n_blocks"], k, v,
                                    s.get("ks"), vs)
        if case["op"] == "attend":
            need = kvq.kvq_sparse_workspace_bytes(s["cache"], n_seq, case["W"],
                                                  case["n_kv"] * case["G"], case["n_sel"])
            s["workspace"] = torch.empty(need, dtype=torch.uint8, device="cuda")
    return s


# ---------------------------------------------------------------------------
# The library's calls
# ---------------------------------------------------------------------------
def _own(s, case):
    import quantized_kv_cache_append_gb300 as kvq
    if case["op"] == "plan":
        o = s["out"]
        kvq.check(kvq.kvq_plan_step(
            s["ctx_in"], s["n_new"], case["n_seq"], case["bs"], s["n_blocks"], s["block_table"],
            case["max_blocks"], s["free_list"], s["free_count"], case["max_tok"], o["ctx_out"],
            o["tok_start"], o["tok_seq"], o["tok_pos"], o["slots"], o["free_count_out"], o["info"]),
            "kvq_plan_step")
        return dict(o, block_table=s["block_table"], free_list=s["free_list"])
    n_seq, width = s["block_table"].shape
    if case["op"] == "bound":
        kvq.check(kvq.kvq_bound_blocks(s["cache"], s["block_table"], n_seq, width, s["start"],
                                       s["ctx_lens"], s["max_new"], s["bounds"], s["scales"]),
                  "kvq_bound_blocks")
        return _bound_values(s["bounds"], s["scales"])
    n_q = case["n_kv"] * case["G"]
    if case["op"] == "select":
        blocks, index, lens = s["out"]
        kvq.check(kvq.kvq_select_blocks(
            s["cache"], s["bounds"], s["scales"], s["q"], n_seq, case["W"], n_q, s["ctx_lens"],
            s["max_ctx"], s["block_table"], width, case["n_sel"], case["n_first"], case["n_last"],
            blocks, index, lens), "kvq_select_blocks")
        return s["out"]
    kvq.check(kvq.kvq_sparse_decode_attn(
        s["cache"], s["q"], n_seq, case["W"], n_q, s["sel_blocks"], s["sel_lens"], case["n_sel"],
        s["sm_scale"], s["out"], s["workspace"], s["workspace"].numel()), "kvq_sparse_decode_attn")
    return s["out"]


# ---------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------
def _bound_values(bounds, scales):
    """The values the bounds' codes stand for."""
    n, kv, _, hd = bounds.shape
    return bounds.view(n, kv, 2, hd // GROUP, GROUP) * scales.view(n, kv, 1, hd // GROUP, 1)


def _plan_plain(s, case):
    bs, width, n_seq, m = case["bs"], case["max_blocks"], case["n_seq"], case["max_tok"]
    n_blocks = s["n_blocks"]
    ctx, n_new = s["ctx_in"].long(), s["n_new"].long()
    table, free, count = s["block_table"].long(), s["free_list"].long(), s["free_count"].long()
    released = n_new < 0
    add = n_new.clamp(min=0)
    have = (ctx + bs - 1) // bs
    grow = torch.where(released, 0, (ctx + add + bs - 1) // bs - have)
    back = torch.where(released, have, 0)
    tok_end, grow_end, back_end = add.cumsum(0), grow.cumsum(0), back.cumsum(0)
    tok_start, grow_start, back_start = tok_end - add, grow_end - grow, back_end - back
    T, A, P = tok_end[-1:], grow_end[-1:], back_end[-1:]
    status = ((T > m).long() + 2 * (ctx + add > width * bs).any().long()
              + 4 * (A > count + P).long() + 8 * (count + P > n_blocks).long())
    ok = status == 0
    # the blocks that come back, and the new ones: first those, last ones first, then the free list's
    j = torch.arange(n_blocks, device="cuda")
    bseq = torch.searchsorted(back_end, j, right=True).clamp(max=n_seq - 1)
    pushed = table[bseq, (j - back_start[bseq]).clamp(0, width - 1)]
    ids = torch.where(j < P, pushed[(P - 1 - j).clamp(0, n_blocks - 1)],
                      free[(count - 1 - (j - P)).clamp(0, n_blocks - 1)])
    gseq = torch.searchsorted(grow_end, j, right=True).clamp(max=n_seq - 1)
    at = torch.where((j < A) & ok, gseq * width + have[gseq] + j - grow_start[gseq], n_seq * width)
    new_table = torch.cat([table.reshape(-1), table.new_zeros(1)])
    new_table[at.clamp(0, n_seq * width)] = ids
    new_table = new_table[:-1].view(n_seq, width)
    k = j - count
    free = torch.where((k >= 0) & (k < P - A) & ok, pushed[k.clamp(0, n_blocks - 1)], free)
    # every token's sequence, position and cell
    t = torch.arange(m, device="cuda")
    seq = torch.searchsorted(tok_end, t, right=True).clamp(max=n_seq - 1)
    live = (t < T) & ok
    pos = ctx[seq] + t - tok_start[seq]
    slot = new_table[seq, (pos // bs).clamp(max=width - 1)] * bs + pos % bs
    none = torch.full_like(t, -1)
    i32 = lambda x: x.int()  # noqa: E731
    return dict(ctx_out=i32(torch.where(ok, torch.where(released, 0, ctx + add), ctx)),
                tok_start=i32(torch.where(ok, torch.cat([tok_start, T]), 0)),
                tok_seq=i32(torch.where(live, seq, none)), tok_pos=i32(torch.where(live, pos, none)),
                slots=i32(torch.where(live, slot, none)),
                free_count_out=i32(torch.where(ok, count + P - A, count)),
                info=i32(torch.cat([torch.where(ok, T, 0), torch.where(ok, A, 0),
                                    torch.where(ok, P, 0), status])),
                block_table=i32(new_table), free_list=i32(free))


def _scale_exponent(m, lowest, highest):
    """The smallest e with 127 * 2^e >= m, in [lowest, highest]."""
    f, x = torch.frexp(m)
    e = x - 7 + (f > 127 / 128).int()
    return torch.where(m == 0, lowest, e).clamp(lowest, highest)


def _pow2(e):
    return torch.exp2(e.double()).float()


def _bound_plain(s, case):
    bs, n_kv, hd = case["bs"], case["n_kv"], case["hd"]
    touched = (s["max_new"] + bs - 2) // bs + 1
    ctx = s["ctx_lens"].long()
    j = torch.minimum((s["start"].long() // bs)[:, None] + torch.arange(touched, device="cuda"),
                      ((ctx - 1) // bs)[:, None])                       # [n_seq][touched]
    phys = s["block_table"].long().gather(1, j)
    k = s["k"][phys].float()                                            # [..][n_kv][bs][hd]
    if s["ks"] is not None:
        k = (k.view(*k.shape[:-1], hd // GROUP, GROUP) * s["ks"][phys].float().unsqueeze(-1)).view(k.shape)
    cell = j[..., None] * bs + torch.arange(bs, device="cuda")
    live = (cell < ctx[:, None, None])[:, :, None, :, None]
    lo = torch.where(live, k, torch.inf).amin(3)
    hi = torch.where(live, k, -torch.inf).amax(3)
    lo, hi = lo.view(*lo.shape[:-1], -1, GROUP), hi.view(*hi.shape[:-1], -1, GROUP)
    scale = _pow2(_scale_exponent(torch.maximum(lo.abs(), hi.abs()).amax(-1), -24, 16))
    s["bounds"][phys] = torch.stack([(lo / scale[..., None]).floor(), (hi / scale[..., None]).ceil()],
                                    3).to(torch.int8).view(*phys.shape, n_kv, 2, hd)
    s["scales"][phys] = scale
    return _bound_values(s["bounds"], s["scales"])


def _visible(s, case):
    """Cells each query token sees: [n_seq][W]."""
    W = case["W"]
    return (s["ctx_lens"].long()[:, None] - W + 1 + torch.arange(W, device="cuda")).clamp(min=0)


def _pick(score, s, case):
    """score [n_seq][W][n_kv][blocks] -> lists, indexes and cell counts."""
    bs, n_sel = case["bs"], case["n_sel"]
    vis = _visible(s, case)[..., None, None]
    nb = (vis + bs - 1) // bs
    n = score.shape[-1]
    col = torch.arange(n, device="cuda")
    table = s["block_table"].long()[:, None, None, :].expand(*score.shape)
    score = torch.where((col < case["n_first"]) | (col >= nb - case["n_last"]), torch.inf, score)
    score = torch.where((col < nb) & (table >= 0) & (table < s["n_blocks"]), score, -torch.inf)
    score = torch.nn.functional.pad(score, (0, max(0, n_sel - n)), value=-torch.inf)
    val, idx = torch.sort(score, dim=-1, descending=True, stable=True)
    idx = torch.where(val[..., :n_sel] > -torch.inf, idx[..., :n_sel], 1 << 30).sort(-1)[0]
    chosen = idx < (1 << 30)
    blocks = torch.where(chosen, table.gather(-1, idx.clamp(max=n - 1)), -1)
    short = torch.where((idx == nb - 1).any(-1), (nb * bs - vis)[..., 0], 0)
    lens = chosen.sum(-1) * bs - short
    return blocks.int(), torch.where(chosen, idx, -1).int(), lens.int()


def _select_plain(s, case):
    W, n_kv, G, hd = case["W"], case["n_kv"], case["G"], case["hd"]
    ng, n_seq = hd // GROUP, case["n_seq"]
    q = s["q"].view(n_seq, W, n_kv, G, ng, GROUP)
    qs = _pow2(_scale_exponent(q.abs().amax(-1), -60, 60))
    code = (q / qs[..., None]).round()
    c = torch.cat([code.clamp(max=0), code.clamp(min=0)], -1)              # against (lo, hi)
    c = c.permute(0, 2, 4, 1, 3, 5).reshape(n_seq, n_kv, ng, W * G, 2 * GROUP)
    phys = s["block_table"].long().clamp(0, s["n_blocks"] - 1)
    b = s["bounds"][phys].view(n_seq, -1, n_kv, 2, ng, GROUP).permute(0, 2, 4, 3, 5, 1)
    b = b.reshape(n_seq, n_kv, ng, 2 * GROUP, -1).float()
    S = c @ b                                                              # whole numbers below 2^24
    ks = s["scales"][phys].permute(0, 2, 3, 1)[:, :, :, None, :]
    qs = qs.permute(0, 2, 4, 1, 3).reshape(n_seq, n_kv, ng, W * G, 1)
    t = S * (ks * qs)
    t = t[:, :, 0::2] + t[:, :, 1::2] if ng > 1 else t
    t = t[:, :, 0::2] + t[:, :, 1::2] if ng > 2 else t
    score = t[:, :, 0].view(n_seq, n_kv, W, G, -1).amax(3)
    return _pick(score.transpose(1, 2), s, case)


def _hadamard(n, dtype):
    i = torch.arange(n, device="cuda")
    bits = (i[:, None, None] & i[None, :, None]) >> torch.arange(8, device="cuda") & 1
    return (1 - 2 * (bits.sum(-1) % 2)).to(dtype)


def _listed_rows(s, case, name, pseudo, dtype):
    """The listed cells' keys or values, dequantised: [lists][n_sel * bs][hd]."""
    blocks = s["sel_blocks"].view(-1, case["n_sel"])[pseudo].long().clamp(min=0)
    heads = (pseudo % case["n_kv"])[:, None]
    x, sc = s[name][blocks, heads], s["ks" if name == "k" else "vs"]
    if FORMATS[case["fmt"]] == K8V4 and name == "v":
        x = torch.stack([x & 15, x >> 4], -1).view(*x.shape[:-1], case["hd"]).to(dtype) - 8
    else:
        x = x.to(dtype)
    if sc is not None:
        sc = sc[blocks, heads].to(dtype)
        x = (x.view(*sc.shape, -1) * sc[..., None]).view(x.shape)
    return x.reshape(len(pseudo), -1, case["hd"])


def _attend(s, case, pseudo, dtype):
    """Softmax attention of the given lists' query rows: [lists][G][hd]."""
    q = s["q"].view(-1, case["G"], case["hd"])[pseudo].to(dtype)
    k = _listed_rows(s, case, "k", pseudo, dtype)
    lens = s["sel_lens"].view(-1)[pseudo].long()[:, None, None]
    live = torch.arange(k.shape[1], device="cuda") < lens
    z = torch.where(live, q @ k.transpose(1, 2) * s["sm_scale"], -torch.inf)
    top = z.amax(-1, keepdim=True)
    p = torch.exp(z - torch.where(top == -torch.inf, 0, top))
    o = p @ _listed_rows(s, case, "v", pseudo, dtype) / p.sum(-1, keepdim=True).clamp(min=1e-30)
    if FORMATS[case["fmt"]] == K8V4:
        o = o @ _hadamard(case["hd"], dtype) / case["hd"]
    return o


def run(state):
    case = state["case"]
    if own:
        return _own(state, case)
    if case["op"] == "plan":
        return _plan_plain(state, case)
    if case["op"] == "bound":
        return _bound_plain(state, case)
    if case["op"] == "select":
        return _select_plain(state, case)
    every = torch.arange(case["n_seq"] * case["W"] * case["n_kv"], device="cuda")
    return _attend(state, case, every, torch.float32).view(state["q"].shape)


# ---------------------------------------------------------------------------
# What one pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    n, bs = case["n_seq"], case["bs"]
    mean = (case["lo"] + case["hi"]) / 2
    if case["op"] == "plan":
        # lengths in and out, the tokens' three numbers (padding too), the blocks handed over
        return dict(bytes=16 * n + 12 * case["max_tok"] + 8 * case["max_tok"] / bs, flops=0)
    n_kv, hd = case["n_kv"], case["hd"]
    if case["op"] == "bound":
        row = 2 * hd if case["fmt"] == "f16" else hd + hd // 32
        cells = n * min(mean, case["new"] if case["new"] >= bs else (bs + 1) / 2)
        entry = 2 * hd + hd // 16
        return dict(bytes=n_kv * (cells * row + math.ceil(cells / bs) * entry), flops=2 * n_kv * cells * hd)
    W, rows = case["W"], case["W"] * case["G"]
    if case["op"] == "select":
        blocks = n * mean / bs
        out = 8 * n * W * n_kv * case["n_sel"]
        return dict(bytes=blocks * n_kv * (2 * hd + hd // 16) + 4 * n * rows * n_kv * hd + out,
                    flops=4 * blocks * n_kv * rows * hd)
    row = {"f16": 4 * hd, "q8": 2 * hd + hd // 16, "k8v4": hd + hd // 32 + hd // 2 + hd // 16}[case["fmt"]]
    cells = n * W * n_kv * min(mean, case["n_sel"] * bs)
    read = min(cells, n * n_kv * mean) * row
    return dict(bytes=read + 8 * n * rows * n_kv * hd, flops=4 * cells * case["G"] * hd)


# ---------------------------------------------------------------------------
# The definitions, in 64 bits and written apart from the plain forms
# ---------------------------------------------------------------------------
def _plan_exact(s, case):
    bs, width, m, n_blocks = case["bs"], case["max_blocks"], case["max_tok"], s["n_blocks"]
    ctx = s["ctx_in"].cpu().numpy().astype(np.int64)
    n_new = s["n_new"].cpu().numpy().astype(np.int64)
    table, free = s["block_table"].cpu().numpy().copy(), s["free_list"].cpu().numpy().copy()
    count = int(s["free_count"].cpu()[0])
    n = len(ctx)
    stack = list(free[:count])
    for b in range(n):
        if n_new[b] < 0:
            stack.extend(table[b, :-(-ctx[b] // bs)])
    back = len(stack) - count
    out_ctx, start = ctx.copy(), np.zeros(n + 1, np.int64)
    tok_seq, tok_pos, slots = (np.full(m, -1, np.int64) for _ in range(3))
    at = handed = 0
    for b in range(n):
        start[b] = at
        if n_new[b] < 0:
            out_ctx[b] = 0
            continue
        end = ctx[b] + n_new[b]
        for c in range(-(-ctx[b] // bs), -(-end // bs)):
            table[b, c] = stack.pop()
            handed += 1
        pos = np.arange(ctx[b], end)
        tok_seq[at:at + len(pos)] = b
        tok_pos[at:at + len(pos)] = pos
        slots[at:at + len(pos)] = table[b, pos // bs].astype(np.int64) * bs + pos % bs
        out_ctx[b] = end
        at += len(pos)
    start[n] = at
    if len(stack) > count:
        free[count:len(stack)] = stack[count:]
    i32 = lambda x: torch.from_numpy(np.asarray(x).astype(np.int32))  # noqa: E731
    return dict(ctx_out=i32(out_ctx), tok_start=i32(start), tok_seq=i32(tok_seq), tok_pos=i32(tok_pos),
                slots=i32(slots), free_count_out=i32([len(stack)]), info=i32([at, handed, back, 0]),
                block_table=i32(table), free_list=i32(free))


def _bound_exact(s, case):
    bs, hd, n_kv = case["bs"], case["hd"], case["n_kv"]
    scales = s["scales"].double()
    values = s["bounds"].double().view(-1, n_kv, 2, hd // GROUP, GROUP) * scales[:, :, None, :, None]
    table = s["block_table"].cpu().numpy()
    ctx, start = s["ctx_lens"].cpu().numpy(), s["start"].cpu().numpy()
    ids, live = [], []
    for b in range(len(ctx)):
        for j in range(start[b] // bs, -(-ctx[b] // bs)):
            ids.append(int(table[b, j]))
            live.append(min(bs, int(ctx[b]) - j * bs))
    step = max(1, (1 << 27) // (n_kv * bs * hd))
    for a in range(0, len(ids), step):
        at = torch.tensor(ids[a:a + step], device="cuda")
        k = s["k"][at].double().view(len(at), n_kv, bs, hd // GROUP, GROUP)
        if s["ks"] is not None:
            k = k * s["ks"][at].double()[..., None]
        off = torch.arange(bs, device="cuda") >= torch.tensor(live[a:a + step], device="cuda")[:, None]
        off = off[:, None, :, None, None]
        lo, hi = k.masked_fill(off, 1e300).amin(2), k.masked_fill(off, -1e300).amax(2)
        top = torch.maximum(-lo, hi).clamp(min=0).amax(-1)
        scale = torch.full_like(top, 2.0 ** -24)
        for e in range(-24, 16):
            scale = torch.where(127 * 2.0 ** e < top, 2.0 ** (e + 1), scale)
        scale = scale[..., None]
        values[at] = torch.stack([torch.floor(lo / scale) * scale, torch.ceil(hi / scale) * scale], 2)
    return values


def _select_exact(s, case):
    W, n_kv, G, hd, bs, n_sel = (case[x] for x in ("W", "n_kv", "G", "hd", "bs", "n_sel"))
    ng = hd // GROUP
    table, ctx = s["block_table"].cpu().numpy(), s["ctx_lens"].cpu().numpy()
    blocks = np.full((case["n_seq"], W, n_kv, n_sel), -1, np.int32)
    index, lens = blocks.copy(), np.zeros((case["n_seq"], W, n_kv), np.int32)
    for b in range(case["n_seq"]):
        q = s["q"][b].double().view(W, n_kv, G, ng, GROUP)
        top = q.abs().amax(-1, keepdim=True)
        scale = torch.full_like(top, 2.0 ** -60)
        for e in range(-60, 60):
            scale = torch.where(127 * 2.0 ** e < top, 2.0 ** (e + 1), scale)
        code = torch.round(q / scale)
        ids = np.clip(table[b, :-(-int(ctx[b]) // bs)], 0, s["n_blocks"] - 1)
        at = torch.from_numpy(ids.astype(np.int64)).cuda()
        bound = s["bounds"][at].double().view(len(ids), n_kv, 2, ng, GROUP)
        # every pair of a query's sign and the bound that can only raise the product, summed exactly
        up = torch.einsum("whgnd,bhnd->whgnb", code.clamp(min=0), bound[:, :, 1])
        up += torch.einsum("whgnd,bhnd->whgnb", code.clamp(max=0), bound[:, :, 0])
        t = up * scale * s["scales"][at].double().permute(1, 2, 0)[None, :, None]
        t = t.float()                             # exact: whole numbers below 2^21 times powers of two
        if ng == 1:
            sc = t[:, :, :, 0]
        elif ng == 2:
            sc = t[:, :, :, 0] + t[:, :, :, 1]
        else:
            sc = (t[:, :, :, 0] + t[:, :, :, 1]) + (t[:, :, :, 2] + t[:, :, :, 3])
        sc = sc.amax(2).cpu().numpy()
        for w in range(W):
            vis = max(0, int(ctx[b]) - W + w + 1)
            nb = -(-vis // bs)
            ok = [j for j in range(nb) if 0 <= table[b, j] < s["n_blocks"]]
            ok = np.array(ok, np.int64)
            for h in range(n_kv):
                val = sc[w, h][ok].astype(np.float64)
                val[(ok < case["n_first"]) | (ok >= nb - case["n_last"])] = np.inf
                best = np.sort(ok[np.lexsort((ok, -val))[:n_sel]])
                index[b, w, h, :len(best)] = best
                blocks[b, w, h, :len(best)] = table[b, best]
                cells = len(best) * bs
                if len(best) and best[-1] == nb - 1:
                    cells -= nb * bs - vis
                lens[b, w, h] = cells
    return tuple(torch.from_numpy(x) for x in (blocks, index, lens))


def _attend_exact(s, case):
    W, n_kv, G, hd, bs = (case[x] for x in ("W", "n_kv", "G", "hd", "bs"))
    fmt = FORMATS[case["fmt"]]
    out = torch.zeros(case["n_seq"], W, n_kv, G, hd, dtype=torch.float64, device="cuda")
    rot = torch.ones(1, 1, dtype=torch.float64, device="cuda")
    while rot.shape[0] < hd:
        rot = torch.cat([torch.cat([rot, rot], 1), torch.cat([rot, -rot], 1)], 0)
    for b in range(case["n_seq"]):
        for w in range(W):
            for h in range(n_kv):
                n = int(s["sel_lens"][b, w, h])
                if n <= 0:
                    continue
                at = s["sel_blocks"][b, w, h].long()[:-(-n // bs)]
                k = s["k"][at, h].reshape(-1, hd)[:n].double()
                v = s["v"][at, h]
                if fmt == K8V4:
                    pair = torch.zeros(*v.shape, 2, dtype=torch.float64, device="cuda")
                    pair[..., 0] = (v % 16).double() - 8
                    pair[..., 1] = torch.div(v, 16, rounding_mode="floor").double() - 8
                    v = pair
                v = v.reshape(-1, hd)[:n].double()
                if fmt != F16:
                    k = k * s["ks"][at, h].reshape(-1, hd // GROUP)[:n].double().repeat_interleave(GROUP, 1)
                    per = 32 if fmt == K8V4 else GROUP
                    v = v * s["vs"][at, h].reshape(-1, hd // per)[:n].double().repeat_interleave(per, 1)
                q = s["q"][b, w].view(n_kv, G, hd)[h].double()
                p = torch.softmax(s["sm_scale"] * (q @ k.T), -1)
                o = p @ v
                out[b, w, h] = o @ rot.T / hd if fmt == K8V4 else o
    return out.view(case["n_seq"], W, n_kv * G, hd)


def exact(case, seed):
    s = _inputs(case, seed)
    if case["op"] == "attend":
        s["sm_scale"] = 1.0 / math.sqrt(case["hd"])
    return {"plan": _plan_exact, "bound": _bound_exact, "select": _select_exact,
            "attend": _attend_exact}[case["op"]](s, case)
