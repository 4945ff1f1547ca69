"""A speculative decoding step around the paged K/V cache, operator by operator:
cases, plain forms in torch, and the definitions in 64 bits.

    rotary  norms of each head's query and key, rotary positions (one axis or several),
            and the new keys and values written into the paged cache, in one pass
    score   decode and verify-window attention over the cache, its scores capped by a tanh,
            biased by the distance, kept to a window or to a first cell
    chunk   the same scores for a prompt chunk over fp16 staging, with document and prefix masks
    verify  drafted tokens accepted or replaced by the target's probabilities, from given
            random numbers
    trim    the cells of rejected drafts taken back, their blocks returned to the free list

`run` computes the plain form, or, with `own` set, calls the library.
"""
import math

import numpy as np
import torch

own = False

FORMATS = {"f16": 0, "q8": 1, "k8v4": 2}            # the library's cache formats
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
TYPE_IDS = {"f32": 0, "f16": 1, "bf16": 2}          # the library's element types
UNIT = 2.0 ** 40                                    # weights of a sampled row are whole multiples of 1 / UNIT


def listed():
    return [
        # what every decode step of 64 running requests pays before its attention
        dict(name="rotary_step", op="rotary", kind="step", dtype="bf16", fmt="f16", n_tok=64, n_q=32, n_kv=8,
             hd=128, rot=128, interleaved=False, axes=1, norm=True, bs=64, top=131071),
        # a 4096-token prompt into an int8 cache, read back as the chunk attention takes it
        dict(name="rotary_prompt_q8", op="rotary", kind="prompt", dtype="bf16", fmt="q8", n_tok=4096, n_q=32,
             n_kv=8, hd=128, rot=128, interleaved=False, axes=1, norm=True, bs=256, top=4096),
        # images and video: time, height and width, half of wide heads rotated, 4-bit values
        dict(name="rotary_video_k8v4", op="rotary", kind="prompt", dtype="f32", fmt="k8v4", n_tok=16381, n_q=16,
             n_kv=2, hd=256, rot=128, interleaved=True, axes=3, norm=False, bs=16, top=16381),
        # one request's token, a layer with a window: only the window's cells are needed
        dict(name="score_window_f16", op="score", fmt="f16", n_seq=1, W=1, n_kv=8, G=4, hd=128, bs=64, lo=32768,
             hi=32768, cap=50.0, window=4096, slopes=False, first=False),
        # 16 ragged requests, capped scores, int8 cache
        dict(name="score_ragged_q8", op="score", fmt="q8", n_seq=16, W=1, n_kv=8, G=4, hd=128, bs=256, lo=1024,
             hi=16384, cap=30.0, window=0, slopes=False, first=False),
        # a 4-token verify window over a long context, distance bias, padding in front, 4-bit values
        dict(name="score_verify_k8v4", op="score", fmt="k8v4", n_seq=2, W=4, n_kv=2, G=8, hd=256, bs=16, lo=65536,
             hi=131072, cap=0.0, window=0, slopes=True, first=True),
        # a short chunk of a prompt with a bidirectional prefix, window and distance bias, narrow heads
        dict(name="chunk_prefix_hd64", op="chunk", T=257, P=4099, n_kv=4, G=3, hd=64, cap=0.0, window=1024,
             slopes=True, docs=1, prefix=130, out="f16"),
        # a full chunk of several packed documents, capped scores
        dict(name="chunk_docs_hd128", op="chunk", T=4096, P=16384, n_kv=8, G=4, hd=128, cap=50.0, window=0,
             slopes=False, docs=3, prefix=0, out="bf16"),
        # three drafts each for 16 requests, a small vocabulary
        dict(name="verify_step", op="verify", n_seq=16, W=4, vocab=32000, dtype="f32", drafts="given"),
        # a full batch, five drafts each, a large vocabulary, 16-bit probabilities
        dict(name="verify_batch", op="verify", n_seq=256, W=6, vocab=131075, dtype="bf16", drafts="given"),
        # after the verify step of 64 requests
        dict(name="trim_step", op="trim", n_seq=64, bs=16, max_blocks=1024, lo=1024, hi=16383, drop=5),
        # many requests cut back to a shared prefix
        dict(name="trim_rollback", op="trim", n_seq=4000, bs=16, max_blocks=256, lo=0, hi=4096, drop=4096),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rotary", "score", "chunk", "verify", "trim"])
    if op == "trim":
        hi = _log_int(rng, 1, 16383)
        bs = rng.choice([16, 32, 64, 256])
        return dict(op=op, n_seq=_log_int(rng, 1, 4000), bs=bs, max_blocks=hi // bs + 1 + rng.randrange(3),
                    lo=rng.randrange(hi), hi=hi, drop=_log_int(rng, 1, hi))
    if op == "verify":
        vocab = _log_int(rng, 300, 150000)
        return dict(op=op, n_seq=max(1, min(_log_int(rng, 1, 256), 30_000_000 // vocab)), W=rng.randrange(2, 9),
                    vocab=vocab, dtype=rng.choice(["f32", "f16", "bf16"]),
                    drafts=rng.choice(["given", "given", "certain"]))
    n_kv, G, hd = rng.choice([(8, 4, 128), (2, 8, 256), (1, 4, 128), (4, 1, 64), (3, 7, 64), (5, 3, 128),
                              (8, 2, 64), (1, 16, 256)])
    cap, slopes = rng.choice([0.0, 20.0, 30.0, 50.0]), rng.random() < 0.4
    if op == "rotary":
        axes = rng.choice([1, 1, 2, 3])
        kind = rng.choice(["step", "prompt"])
        n_tok = _log_int(rng, 1, 512 if kind == "step" else 16384 * 1024 // (n_kv * (G + 2) * hd) + 1)
        return dict(op=op, kind=kind, dtype=rng.choice(["f32", "f16", "bf16"]),
                    fmt="f16" if kind == "step" else rng.choice(["f16", "q8", "k8v4"]), n_tok=n_tok, n_q=n_kv * G,
                    n_kv=n_kv, hd=hd, rot=rng.choice([hd, hd, hd // 2, 32]), interleaved=rng.random() < 0.4,
                    axes=axes, norm=rng.random() < 0.7, bs=rng.choice([16, 64, 256]),
                    top=_log_int(rng, 1, 262143) if kind == "step" else n_tok)
    window = rng.choice([0, 0, _log_int(rng, 16, 8192)])
    if op == "score":
        W = rng.choice([w for w in (1, 1, 1, 2, 3, 4) if w * G <= 32])
        n_seq = _log_int(rng, 1, 64)
        hi = max(W, min(_log_int(rng, 1, 131072), 16 * 16384 * 1024 // (n_seq * n_kv * hd)))
        return dict(op=op, fmt=rng.choice(["f16", "q8", "k8v4"]), n_seq=n_seq, W=W, n_kv=n_kv, G=G, hd=hd,
                    bs=rng.choice([16, 32, 64, 256]), lo=rng.randrange(W, hi + 1), hi=hi, cap=cap, window=window,
                    slopes=slopes, first=rng.random() < 0.4)
    T = _log_int(rng, 1, 2048)
    P = max(T, min(_log_int(rng, T, 32768), 40_000_000_000 // (T * n_kv * G * hd)))
    docs = rng.choice([1, 1, 3, 8])
    return dict(op=op, T=T, P=P, n_kv=n_kv, G=G, hd=hd, cap=cap, window=window, slopes=slopes, docs=min(docs, T),
                prefix=rng.randrange(T + 1) if docs == 1 and rng.random() < 0.4 else 0,
                out=rng.choice(["f16", "bf16"]))


# ---------------------------------------------------------------------------
# Inputs, from the seed alone
# ---------------------------------------------------------------------------
def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _ints(a):
    return _dev(np.asarray(a).astype(np.int32))


def _lengths(rng, case):
    """The case's lengths (the same ones for every seed, so that a pool holds any) in the seed's order."""
    lens = np.random.default_rng([case["n_seq"], case["lo"], case["hi"]]).integers(
        case["lo"], case["hi"] + 1, case["n_seq"])
    return rng.permutation(lens.astype(np.int64))


def _table(rng, lens, bs, width=None, spare=0):
    """Every sequence's blocks at shuffled places of a pool with `spare` blocks more."""
    nb = -(-lens // bs)
    total = int(nb.sum())
    perm = rng.permutation(max(total + spare, 1))
    col = np.arange(width or max(int(nb.max()), 1))
    start = np.cumsum(nb) - nb
    table = np.where(col[None, :] < nb[:, None], perm[np.minimum(start[:, None] + col, len(perm) - 1)], -1)
    return table, perm, total


def _int8_rows(x):
    """int8 codes with one fp16 scale per 64 dims."""
    g = x.view(*x.shape[:-1], -1, 64)
    s = (g.abs().amax(-1).float() / 127).half()
    return (g / s.unsqueeze(-1)).round_().clamp_(-127, 127).to(torch.int8).view(x.shape), s


def _pool(gen, fmt, n_blocks, n_kv, bs, hd):
    """One layer's pool arrays in the library's layout, a few channels of the keys far larger than the rest."""
    shape = (n_blocks, n_kv, bs)
    half = lambda: torch.randn(*shape, hd, generator=gen, device="cuda", dtype=torch.float16)  # noqa: E731
    gain = torch.ones(n_kv, 1, hd, device="cuda", dtype=torch.float16)
    gain.scatter_(2, torch.rand(n_kv, 1, hd, generator=gen, device="cuda").argsort(2)[:, :, :4], 6.0)
    p = {"k": half().mul_(gain), "v": None, "ks": None, "vs": None}
    if fmt != "f16":
        p["k"], p["ks"] = _int8_rows(p["k"])
    if fmt == "f16":
        p["v"] = half()
    elif fmt == "q8":
        p["v"], p["vs"] = _int8_rows(half())
    else:       # 4-bit codes of the rotated row (about N(0, hd)), a scale per 32 dims
        p["v"] = torch.randint(0, 256, (*shape, hd // 2), generator=gen, device="cuda", dtype=torch.uint8)
        p["vs"] = (torch.rand(*shape, hd // 32, generator=gen, device="cuda") * 0.1 + 0.25).mul_(
            math.sqrt(hd)).half()
    return p


def _empty_pool(fmt, n_blocks, n_kv, bs, hd):
    z = lambda n, dt: torch.zeros(n_blocks, n_kv, bs, n, dtype=dt, device="cuda")  # noqa: E731
    if fmt == "f16":
        return dict(k=z(hd, torch.float16), v=z(hd, torch.float16), ks=None, vs=None)
    p = dict(k=z(hd, torch.int8), ks=z(hd // 64, torch.float16))
    if fmt == "q8":
        return dict(p, v=z(hd, torch.int8), vs=z(hd // 64, torch.float16))
    return dict(p, v=z(hd // 2, torch.uint8), vs=z(hd // 32, torch.float16))


def _rotary_inputs(case, rng, gen):
    n, n_q, n_kv, hd, bs, rot = (case[x] for x in ("n_tok", "n_q", "n_kv", "hd", "bs", "rot"))
    qkv = torch.randn(n, (n_q + 2 * n_kv) * hd, generator=gen, device="cuda").to(TYPES[case["dtype"]])
    s = dict(q_in=qkv[:, :n_q * hd], k_in=qkv[:, n_q * hd:(n_q + n_kv) * hd], v_in=qkv[:, (n_q + n_kv) * hd:])
    if case["kind"] == "step":      # one token of each sequence, anywhere in it
        pos, seq = rng.integers(0, case["top"] + 1, n), np.arange(n)
        table = np.full((n, case["top"] // bs + 1), -1)
        table[seq, pos // bs] = rng.permutation(n)
        n_blocks = n
    else:
        pos, seq = np.arange(n), np.zeros(n, np.int64)
        table, _, n_blocks = _table(rng, np.array([n]), bs)
    s.update(tok_seq=_ints(seq), tok_pos=_ints(pos), block_table=_ints(table), n_blocks=n_blocks, positions=None,
             pair_axis=None, q_norm=None, k_norm=None, q_out=torch.empty(n, n_q, hd, device="cuda"))
    pair = np.arange(rot // 2)
    s["inv_freq"] = _dev((10000.0 ** (-2.0 * pair / max(rot, 1))).astype(np.float32))
    if case["axes"] > 1:            # a frame number, a row and a column
        grid = [pos // 256, pos % 256 // 16, pos % 16][-case["axes"]:]
        s["positions"] = _ints(np.stack(grid))
        s["pair_axis"] = _ints(pair * case["axes"] // max(rot // 2, 1))
    if case["norm"]:
        s["q_norm"], s["k_norm"] = (1 + 0.3 * torch.randn(2, hd, generator=gen, device="cuda")).unbind(0)
        s["k_norm"][::17] *= 5.0
    s.update(_empty_pool(case["fmt"], n_blocks, n_kv, bs, hd))
    if case["kind"] == "prompt":
        s["staging"] = torch.empty(2, n_kv, n, hd, dtype=torch.float16, device="cuda")
    return s


def _head_slopes(n_q):
    """One slope per query head, a geometric series from steep to flat."""
    return (2.0 ** (-8.0 * (torch.arange(n_q, device="cuda") + 1) / n_q)).float()


def _score_inputs(case, rng, gen):
    W, n_q = case["W"], case["n_kv"] * case["G"]
    lens = _lengths(rng, case)
    table, _, n_blocks = _table(rng, lens, case["bs"])
    s = dict(ctx_lens=_ints(lens), block_table=_ints(table), n_blocks=n_blocks, max_ctx=int(lens.max()))
    s["q"] = torch.randn(case["n_seq"], W, n_q, case["hd"], generator=gen, device="cuda")
    s["slopes"] = _head_slopes(n_q) if case["slopes"] else None
    s["first"] = _ints(rng.integers(0, np.maximum(lens // 4, 1))) if case["first"] else None
    s.update(_pool(gen, case["fmt"], n_blocks, case["n_kv"], case["bs"], case["hd"]))
    s["out"] = torch.empty_like(s["q"])
    return s


def _chunk_inputs(case, rng, gen):
    T, P, n_kv, hd = case["T"], case["P"], case["n_kv"], case["hd"]
    n_q = n_kv * case["G"]
    half = lambda: torch.randn(n_kv, P, hd, generator=gen, device="cuda", dtype=torch.float16)  # noqa: E731
    s = dict(k=half(), v=half(), q=torch.randn(T, n_q, hd, generator=gen, device="cuda") * 2, first=None, last=None)
    if case["docs"] > 1:            # the first one began before the chunk
        cut = np.sort(rng.choice(np.arange(1, T), case["docs"] - 1, replace=False)) + P - T
        starts = np.concatenate([[max(0, (P - T) // 2)], cut])
        s["first"] = _ints(starts[np.searchsorted(cut, np.arange(P - T, P), side="right")])
    if case["prefix"]:              # the chunk's first tokens belong to a prefix that sees itself whole
        pos = np.arange(P - T, P)
        end = P - T + case["prefix"] - 1
        s["last"] = _ints(np.where(pos <= end, end, pos))
    s["slopes"] = _head_slopes(n_q) if case["slopes"] else None
    s["out"] = torch.empty(T, n_q, hd, dtype=TYPES[case["out"]], device="cuda")
    return s


def _verify_inputs(case, rng, gen):
    n, W, V = case["n_seq"], case["W"], case["vocab"]
    dt = TYPES[case["dtype"]]
    logits = torch.randn(n, W, V, generator=gen, device="cuda") * 2.5
    target = torch.softmax(logits, -1)
    drafts = logits[:, :W - 1] + torch.randn(n, W - 1, V, generator=gen, device="cuda") * 0.4
    del logits
    draft = torch.softmax(drafts, -1)
    pick = draft.cumsum(-1)
    u = torch.rand(n, W - 1, 1, generator=gen, device="cuda")
    tokens = torch.searchsorted(pick, u * pick[..., -1:]).clamp(max=V - 1)[..., 0]
    s = dict(target=target.to(dt), draft=draft.to(dt), tokens=tokens.int(),
             u=torch.rand(n, W - 1, generator=gen, device="cuda"), u_sample=torch.rand(n, generator=gen, device="cuda"),
             n_draft=_ints(np.where(rng.random(n) < 0.2, rng.integers(0, W, n), W - 1)))
    if case["drafts"] == "certain":     # each draft is what a lookup found: no probabilities, high target ones
        s["draft"] = None
        s["tokens"] = torch.where(torch.rand(n, W - 1, generator=gen, device="cuda") < 0.8,
                                  target[:, :W - 1].argmax(-1), tokens).int()
        s["target"] = (target.square() / target.square().sum(-1, keepdim=True)).to(dt)
    new = lambda *shape: torch.empty(*shape, dtype=torch.int32, device="cuda")  # noqa: E731
    s["out"] = (new(n), new(n, W), new(n))
    return s


def _trim_inputs(case, rng, gen):
    n, bs = case["n_seq"], case["bs"]
    lens = _lengths(rng, case)
    need = int((-(-lens // bs)).sum()) + 16
    table, perm, used = _table(rng, lens, bs, case["max_blocks"], 16)
    free = np.full(need, -1)
    free[:need - used] = perm[used:]
    new = lambda m: torch.empty(m, dtype=torch.int32, device="cuda")  # noqa: E731
    return dict(ctx_in=_ints(lens), n_drop=_ints(np.minimum(rng.integers(0, case["drop"] + 1, n), lens)),
                block_table=_ints(table), free_list=_ints(free), free_count=_ints([need - used]), n_blocks=need,
                out=dict(ctx_out=new(n), free_count_out=new(1), info=new(4)))


def _inputs(case, seed):
    rng = np.random.default_rng([int(seed), 78])
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    make = {"rotary": _rotary_inputs, "score": _score_inputs, "chunk": _chunk_inputs, "verify": _verify_inputs,
            "trim": _trim_inputs}[case["op"]]
    return make(case, rng, gen)


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    s["sm_scale"] = 1.0 / math.sqrt(case.get("hd", 1))
    if own and case["op"] in ("rotary", "score"):
        import quantized_kv_cache_append_gb300 as kvq
        s["cache"] = kvq.make_cache(FORMATS[case["fmt"]], case["n_kv"], case["hd"], case["bs"], s["n_blocks"],
                                    s["k"], s["v"], s["ks"], s["vs"])
    if own and case["op"] == "rotary":
        s["rotary"] = kvq.make_rotary(TYPE_IDS[case["dtype"]], case["rot"], case["interleaved"], s["inv_freq"],
                                      pair_axis=s["pair_axis"], n_axes=case["axes"], q_norm=s["q_norm"],
                                      k_norm=s["k_norm"], eps=1e-6)
    if own and case["op"] in ("score", "chunk"):
        import quantized_kv_cache_append_gb300 as kvq
        s["scores"] = kvq.make_scores(softcap=case["cap"], window=case["window"], slopes=s["slopes"],
                                      first=s["first"], last=s.get("last"))
    if own and case["op"] == "score":
        need = kvq.kvq_scored_workspace_bytes(s["cache"], s["scores"], case["n_seq"], case["W"],
                                              case["n_kv"] * case["G"], s["max_ctx"])
        s["workspace"] = torch.empty(need, dtype=torch.uint8, device="cuda")
    return s


# ---------------------------------------------------------------------------
# The library's calls
# ---------------------------------------------------------------------------
def _own(s, case):
    import quantized_kv_cache_append_gb300 as kvq
    if case["op"] == "rotary":
        n_seq, width = s["block_table"].shape
        kvq.check(kvq.kvq_append_rotary(
            s["cache"], s["rotary"], s["q_in"], s["k_in"], s["v_in"], s["q_in"].stride(0), s["k_in"].stride(0),
            s["v_in"].stride(0), case["n_tok"], case["n_q"], s["tok_seq"], s["tok_pos"], s["positions"],
            s["block_table"], n_seq, width, s["q_out"]), "kvq_append_rotary")
        if case["kind"] == "step":
            return dict(q=s["q_out"], k=s["k"], v=s["v"])
        k, v = s["staging"]
        kvq.check(kvq.kvq_compact_f16(s["cache"], s["block_table"][0], case["n_tok"], k, v), "kvq_compact_f16")
        return dict(q=s["q_out"], k=k, v=v)
    if case["op"] == "score":
        n_seq, width = s["block_table"].shape
        kvq.check(kvq.kvq_decode_attn_scored(
            s["cache"], s["scores"], s["q"], n_seq, case["W"], case["n_kv"] * case["G"], s["ctx_lens"],
            s["max_ctx"], s["block_table"], width, s["sm_scale"], s["out"], s["workspace"],
            s["workspace"].numel()), "kvq_decode_attn_scored")
        return s["out"]
    if case["op"] == "chunk":
        kvq.check(kvq.kvq_chunk_attn_scored(
            s["k"], s["v"], case["n_kv"], case["P"], case["hd"], s["scores"], s["q"], case["T"],
            case["n_kv"] * case["G"], s["sm_scale"], s["out"], TYPE_IDS[case["out"]]), "kvq_chunk_attn_scored")
        return s["out"]
    if case["op"] == "verify":
        accepted, tokens, dropped = s["out"]
        V = case["vocab"]
        kvq.check(kvq.kvq_verify_draft(
            s["target"], s["draft"], TYPE_IDS[case["dtype"]], V, V, case["n_seq"], case["W"], V, s["tokens"],
            s["n_draft"], s["u"], s["u_sample"], accepted, tokens, dropped), "kvq_verify_draft")
        return s["out"]
    o = s["out"]
    kvq.check(kvq.kvq_trim_step(
        s["ctx_in"], s["n_drop"], case["n_seq"], case["bs"], s["n_blocks"], s["block_table"], case["max_blocks"],
        s["free_list"], s["free_count"], o["ctx_out"], o["free_count_out"], o["info"]), "kvq_trim_step")
    return dict(o, free_list=s["free_list"])


# ---------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------
def _rotate(x, s, case, weight):
    """Norm of each head, then the rotation of its first `rot` dims: x [n][heads][hd] in 32 bits."""
    rot, half = case["rot"], case["rot"] // 2
    if weight is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * weight
    pos = s["tok_pos"].double()[:, None]
    if s["positions"] is not None:
        pos = s["positions"].double().T[:, s["pair_axis"].long()]
    angle = pos * s["inv_freq"].double()                              # far positions: 64 bits
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    if case["interleaved"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :half], x[..., half:rot]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([turned, x[..., rot:]], -1)


def _hadamard(n, dtype):
    i = torch.arange(n, device="cuda")
    bits = (i[:, None, None] & i[None, :, None]) >> torch.arange(8, device="cuda") & 1
    return (1 - 2 * (bits.sum(-1) % 2)).to(dtype)


def _through_int8(x):
    g = x.view(*x.shape[:-1], -1, 64)
    scale = (g.abs().amax(-1, keepdim=True) / 127).half().float()
    return ((g / scale).round().clamp(-127, 127) * scale).view(x.shape).half()


def _through_q4(x):
    h = _hadamard(x.shape[-1], torch.float32)
    y = (x @ h).view(*x.shape[:-1], -1, 32)
    top = y.gather(-1, y.abs().argmax(-1, keepdim=True))
    scale = (top / -8).half().float()
    code = (y / scale).round().clamp(-8, 7)
    return ((code * scale).view(x.shape) @ h / x.shape[-1]).half()


def _rotary_plain(s, case):
    n, n_q, n_kv, hd, bs = (case[x] for x in ("n_tok", "n_q", "n_kv", "hd", "bs"))
    q = _rotate(s["q_in"].float().view(n, n_q, hd), s, case, s["q_norm"])
    k = _rotate(s["k_in"].float().view(n, n_kv, hd), s, case, s["k_norm"])
    v = s["v_in"].float().view(n, n_kv, hd)
    k = k.half() if case["fmt"] == "f16" else _through_int8(k)
    v = v.half() if case["fmt"] == "f16" else _through_int8(v) if case["fmt"] == "q8" else _through_q4(v)
    if case["kind"] == "prompt":
        return dict(q=q, k=k.transpose(0, 1), v=v.transpose(0, 1))
    pos = s["tok_pos"].long()
    blk = s["block_table"].long()[s["tok_seq"].long(), pos // bs]
    s["k"][blk, :, pos % bs], s["v"][blk, :, pos % bs] = k, v
    return dict(q=q, k=s["k"], v=s["v"])


def _cells(s, case, name, rows, dtype):
    """The table rows' keys or values, dequantised (4-bit values in the rotated basis): [rows][n_kv][cells][hd]."""
    ids = s["block_table"][rows].long().clamp(min=0)
    x, sc = s[name][ids], s["ks" if name == "k" else "vs"]
    if case["fmt"] == "k8v4" and name == "v":
        x = torch.stack([x & 15, x >> 4], -1).flatten(-2).to(dtype) - 8
    else:
        x = x.to(dtype)
    if sc is not None:
        sc = sc[ids].to(dtype)
        x = (x.view(*sc.shape, -1) * sc[..., None]).view(x.shape)
    return x.transpose(1, 2).flatten(2, 3)


def _capped(z, cap):
    return cap * torch.tanh(z / cap) if cap else z


def _softmax_rows(z, seen):
    z = torch.where(seen, z, -torch.inf)
    top = z.amax(-1, keepdim=True)
    p = torch.exp(z - torch.where(top == -torch.inf, 0, top))
    return p / p.sum(-1, keepdim=True).clamp(min=1e-30)


def _score_plain(s, case):
    n, W, n_kv, G, hd = (case[x] for x in ("n_seq", "W", "n_kv", "G", "hd"))
    rows = torch.arange(n, device="cuda")
    k = _cells(s, case, "k", rows, torch.float32)
    cell = torch.arange(k.shape[2], device="cuda")
    q = s["q"].view(n, W, n_kv, G, hd).permute(0, 2, 3, 1, 4)                      # [n][n_kv][G][W][hd]
    pos = s["ctx_lens"].long()[:, None] - W + torch.arange(W, device="cuda")      # [n][W]
    low = torch.zeros_like(pos) if s["first"] is None else s["first"].long()[:, None].expand(n, W)
    if case["window"]:
        low = torch.maximum(low, pos - case["window"] + 1)
    seen = (cell >= low[..., None]) & (cell <= pos[..., None])                     # [n][W][cells]
    z = _capped((q.reshape(n, n_kv, G * W, hd) @ k.transpose(2, 3)).view(n, n_kv, G, W, -1) * s["sm_scale"], case["cap"])
    if s["slopes"] is not None:
        far = (pos[..., None] - cell).abs().float()
        z = z - s["slopes"].view(1, n_kv, G, 1, 1) * far[:, None, None]
    p = _softmax_rows(z, seen[:, None, None])
    o = p.view(n, n_kv, G * W, -1) @ _cells(s, case, "v", rows, torch.float32)
    if case["fmt"] == "k8v4":
        o = o @ _hadamard(hd, torch.float32) / hd
    return o.view(n, n_kv, G, W, hd).permute(0, 3, 1, 2, 4).reshape(n, W, n_kv * G, hd)


def _chunk_plain(s, case):
    T, P, n_kv, G, hd = (case[x] for x in ("T", "P", "n_kv", "G", "hd"))
    q = s["q"].view(T, n_kv, G, hd).permute(1, 2, 0, 3).reshape(n_kv, G * T, hd)
    z = _capped((q @ s["k"].float().transpose(1, 2)).view(n_kv, G, T, P) * s["sm_scale"], case["cap"])
    pos, cell = torch.arange(P - T, P, device="cuda")[:, None], torch.arange(P, device="cuda")
    if s["slopes"] is not None:
        z = z - s["slopes"].view(n_kv, G, 1, 1) * (pos - cell).abs().float()
    high = pos if s["last"] is None else torch.maximum(pos, s["last"].long()[:, None])
    seen = cell <= high
    if s["first"] is not None:
        seen = seen & (cell >= s["first"].long()[:, None])
    if case["window"]:
        seen = seen & (cell > pos - case["window"])
    o = _softmax_rows(z, seen).view(n_kv, G * T, P) @ s["v"].float()
    return o.view(n_kv, G, T, hd).permute(2, 0, 1, 3).reshape(T, n_kv * G, hd).to(TYPES[case["out"]])


def _verify_plain(s, case):
    n, W, V = case["n_seq"], case["W"], case["vocab"]
    i = torch.arange(W - 1, device="cuda")
    tok = s["tokens"].long()
    nd = s["n_draft"].long()
    p_tok = s["target"][:, :W - 1].gather(-1, tok[..., None])[..., 0].double()
    q_tok = torch.ones_like(p_tok) if s["draft"] is None else s["draft"].gather(-1, tok[..., None])[..., 0].double()
    ok = (s["u"].double() * q_tok < p_tok) & (i < nd[:, None])
    a = ok.long().cumprod(1).sum(1)                                                # drafts accepted
    r = torch.arange(n, device="cuda")
    rejected = a < nd
    at = a.clamp(max=W - 2)
    row = s["target"][r, a].float()
    if s["draft"] is None:
        rest = torch.where(torch.arange(V, device="cuda") == tok[r, at][:, None], 0.0, row)
    else:
        rest = (row - s["draft"][r, at].float()).clamp(min=0)
    units = lambda x: (x.double().clamp(0, 1) * UNIT).floor().long()  # noqa: E731
    w = units(torch.where(rejected[:, None], rest, row))
    w = torch.where(w.sum(1, keepdim=True) > 0, w, units(row))
    c = w.cumsum(1)
    total = c[:, -1]
    u = (s["u_sample"].double() * 2 ** 24).floor().long()
    mark = (total >> 24) * u + ((total & (2 ** 24 - 1)) * u >> 24)
    new = torch.where(total > 0, (c <= mark[:, None]).sum(1), -1)
    col = torch.arange(W, device="cuda")
    out = torch.where(col < a[:, None], torch.nn.functional.pad(tok, (0, 1)), -1)
    out = torch.where(col == a[:, None], new[:, None], out)
    return a.int(), out.int(), (nd - a).int()


def _trim_plain(s, case):
    bs, width, n_blocks = case["bs"], case["max_blocks"], s["n_blocks"]
    ctx, drop, count = s["ctx_in"].long(), s["n_drop"].long(), s["free_count"].long()
    bad = ((drop < 0) | (drop > ctx) | (ctx > width * bs)).any()
    left = ctx - drop
    kept = (left + bs - 1) // bs
    back = (ctx + bs - 1) // bs - kept
    end = back.cumsum(0)
    P = end[-1:]
    status = 2 * bad.long() + 8 * ((count < 0) | (count + P > n_blocks)).long()
    ok = status == 0
    j = torch.arange(n_blocks, device="cuda")
    seq = torch.searchsorted(end, j - count, right=True).clamp(max=case["n_seq"] - 1)
    col = (kept[seq] + j - count - (end - back)[seq]).clamp(0, width - 1)
    pushed = s["block_table"].long()[seq, col]
    free = torch.where((j >= count) & (j < count + P) & ok, pushed, s["free_list"].long())
    info = torch.cat([torch.where(ok, drop.sum()[None], 0), torch.zeros_like(P), torch.where(ok, P, 0), status])
    return dict(ctx_out=torch.where(ok, left, ctx).int(), free_count_out=torch.where(ok, count + P, count).int(),
                info=info.int(), free_list=free.int())


def run(state):
    case = state["case"]
    if own:
        return _own(state, case)
    return {"rotary": _rotary_plain, "score": _score_plain, "chunk": _chunk_plain, "verify": _verify_plain,
            "trim": _trim_plain}[case["op"]](state, case)


# ---------------------------------------------------------------------------
# What one pass cannot do without
# ---------------------------------------------------------------------------
def _row_bytes(fmt, hd):
    """A cell's keys and values of one KV head."""
    return {"f16": 4 * hd, "q8": 2 * hd + hd // 16, "k8v4": hd + hd // 32 + hd // 2 + hd // 16}[fmt]


def _mean_seen(lo, hi, case):
    """Cells the mean query token sees."""
    mean = (lo + hi) / 2
    if case.get("first"):
        mean *= 7 / 8
    return min(mean, case["window"]) if case["window"] else mean


def work(case):
    if case["op"] == "rotary":
        n, hd, n_q, n_kv = (case[x] for x in ("n_tok", "hd", "n_q", "n_kv"))
        size = 4 if case["dtype"] == "f32" else 2
        b = n * hd * (size * (n_q + 2 * n_kv) + 4 * n_q) + n * n_kv * _row_bytes(case["fmt"], hd)
        if case["kind"] == "prompt":
            b += n * n_kv * (_row_bytes(case["fmt"], hd) + 4 * hd)
        return dict(bytes=b, flops=10 * n * hd * (n_q + n_kv))
    if case["op"] == "score":
        seen = case["n_seq"] * case["n_kv"] * _mean_seen(case["lo"], case["hi"], case)
        rows = case["W"] * case["G"]
        return dict(bytes=seen * _row_bytes(case["fmt"], case["hd"])
                    + 8 * case["n_seq"] * rows * case["n_kv"] * case["hd"], flops=4 * seen * rows * case["hd"])
    if case["op"] == "chunk":
        T, P, hd, n_kv = case["T"], case["P"], case["hd"], case["n_kv"]
        n_q = n_kv * case["G"]
        seen = _mean_seen(P - T, P, dict(case, first=False))
        if case["docs"] > 1:        # tokens of a later document see their own alone
            seen = min(seen, T / case["docs"] / 2 + (P - T) / 2 / case["docs"])
        cells = min(P, T + (case["window"] or P))
        return dict(bytes=4 * n_kv * cells * hd + 6 * T * n_q * hd, flops=4 * T * n_q * seen * hd)
    if case["op"] == "verify":
        size = 4 if case["dtype"] == "f32" else 2
        rows = 1 if case["drafts"] == "certain" else 1.6
        return dict(bytes=case["n_seq"] * (rows * size * case["vocab"] + 24 * case["W"]), flops=0)
    given = case["n_seq"] * min(case["drop"], (case["lo"] + case["hi"]) / 2) / 2 / case["bs"]
    return dict(bytes=12 * case["n_seq"] + 8 * given + 32, flops=0)


# ---------------------------------------------------------------------------
# The definitions, in 64 bits and written apart from the plain forms
# ---------------------------------------------------------------------------
def _rotary_exact(s, case):
    n, n_q, n_kv, hd, bs, rot = (case[x] for x in ("n_tok", "n_q", "n_kv", "hd", "bs", "rot"))
    if s["positions"] is None:
        pos = s["tok_pos"].cpu().numpy().astype(np.float64)[:, None].repeat(rot // 2, 1)
    else:
        pos = s["positions"].cpu().numpy().astype(np.float64)[s["pair_axis"].cpu().numpy()].T
    turn = torch.polar(torch.ones(1, dtype=torch.float64, device="cuda"),
                       _dev(pos * s["inv_freq"].cpu().numpy().astype(np.float64)))     # [n][rot / 2], complex

    def turned(x, weight):
        x = x.double()
        if weight is not None:
            x = x / (x.pow(2).sum(-1, keepdim=True) / hd + float(np.float32(1e-6))).sqrt() * weight.double()
        first = torch.arange(rot // 2, device="cuda")
        first, second = (2 * first, 2 * first + 1) if case["interleaved"] else (first, first + rot // 2)
        c = torch.complex(x[..., first], x[..., second]) * turn[:, None]
        y = x.clone()
        y[..., first], y[..., second] = c.real, c.imag
        return y

    q = turned(s["q_in"].reshape(n, n_q, hd), s["q_norm"])
    k = turned(s["k_in"].reshape(n, n_kv, hd), s["k_norm"])
    v = s["v_in"].reshape(n, n_kv, hd).double()

    def coded(x, group, divisor, low, high):
        g = x.reshape(n, n_kv, hd // group, group)
        if divisor > 0:
            top = g.abs().max(-1, keepdim=True)[0]
        else:
            top = torch.gather(g, -1, g.abs().max(-1, keepdim=True)[1])
        scale = (top / divisor).float().half().double()
        return (torch.round(g / scale).clamp(low, high) * scale).reshape(n, n_kv, hd)

    if case["fmt"] != "f16":
        k = coded(k, 64, 127, -127, 127)
    if case["fmt"] == "q8":
        v = coded(v, 64, 127, -127, 127)
    if case["fmt"] == "k8v4":
        rotor = torch.ones(1, 1, dtype=torch.float64, device="cuda")
        while rotor.shape[0] < hd:
            rotor = torch.cat([torch.cat([rotor, rotor], 1), torch.cat([rotor, -rotor], 1)], 0)
        v = coded(v @ rotor, 32, -8, -8, 7) @ rotor / hd
    if case["kind"] == "prompt":
        return dict(q=q, k=k.permute(1, 0, 2), v=v.permute(1, 0, 2))
    table, seq, at = (s[x].cpu().numpy() for x in ("block_table", "tok_seq", "tok_pos"))
    blk = torch.from_numpy(table[seq, at // bs].astype(np.int64)).cuda()
    slot = torch.from_numpy(at.astype(np.int64) % bs).cuda()
    pool_k, pool_v = s["k"].double(), s["v"].double()
    pool_k[blk, :, slot], pool_v[blk, :, slot] = k, v
    return dict(q=q, k=pool_k, v=pool_v)


def _weights_exact(z, slope, low, high, pos, cap):
    """Softmax of one head's raw scores z [rows][cells] over cells [low, high] of each row; no cell: zeros."""
    cell = torch.arange(z.shape[1], device=z.device)[None, :]
    if cap:
        z = torch.tanh(z / cap) * cap
    if slope is not None:
        z = z - slope.double() * (cell - pos[:, None]).abs()
    hidden = (cell < low[:, None]) | (cell > high[:, None])
    z = z.masked_fill(hidden, -1e300)
    return torch.softmax(z, -1).masked_fill(hidden, 0.0)


def _score_exact(s, case):
    W, n_kv, G, hd, bs = (case[x] for x in ("W", "n_kv", "G", "hd", "bs"))
    out = torch.zeros(case["n_seq"], W, n_kv, G, hd, dtype=torch.float64, device="cuda")
    rot = torch.ones(1, 1, dtype=torch.float64, device="cuda")
    while rot.shape[0] < hd:
        rot = torch.cat([torch.cat([rot, rot], 1), torch.cat([rot, -rot], 1)], 0)
    for b in range(case["n_seq"]):
        L = int(s["ctx_lens"][b])
        at = s["block_table"][b].long()[:-(-L // bs)]
        pos = torch.arange(L - W, L, device="cuda")
        low = torch.zeros_like(pos)
        if s["first"] is not None:
            low = low + int(s["first"][b])
        if case["window"]:
            low = torch.where(pos + 1 - case["window"] > low, pos + 1 - case["window"], low)
        for h in range(n_kv):
            k = s["k"][at, h].reshape(-1, hd)[:L].double()
            v = s["v"][at, h]
            if case["fmt"] == "k8v4":
                v = torch.stack([v % 16, torch.div(v, 16, rounding_mode="floor")], -1).double() - 8
            v = v.reshape(-1, hd)[:L].double()
            if case["fmt"] != "f16":
                per = 32 if case["fmt"] == "k8v4" else 64
                k = k * s["ks"][at, h].reshape(-1, hd // 64)[:L].double().repeat_interleave(64, 1)
                v = v * s["vs"][at, h].reshape(-1, hd // per)[:L].double().repeat_interleave(per, 1)
            for g in range(G):
                z = s["sm_scale"] * (s["q"][b, :, h * G + g].double() @ k.T)
                slope = None if s["slopes"] is None else s["slopes"][h * G + g]
                o = _weights_exact(z, slope, low, pos, pos, case["cap"]) @ v
                out[b, :, h, g] = o @ rot.T / hd if case["fmt"] == "k8v4" else o
    return out.view(case["n_seq"], W, n_kv * G, hd)


def _chunk_exact(s, case):
    T, P, n_kv, G, hd = (case[x] for x in ("T", "P", "n_kv", "G", "hd"))
    out = torch.zeros(T, n_kv * G, hd, dtype=torch.float64, device="cuda")
    pos = torch.arange(P - T, P, device="cuda")
    low, high = torch.zeros_like(pos), pos.clone()
    if s["first"] is not None:
        low = s["first"].long()
    if s["last"] is not None:
        high = torch.where(s["last"] > high, s["last"].long(), high)
    if case["window"]:
        low = torch.where(pos + 1 - case["window"] > low, pos + 1 - case["window"], low)
    for h in range(n_kv * G):
        z = s["sm_scale"] * (s["q"][:, h].double() @ s["k"][h // G].double().T)
        slope = None if s["slopes"] is None else s["slopes"][h]
        out[:, h] = _weights_exact(z, slope, low, high, pos, case["cap"]) @ s["v"][h // G].double()
    return out


def _verify_exact(s, case):
    n, W, V = case["n_seq"], case["W"], case["vocab"]
    tok, nd = s["tokens"].cpu().numpy(), s["n_draft"].cpu().numpy()
    u, us = s["u"].cpu().numpy().astype(np.float64), s["u_sample"].cpu().numpy().astype(np.float64)
    accepted, out, dropped = np.zeros(n, np.int32), np.full((n, W), -1, np.int32), np.zeros(n, np.int32)

    def units(x):
        return np.floor(np.clip(x.astype(np.float64), 0, 1) * UNIT).astype(np.int64)

    for b in range(n):
        a = 0
        while a < nd[b]:
            x = int(tok[b, a])
            q = 1.0 if s["draft"] is None else float(s["draft"][b, a, x])
            if not u[b, a] * q < float(s["target"][b, a, x]):
                break
            out[b, a] = x
            a += 1
        p = s["target"][b, a].float().cpu().numpy()
        w = units(p)
        if a < nd[b]:
            if s["draft"] is None:
                rest = w.copy()
                rest[int(tok[b, a])] = 0
            else:
                rest = units(np.maximum(p - s["draft"][b, a].float().cpu().numpy(), np.float32(0)))
            w = rest if rest.any() else w
        c = np.cumsum(w)
        mark = int(c[-1]) * int(math.floor(us[b] * 2 ** 24)) >> 24
        out[b, a] = int(np.searchsorted(c, mark, side="right")) if c[-1] else -1
        accepted[b], dropped[b] = a, nd[b] - a
    return tuple(torch.from_numpy(x) for x in (accepted, out, dropped))


def _trim_exact(s, case):
    bs = case["bs"]
    ctx, drop, table, free = (s[x].cpu().numpy().astype(np.int64) for x in ("ctx_in", "n_drop", "block_table",
                                                                           "free_list"))
    count = int(s["free_count"].cpu()[0])
    stack = list(free[:count])
    for b in range(len(ctx)):
        stack.extend(table[b, -(-(ctx[b] - drop[b]) // bs):-(-ctx[b] // bs)])
    free[count:len(stack)] = stack[count:]
    i32 = lambda x: torch.from_numpy(np.asarray(x).astype(np.int32))  # noqa: E731
    return dict(ctx_out=i32(ctx - drop), free_count_out=i32([len(stack)]),
                info=i32([drop.sum(), 0, len(stack) - count, 0]), free_list=i32(free))


def exact(case, seed):
    s = _inputs(case, seed)
    s["sm_scale"] = 1.0 / math.sqrt(case.get("hd", 1))
    return {"rotary": _rotary_exact, "score": _score_exact, "chunk": _chunk_exact, "verify": _verify_exact,
            "trim": _trim_exact}[case["op"]](s, case)
