"""The operators on the paged KV cache as measurable cases: listed and drawn problems, their inputs,
one pass through each operator, and what the pass cannot do without.

A case is a dict of plain values. ``prepare`` makes what a serving program holds before the call,
``run`` makes one pass: with ``own`` false in elementary torch operations (fp32, fp64 where a whole
number has to come out exact), with ``own`` true through the package's entry points. ``exact`` is
the definition in fp64, written apart from the plain form.

Operators (H kv heads, G query heads per kv head, D head_dim, bs tokens per page):
  verify_tree     the ShortConv K/V step for a tree of drafted tokens (windows along the ancestors)
  tree_attention  attention of drafted tokens (a tree, or one token) over the paged cache
  block_sparse    page summaries refreshed, pages selected per query by an integer score, attention
                  over the selected pages
  cache_scores    attention weight each cached key received, accumulated
  cache_evict     the cache cut down to a budget of entries per sequence and head by those scores
"""
import math

import numpy as np
import torch

own = False

EPS = 1e-6
DEV = "cuda"


# ------------------------------------------------------------------------------------------------
# Cases. Heads and head_dim are those of the decode, mixed and tiny workloads (8 or 16 kv heads of
# 128, fp32 heads of 64); contexts go up to the decode workload's 32768 and the long prefill's
# 131072; pages hold 16 or 64 tokens.
# ------------------------------------------------------------------------------------------------
def listed():
    return [
        # one request, a small tree: a latency-bound step of interactive serving
        dict(name="verify_tree_one", op="verify_tree", dtype="f32", H=8, D=128, W=4, seqs=1,
             draft_lo=7, draft_hi=7),
        # a full serving batch, 4 to 32 drafted tokens per request
        dict(name="verify_tree_batch", op="verify_tree", dtype="bf16", H=16, D=128, W=4, seqs=256,
             draft_lo=4, draft_hi=32),
        # plain decode of one request with a short context: the smallest call
        dict(name="tree_decode_one", op="tree_attention", dtype="bf16", H=8, G=4, D=128, bs=16,
             seqs=1, draft_lo=1, draft_hi=1, ctx_lo=777, ctx_hi=777),
        # the fp32 reference path with odd sizes
        dict(name="tree_fp32", op="tree_attention", dtype="f32", H=2, G=3, D=64, bs=16, seqs=5,
             draft_lo=2, draft_hi=9, ctx_lo=1, ctx_hi=2011),
        # an ordinary serving batch over an MXFP8 cache, trees of 16 drafted tokens
        dict(name="tree_batch_mxfp8", op="tree_attention", dtype="mxfp8", H=8, G=4, D=128, bs=64,
             seqs=64, draft_lo=16, draft_hi=16, ctx_lo=512, ctx_hi=8192),
        # two requests with long contexts and odd trees: the largest read
        dict(name="tree_long", op="tree_attention", dtype="bf16", H=8, G=8, D=128, bs=64, seqs=2,
             draft_lo=31, draft_hi=33, ctx_lo=130000, ctx_hi=131072),
        # decode steps at 32k with 64 pages of 64 tokens kept per query
        dict(name="sparse_decode", op="block_sparse", dtype="bf16", H=8, G=4, D=128, bs=64,
             seqs=32, draft_lo=1, draft_hi=1, ctx_lo=30000, ctx_hi=32767, topk=64, fresh=0),
        # a chunk of a long prompt over an MXFP8 cache, every summary built anew
        dict(name="sparse_chunk_mxfp8", op="block_sparse", dtype="mxfp8", H=8, G=4, D=128, bs=64,
             seqs=1, draft_lo=512, draft_hi=512, ctx_lo=65000, ctx_hi=65000, topk=32, fresh=1),
        # weights of the last 32 prompt tokens, as taken before a prompt is cut down
        dict(name="scores_window", op="cache_scores", dtype="bf16", H=8, G=4, D=128, bs=16,
             seqs=16, draft_lo=32, draft_hi=32, ctx_lo=2000, ctx_hi=8192),
        # weights of one decode step over an MXFP8 cache
        dict(name="scores_decode_mxfp8", op="cache_scores", dtype="mxfp8", H=8, G=4, D=128, bs=64,
             seqs=64, draft_lo=1, draft_hi=1, ctx_lo=1, ctx_hi=8192),
        # a decode batch over its budget by a few tokens: the eviction of every few steps
        dict(name="evict_step", op="cache_evict", dtype="bf16", H=8, D=128, bs=16, seqs=64,
             len_lo=4097, len_hi=4112, budget=4096, sinks=4, recent=128),
        # prompts cut down to a budget once
        dict(name="evict_prompt", op="cache_evict", dtype="bf16", H=8, D=128, bs=64, seqs=8,
             len_lo=2000, len_hi=32768, budget=4096, sinks=4, recent=512),
    ]


def _spread(rng, lo, hi):
    """A whole number from [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)) - 1e-9)))))


def draw(rng):
    op = rng.choice(["verify_tree", "tree_attention", "block_sparse", "cache_scores",
                     "cache_evict"])
    H = rng.choice([1, 2, 5, 8, 16])
    D = rng.choice([64, 128, 128, 256])
    if op == "verify_tree":
        hi = _spread(rng, 1, 64)
        return dict(op=op, dtype=rng.choice(["f32", "bf16"]), H=H, D=D, W=rng.randint(1, 8),
                    seqs=_spread(rng, 1, max(1, 1024 // (hi * max(1, H * D // 2048)))),
                    draft_lo=rng.randint(1, hi), draft_hi=hi)
    bs = rng.choice([16, 32, 64, 128])
    dtype = rng.choice(["f32", "bf16", "bf16", "mxfp8"])
    if op == "cache_evict":
        hi = _spread(rng, 17, 32768)
        seqs = _spread(rng, 1, max(1, min(64, (1 << 27) // (hi * H * D))))
        budget = _spread(rng, 1, hi)
        return dict(op=op, dtype=dtype, H=H, D=D, bs=bs, seqs=seqs, len_lo=rng.randint(1, hi),
                    len_hi=hi, budget=budget, sinks=rng.randint(0, 4),
                    recent=_spread(rng, 1, max(1, budget // 2)))
    G = rng.choice([1, 2, 3, 4, 7, 8, 16])
    row = H * D * (4 if dtype == "f32" else 2)
    if op == "block_sparse":
        chunk = rng.random() < 0.3
        hi = _spread(rng, 1, 65536 if chunk and row < 8192 else 32768)
        drafts = _spread(rng, 2, 256) if chunk else 1
        seqs = 1 if chunk else _spread(rng, 1, max(1, min(32, (1 << 28) // (hi * row))))
        topk = _spread(rng, 2, 64)
        while H * G * D * drafts * topk * bs > 1 << 32:
            topk //= 2
        return dict(op=op, dtype=dtype, H=H, G=G, D=D, bs=bs, seqs=seqs, draft_lo=drafts,
                    draft_hi=drafts, ctx_lo=rng.randint(0, hi), ctx_hi=hi, topk=topk,
                    fresh=rng.randint(0, 1))
    hi = _spread(rng, 1, 32768)
    dhi = _spread(rng, 1, min(64, 256 // G))
    seqs = _spread(rng, 1, max(1, min(64, (1 << 29) // (hi * row))))
    return dict(op=op, dtype=dtype, H=H, G=G, D=D, bs=bs, seqs=seqs, draft_lo=rng.randint(1, dhi),
                draft_hi=dhi, ctx_lo=rng.randint(0, hi), ctx_hi=hi)


def _lengths(lo, hi, n):
    """n whole numbers spread over [lo, hi], the same for every seed (the sizes are the case's)."""
    if n == 1:
        return [hi]
    return [lo + int((hi - lo + 1) * ((i * 0.6180339887498949 + 0.31) % 1.0)) for i in range(n)]


def _sizes(case):
    if case["op"] == "cache_evict":
        return _lengths(case["len_lo"], case["len_hi"], case["seqs"]), None
    drafts = _lengths(case["draft_lo"], case["draft_hi"], case["seqs"])
    if case["op"] == "verify_tree":
        return None, drafts
    return _lengths(case["ctx_lo"], case["ctx_hi"], case["seqs"]), drafts


# ------------------------------------------------------------------------------------------------
# What a pass cannot do without
# ------------------------------------------------------------------------------------------------
def work(case):
    ctx, drafts = _sizes(case)
    H, D = case["H"], case["D"]
    e = {"f32": 4.0, "bf16": 2.0, "mxfp8": 1.0 + 1.0 / 32}[case["dtype"]]
    eq = 4 if case["dtype"] == "f32" else 2
    if case["op"] == "verify_tree":
        W, T, N = case["W"], sum(drafts), case["seqs"]
        rows = 2 * T + N * (W - 1) + T * (W - 1)  # inputs, cache rows, states, snapshots
        return {"bytes": 2 * H * D * (rows * e + (W + 1) * 4), "flops": 2 * T * H * D * (2 * W + 5)}
    if case["op"] == "cache_evict":
        moved = 2 * sum(max(0, n - case["budget"]) * min(1.0, case["budget"] / n) for n in ctx)
        kept = sum(min(n, case["budget"]) for n in ctx)
        return {"bytes": H * (8 * sum(ctx) + 8 * kept + 2 * D * e * moved), "flops": H * sum(ctx)}
    G = case["G"]
    T = sum(drafts)
    keys = sum(c + t for c, t in zip(ctx, drafts))
    pairs = sum(t * (c + t) for c, t in zip(ctx, drafts))
    qo = 2 * T * H * G * D * eq
    if case["op"] == "tree_attention":
        return {"bytes": 2 * H * D * e * keys + qo, "flops": 4 * G * H * D * pairs}
    if case["op"] == "cache_scores":
        return {"bytes": H * D * e * keys + qo / 2 + 8 * H * keys, "flops": 2 * G * H * D * pairs}
    bs, k = case["bs"], case["topk"]
    pages = sum(-(-(c + t) // bs) for c, t in zip(ctx, drafts))
    picked = sum(min(t * k * bs, c + t) for c, t in zip(ctx, drafts))
    fresh = keys if case["fresh"] else sum(min(c % bs + t, c + t) for c, t in zip(ctx, drafts))
    per_query = sum(t * min(k, -(-(c + t) // bs)) * bs for c, t in zip(ctx, drafts))
    score = sum(t * -(-(c + t) // bs) for c, t in zip(ctx, drafts))
    return {"bytes": H * (2 * D * e * picked + D * e * fresh + (2 * D + 1) * pages) + qo,
            "flops": 4 * G * H * D * (per_query + score)}


# ------------------------------------------------------------------------------------------------
# Inputs
# ------------------------------------------------------------------------------------------------
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed * 7919 + 17)


def _randn(shape, gen, dtype, scale=1.0):
    t = torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32)
    return (t * scale).to(dtype)


def _pow2(e, dt):
    """2^e for whole numbers e, from the bits (normal results only)."""
    if dt == torch.float64:
        return ((e.long() + 1023) << 52).view(torch.float64)
    return ((e.int() + 127) << 23).view(torch.float32)


def _mx_encode(x):
    """[..., D] fp32 -> E4M3 codes (uint8) and E8M0 scale bytes per 32 elements."""
    b = x.unflatten(-1, (-1, 32))
    top = b.abs().amax(-1, keepdim=True)
    ex = ((top.view(torch.int32) >> 23) - 135).clamp(min=-127)
    codes = (b * _pow2(-ex, b.dtype)).clamp(-448, 448).to(torch.float8_e4m3fn)
    return (codes.flatten(-2).view(torch.uint8).contiguous(),
            (ex + 127).to(torch.uint8).squeeze(-1).contiguous())


def _cache_rows(slots, H, D, dtype, gen):
    """One cache tensor as a tuple of stored buffers: normalized rows, some channels larger."""
    chan = 1.0 + 0.25 * torch.randn((1, 1, D), generator=gen, device=DEV)
    chan[..., ::17] *= 3.0
    step = max(1, (1 << 26) // (H * D))
    if dtype != "mxfp8":
        out = torch.empty((slots, H, D), device=DEV,
                          dtype=torch.float32 if dtype == "f32" else torch.bfloat16)
        for a in range(0, slots, step):
            n = min(step, slots - a)
            out[a:a + n] = torch.randn((n, H, D), generator=gen, device=DEV) * chan
        return (out,)
    codes = torch.empty((slots, H, D), dtype=torch.uint8, device=DEV)
    scales = torch.empty((slots, H, D // 32), dtype=torch.uint8, device=DEV)
    for a in range(0, slots, step):
        n = min(step, slots - a)
        codes[a:a + n], scales[a:a + n] = _mx_encode(
            torch.randn((n, H, D), generator=gen, device=DEV) * chan)
    return (codes, scales)


def _tables(lens, bs, rng, spare=3):
    """Page tables over one random permutation of a pool, and the pool's number of pages."""
    need = [-(-n // bs) for n in lens]
    total = sum(need) + spare
    perm = rng.permutation(total).astype(np.int32)
    table = np.full((len(lens), max(1, max(need))), -1, np.int32)
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = perm[at:at + n]
        at += n
    return table, total


def _parents(drafts, rng):
    """A random tree per sequence: each token hangs from one of the few before it."""
    out = []
    for n in drafts:
        for i in range(n):
            out.append(-1 if i == 0 else int(rng.integers(max(0, i - 5), i)))
    return out


def _ancestor_bits(drafts, parents):
    """Bit j of row t: drafted token j of the same sequence is t or an ancestor of t."""
    words = max(1, -(-max(drafts) // 64))
    mask = np.zeros((sum(drafts), words), np.uint64)
    at = 0
    for n in drafts:
        for i in range(n):
            p = parents[at + i]
            if p >= 0:
                mask[at + i] = mask[at + p]
            mask[at + i, i // 64] |= np.uint64(1 << (i % 64))
        at += n
    return mask.view(np.int64)


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def _cumulative(drafts):
    return np.concatenate([[0], np.cumsum(drafts)]).astype(np.int32)


def prepare(case, seed):
    gen = _gen(seed)
    rng = np.random.default_rng([seed, 5])
    ctx, drafts = _sizes(case)
    H, D, dtype = case["H"], case["D"], case["dtype"]
    st = dict(case=case, ctx=ctx, drafts=drafts)
    if case["op"] == "verify_tree":
        return _prepare_verify(case, drafts, gen, rng, st)
    tdt = torch.float32 if dtype == "f32" else torch.bfloat16
    bs = case["bs"]
    lens = ctx if drafts is None else [c + t for c, t in zip(ctx, drafts)]
    table, pages = _tables(lens, bs, rng)
    st.update(lens=lens, table=_dev(table), k=_cache_rows(pages * bs, H, D, dtype, gen),
              v=_cache_rows(pages * bs, H, D, dtype, gen))
    cap = table.shape[1] * bs
    if case["op"] == "cache_evict":
        sc = torch.exp(2.0 * torch.randn((case["seqs"], H, cap), generator=gen, device=DEV))
        sc[torch.rand(sc.shape, generator=gen, device=DEV) < 0.1] = 0.0  # never attended to
        pos = torch.arange(cap, dtype=torch.int32, device=DEV).expand(case["seqs"], H, cap)
        st.update(scores=sc, positions=pos.contiguous(), lens_dev=_dev(np.array(lens, np.int32)),
                  seen=_dev(np.array(lens, np.int32)), scores_out=torch.zeros_like(sc),
                  positions_out=torch.full_like(sc, -1, dtype=torch.int32),
                  lens_out=torch.zeros(case["seqs"], dtype=torch.int32, device=DEV))
        return st
    T, Hq = sum(drafts), H * case["G"]
    st.update(q=_randn((T, Hq, D), gen, tdt, 1.5), scale=D ** -0.5,
              cu=_dev(_cumulative(drafts)), ctx_dev=_dev(np.array(ctx, np.int32)),
              out=torch.zeros((T, Hq, D), dtype=tdt, device=DEV),
              lse=torch.zeros((T, Hq), dtype=torch.float32, device=DEV), mask=None)
    if case["op"] != "block_sparse":
        bits = _ancestor_bits(drafts, _parents(drafts, rng))
        st.update(bits=bits, mask=_dev(bits))
    if case["op"] == "cache_scores":
        # what the accumulation starts from, and the log-sum-exp that the attention returned
        st.update(scores=torch.rand((case["seqs"], H, cap), generator=gen, device=DEV),
                  scores_out=torch.zeros((case["seqs"], H, cap), device=DEV))
        st["lse"] = _plain_tree_attention(st, torch.float32)[1]
    if case["op"] == "block_sparse":
        st.update(summary=torch.zeros((pages, H, 2, D), dtype=torch.int8, device=DEV),
                  exponents=torch.zeros((pages, H), dtype=torch.uint8, device=DEV),
                  selected=torch.full((T, H, case["topk"]), -1, dtype=torch.int32, device=DEV))
        _plain_summary(st, [0] * len(lens))
    return st


def _prepare_verify(case, drafts, gen, rng, st):
    H, D, W, N = case["H"], case["D"], case["W"], case["seqs"]
    tdt = torch.float32 if case["dtype"] == "f32" else torch.bfloat16
    T, longest = sum(drafts), max(drafts)
    parents = _parents(drafts, rng)
    slots = T + 5
    st.update(
        parents=parents, parents_dev=_dev(np.array(parents, np.int32)),
        cu=_dev(_cumulative(drafts)), x=[_randn((T, H, D), gen, tdt) for _ in range(2)],
        taps=[_randn((W, H, D), gen, torch.float32, W ** -0.5) for _ in range(2)],
        gamma=[1.0 + 0.1 * torch.randn((D,), generator=gen, device=DEV) for _ in range(2)],
        state=[_randn((N, W - 1, H, D), gen, tdt) for _ in range(2)] if W > 1 else [None, None],
        state_idx=_dev(rng.permutation(N).astype(np.int32)),
        snap=[torch.zeros((N, longest, W - 1, H, D), dtype=tdt, device=DEV) for _ in range(2)]
        if W > 1 else [None, None],
        slot=_dev(rng.permutation(slots)[:T].astype(np.int64)),
        cache=[torch.zeros((slots, H, D), dtype=tdt, device=DEV) for _ in range(2)],
        mask=torch.zeros((T, max(1, -(-longest // 64))), dtype=torch.int64, device=DEV))
    return st


# ------------------------------------------------------------------------------------------------
# The plain forms
# ------------------------------------------------------------------------------------------------
def _plain_rows(stored, slots, dt):
    """Cache rows at the given slots as dt values."""
    if len(stored) == 1:
        return stored[0].index_select(0, slots).to(dt)
    codes = stored[0].index_select(0, slots).view(torch.float8_e4m3fn).to(dt)
    scale = (stored[1].index_select(0, slots).to(torch.int32) << 23).view(torch.float32).to(dt)
    return codes * scale.repeat_interleave(32, dim=-1)


def _plain_slots(st, s, n):
    bs = st["case"]["bs"]
    p = torch.arange(n, device=DEV)
    return st["table"][s].long()[p // bs] * bs + p % bs


def _plain_visible(st, s):
    """[T_s, L_s] truth values: the cached keys, and the drafted ones the mask names."""
    c, t = st["ctx"][s], st["drafts"][s]
    a = int(sum(st["drafts"][:s]))
    j = torch.arange(t, device=DEV)
    own_bits = (st["mask"][a:a + t][:, j // 64] >> (j % 64)) & 1
    return torch.cat([torch.ones((t, c), dtype=torch.bool, device=DEV), own_bits.bool()], 1)


def _plain_scores(q, k, scale):
    """q [t, Hq, D], k [L, H, D] -> [H, t, G, L]"""
    t, hq, d = q.shape
    h = k.shape[1]
    qh = q.view(t, h, hq // h, d).permute(1, 0, 2, 3).reshape(h, t * (hq // h), d) * scale
    return torch.matmul(qh, k.permute(1, 2, 0).contiguous()).view(h, t, hq // h, -1)


def _plain_softmax(x):
    top = x.amax(-1, keepdim=True)
    top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    p = torch.exp(x - top)
    total = p.sum(-1, keepdim=True)
    lse = (top + torch.log(total)).squeeze(-1)
    return p / torch.where(total > 0, total, torch.ones_like(total)), lse


def _plain_tree_attention(st, dt):
    outs, lses = [], []
    a = 0
    for s, t in enumerate(st["drafts"]):
        slots = _plain_slots(st, s, st["lens"][s])
        k, v = _plain_rows(st["k"], slots, dt), _plain_rows(st["v"], slots, dt)
        x = _plain_scores(st["q"][a:a + t].to(dt), k, st["scale"])
        x.masked_fill_(~_plain_visible(st, s)[None, :, None, :], float("-inf"))
        p, lse = _plain_softmax(x)
        h, _, g, n = p.shape
        o = torch.matmul(p.view(h, t * g, n), v.permute(1, 0, 2).contiguous()).view(h, t, g, -1)
        outs.append(o.permute(1, 0, 2, 3).reshape(t, h * g, -1))
        lses.append(lse.permute(1, 0, 2).reshape(t, h * g))
        a += t
    return torch.cat(outs).to(st["q"].dtype), torch.cat(lses).float()


def _plain_cache_scores(st):
    out = st["scores_out"]
    a = 0
    for s, t in enumerate(st["drafts"]):
        n, c = st["lens"][s], st["ctx"][s]
        k = _plain_rows(st["k"], _plain_slots(st, s, n), torch.float32)
        x = _plain_scores(st["q"][a:a + t].float(), k, st["scale"])
        h, _, g, _ = x.shape
        lse = st["lse"][a:a + t].view(t, h, g).permute(1, 0, 2)[..., None]
        w = torch.exp(x - lse) * _plain_visible(st, s)[None, :, None, :]
        out[s, :, :n] = w.sum((1, 2))
        out[s, :, :c] += st["scores"][s, :, :c]
        a += t
    return out


def _plain_summary(st, starts):
    """Per page and head the rows' minimum and maximum, as int8 codes with one exponent."""
    bs = st["case"]["bs"]
    for s, n in enumerate(st["lens"]):
        first = starts[s] // bs
        pages = -(-n // bs)
        if pages <= first:
            continue
        p = torch.arange(first * bs, pages * bs, device=DEV)
        slots = st["table"][s].long()[p // bs] * bs + p % bs
        rows = _plain_rows(st["k"], slots, torch.float32)
        live = (p < n)[:, None, None]
        top = torch.where(live, rows, float("-inf")).unflatten(0, (-1, bs)).amax(1)
        low = torch.where(live, rows, float("inf")).unflatten(0, (-1, bs)).amin(1)
        both = torch.stack([low, top], 2)  # [pages, H, 2, D]
        ex = ((both.abs().amax((2, 3)).view(torch.int32) >> 23) - 133).clamp(min=-127)
        codes = (both * _pow2(-ex, both.dtype)[..., None, None]).round().clamp(-127, 127)
        ids = st["table"][s, first:pages].long()
        st["summary"][ids] = codes.to(torch.int8)
        st["exponents"][ids] = (ex + 127).to(torch.uint8)


def _plain_block_sparse(st):
    case = st["case"]
    bs, topk, H, G, D = case["bs"], case["topk"], case["H"], case["G"], case["D"]
    _plain_summary(st, [0] * len(st["ctx"]) if case["fresh"] else st["ctx"])
    a = 0
    for s, t in enumerate(st["drafts"]):
        n, c = st["lens"][s], st["ctx"][s]
        pages = -(-n // bs)
        ids = st["table"][s, :pages].long()
        q = st["q"][a:a + t].float().view(t, H, G, D)
        ex = ((q.abs().amax((2, 3)).view(torch.int32) >> 23) - 133).clamp(min=-127)
        code = (q * _pow2(-ex, q.dtype)[..., None, None]).round().clamp(-127, 127).double()
        up = code.clamp(min=0).sum(2).permute(1, 0, 2)    # [H, t, D]
        down = code.clamp(max=0).sum(2).permute(1, 0, 2)
        box = st["summary"][ids].double().permute(1, 2, 3, 0).contiguous()  # [H, 2, D, pages]
        whole = torch.matmul(down, box[:, 0]) + torch.matmul(up, box[:, 1])  # exact
        size = _pow2(st["exponents"][ids].int().t() - 127, torch.float64)
        score = whole.float().double() * size[:, None, :]
        page = torch.arange(pages, device=DEV)
        count = (c + torch.arange(t, device=DEV)) // bs + 1
        seen = page[None] < count[:, None]
        forced = seen & ((page[None] < 1) | (page[None] >= count[:, None] - 1))
        score = torch.where(forced, float("inf"), torch.where(seen, score, float("-inf")))
        order = torch.sort(score, dim=-1, descending=True, stable=True).indices[..., :topk]
        picked = torch.where(torch.arange(order.shape[-1], device=DEV) < count[:, None], order,
                             pages)
        picked = picked.sort(-1).values
        sel = torch.full((H, t, topk), -1, dtype=torch.int32, device=DEV)
        sel[..., :picked.shape[-1]] = torch.where(picked < pages, picked, -1).int()
        st["selected"][a:a + t] = sel.permute(1, 0, 2)
        # attention over the selected pages, in pieces that bound the gathered rows
        step = max(1, (1 << 28) // (H * topk * bs * D))
        for i in range(0, t, step):
            m = min(step, t - i)
            pg = st["selected"][a + i:a + i + m].long()  # [m, H, topk]
            pos = (pg[..., None] * bs + torch.arange(bs, device=DEV)).flatten(2)
            ok = (pg >= 0)[..., None].expand(-1, -1, -1, bs).flatten(2)
            ok = ok & (pos <= c + torch.arange(i, i + m, device=DEV)[:, None, None])
            slot = st["table"][s].long()[pos.clamp(min=0) // bs] * bs + pos % bs
            flat = torch.where(ok, slot, 0) * H + torch.arange(H, device=DEV)[:, None]

            def rows(stored):
                per_head = tuple(b.flatten(0, 1) for b in stored)
                return _plain_rows(per_head, flat.flatten(), torch.float32).view(m * H, -1, D)

            k = rows(st["k"])
            x = torch.matmul(q[i:i + m].reshape(m * H, G, D) * st["scale"],
                             k.transpose(1, 2).contiguous())
            x.masked_fill_(~ok.view(m * H, 1, -1), float("-inf"))
            del k
            p, lse = _plain_softmax(x)
            o = torch.matmul(p, rows(st["v"]))
            st["out"][a + i:a + i + m] = o.view(m, H * G, D).to(st["out"].dtype)
            st["lse"][a + i:a + i + m] = lse.view(m, H * G)
        a += t
    return st["summary"], st["exponents"], st["selected"], st["out"], st["lse"]


def _plain_evict(st):
    case = st["case"]
    H, bs, budget = case["H"], case["bs"], case["budget"]
    for s, n in enumerate(st["lens"]):
        pos = st["positions"][s, :, :n]
        sc = st["scores"][s, :, :n]
        kept = min(n, budget)
        src = torch.arange(kept, device=DEV).expand(H, kept).clone()
        if n > budget:
            guard = (pos < case["sinks"]) | (pos >= n - case["recent"])
            rank = torch.sort(torch.where(guard, float("inf"), sc), dim=-1, descending=True,
                              stable=True).indices[:, :budget]
            keep = torch.zeros((H, n), dtype=torch.bool, device=DEV).scatter_(1, rank, True)
            # holes below the budget, ascending, take the kept entries above it, ascending
            src[~keep[:, :budget]] = (keep[:, budget:].nonzero()[:, 1] + budget)
        slots = _plain_slots(st, s, n)
        head = torch.arange(H, device=DEV)[:, None]
        dst = torch.arange(kept, device=DEV)
        moved = src != dst
        to = (slots[dst].expand(H, kept) * H + head)[moved]
        frm = (slots[src] * H + head)[moved]
        for buf in st["k"] + st["v"]:
            flat = buf.view(-1, buf.shape[-1])
            flat[to] = flat[frm]
        st["scores_out"][s, :, :kept] = sc.gather(1, src)
        st["positions_out"][s, :, :kept] = pos.gather(1, src)
        st["lens_out"][s] = kept
    return st["scores_out"], st["positions_out"], st["lens_out"], st["k"], st["v"]


def _plain_verify(st):
    case = st["case"]
    W, H, D = case["W"], case["H"], case["D"]
    T = sum(st["drafts"])
    seq = torch.repeat_interleave(torch.arange(case["seqs"], device=DEV),
                                  (st["cu"][1:] - st["cu"][:-1]).long())
    start = st["cu"].long()[seq]
    parent = st["parents_dev"].long()
    state_row = st["state_idx"].long()[seq]
    # window row k of token t: an index into the new rows, or into the state rows behind them
    at = torch.arange(T, device=DEV)
    depth = torch.full((T,), W - 2, device=DEV)  # the next state row once the root is passed
    rows = [at]
    inside = torch.ones((T,), dtype=torch.bool, device=DEV)
    for _ in range(W - 1):
        up = parent[at.clamp(max=T - 1)]
        climb = inside & (up >= 0)
        past = T + state_row * (W - 1) + depth
        depth = torch.where(climb, depth, depth - 1)
        at = torch.where(climb, start + up, past)
        inside = climb
        rows.insert(0, at)
    window = torch.stack(rows)  # [W, T], oldest first
    for i in range(2):
        x = st["x"][i]
        pool = x if W == 1 else torch.cat([x, st["state"][i].view(-1, H, D)])
        win = pool[window]  # [W, T, H, D]
        c = (win.float() * st["taps"][i][:, None]).sum(0)
        y = c / torch.sqrt(c.square().mean(-1, keepdim=True) + EPS) * st["gamma"][i]
        st["cache"][i][st["slot"]] = y.to(x.dtype)
        if W > 1:
            st["snap"][i][seq, torch.arange(T, device=DEV) - start] = win[1:].transpose(0, 1)
    words = st["mask"].shape[1]
    mask = torch.zeros_like(st["mask"])
    local = torch.arange(T, device=DEV) - start
    bit = torch.zeros_like(mask).scatter_(1, (local // 64)[:, None],
                                          torch.ones_like(local)[:, None] << (local % 64)[:, None])
    at, alive = torch.arange(T, device=DEV), torch.ones((T,), dtype=torch.bool, device=DEV)
    for _ in range(max(st["drafts"])):
        mask |= torch.where(alive[:, None], bit[at], 0)
        up = parent[at]
        alive = alive & (up >= 0)
        at = torch.where(alive, start + up, at)
    st["mask"].copy_(mask.view(T, words))
    return st["cache"], st["snap"], st["mask"]


# ------------------------------------------------------------------------------------------------
# One pass
# ------------------------------------------------------------------------------------------------
def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_plain(st):
    op = st["case"]["op"]
    if op == "verify_tree":
        cache, snap, mask = _plain_verify(st)
        return _verify_outputs(st, cache, snap, mask)
    if op == "tree_attention":
        return _plain_tree_attention(st, torch.float32)
    if op == "block_sparse":
        return _plain_block_sparse(st)
    if op == "cache_scores":
        return _plain_cache_scores(st)
    return _plain_evict(st)


def _verify_outputs(st, cache, snap, mask):
    return (cache[0], cache[1], mask) if st["case"]["W"] == 1 else (*cache, *snap, mask)


def _run_own(st):
    import causal_short_convolution_amd as sc
    case = st["case"]
    op = case["op"]
    mx = case["dtype"] == "mxfp8"
    if op == "verify_tree":
        sc.shortconv_kv_verify_tree(*st["x"], st["cu"], st["parents_dev"], *st["taps"],
                                    *st["gamma"], EPS, *st["state"], st["state_idx"], *st["snap"],
                                    st["slot"], *st["cache"], mask=st["mask"])
        return _verify_outputs(st, st["cache"], st["snap"], st["mask"])
    if op == "cache_evict":
        args = (st["scores"], st["positions"], st["lens_dev"], st["seen"], case["budget"],
                st["table"], case["bs"])
        outs = (st["scores_out"], st["positions_out"], st["lens_out"])
        kw = dict(sinks=case["sinks"], recent=case["recent"])
        if mx:
            sc.shortconv_cache_evict_mxfp8(*args, st["k"][0], st["v"][0], st["k"][1], st["v"][1],
                                           *outs, **kw)
        else:
            sc.shortconv_cache_evict(*args, st["k"][0], st["v"][0], *outs, **kw)
        return (*outs, st["k"], st["v"])
    where = (st["cu"], st["ctx_dev"], st["table"], case["bs"])
    kv = (st["k"][0], st["v"][0], st["k"][1], st["v"][1]) if mx else (st["k"][0], st["v"][0])
    if op == "tree_attention":
        f = sc.shortconv_tree_attention_mxfp8 if mx else sc.shortconv_tree_attention
        f(st["q"], *where, *kv, st["out"], scale=st["scale"], mask=st["mask"], lse=st["lse"])
        return st["out"], st["lse"]
    if op == "cache_scores":
        f = sc.shortconv_cache_scores_mxfp8 if mx else sc.shortconv_cache_scores
        f(st["q"], st["lse"], *where, *st["k"], st["scores"], st["scores_out"], scale=st["scale"],
          mask=st["mask"])
        return st["scores_out"]
    f = sc.shortconv_block_summary_mxfp8 if mx else sc.shortconv_block_summary
    f(*st["k"], *where, st["summary"], st["exponents"], rebuild=bool(case["fresh"]))
    sc.shortconv_block_select(st["q"], *where, st["summary"], st["exponents"], st["selected"],
                              sink_blocks=1, recent_blocks=1)
    f = sc.shortconv_block_attention_mxfp8 if mx else sc.shortconv_block_attention
    f(st["q"], *where, st["selected"], *kv, st["out"], scale=st["scale"], lse=st["lse"])
    return st["summary"], st["exponents"], st["selected"], st["out"], st["lse"]


# ------------------------------------------------------------------------------------------------
# The definitions in 64 bits
# ------------------------------------------------------------------------------------------------
def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "verify_tree":
        return _exact_verify(case, st)
    if op == "cache_evict":
        return _exact_evict(case, st)
    if op == "block_sparse":
        return _exact_sparse(case, st)
    H, G, D = case["H"], case["G"], case["D"]
    first = _cumulative(st["drafts"])
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.zeros(st["lse"].shape, dtype=torch.float64, device=DEV)
    weight = torch.zeros((case["seqs"], H, st["table"].shape[1] * case["bs"]),
                         dtype=torch.float64, device=DEV)
    for s in range(case["seqs"]):
        c, n, a, b = st["ctx"][s], st["lens"][s], int(first[s]), int(first[s + 1])
        see = np.ones((b - a, n), bool)
        for i in range(b - a):
            for j in range(b - a):
                word = int(st["bits"][a + i, j // 64]) & (2 ** 64 - 1)
                see[i, c + j] = bool(word >> (j % 64) & 1)
        see = _dev(see)
        for h in range(H):
            k, v = (_exact_rows(st, name, s, h, n) for name in ("k", "v"))
            qh = st["q"][a:b, h * G:(h + 1) * G].double()
            x = torch.matmul(qh.reshape(-1, D), k.t().contiguous()).view(b - a, G, n) * st["scale"]
            if op == "cache_scores":
                w = torch.exp(x - st["lse"][a:b, h * G:(h + 1) * G, None].double())
                weight[s, h, :n] = (w * see[:, None]).sum((0, 1))
                weight[s, h, :c] += st["scores"][s, h, :c].double()
                continue
            x = x.masked_fill(~see[:, None], float("-inf"))
            z = torch.logsumexp(x, -1)
            lse[a:b, h * G:(h + 1) * G] = z
            w = torch.exp(x - torch.nan_to_num(z, neginf=0.0)[..., None])
            out[a:b, h * G:(h + 1) * G] = torch.matmul(w.view(-1, n), v).view(b - a, G, D)
    return weight if op == "cache_scores" else (out, lse)


def _exact_rows(st, name, s, h, n):
    """Rows 0..n-1 of head h of sequence s in fp64."""
    bs = st["case"]["bs"]
    pages = st["table"][s, :-(-n // bs)].long()
    buf = st[name]
    part = buf[0].unflatten(0, (-1, bs))[pages, :, h].flatten(0, 1)[:n]
    if len(buf) == 1:
        return part.double()
    ex = buf[1].unflatten(0, (-1, bs))[pages, :, h].flatten(0, 1)[:n].int() - 127
    val = part.view(torch.float8_e4m3fn).double().unflatten(-1, (-1, 32))
    return (val * _pow2(ex, val.dtype)[..., None]).flatten(-2)


def _exact_codes(x):
    """Whole numbers in [-127, 127] and the exponent of one group of fp64 values."""
    top = float(x.abs().max())
    e = -127 if top < 2.0 ** -126 else max(-127, math.frexp(top)[1] - 1 - 6)
    return torch.round(x * 2.0 ** -e).clamp(-127, 127)


def _exact_sparse(case, st):
    H, G, D, bs, topk = case["H"], case["G"], case["D"], case["bs"], case["topk"]
    summary, exps = st["summary"].clone(), st["exponents"].clone()
    sel = torch.full(st["selected"].shape, -1, dtype=torch.int32)
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.zeros(st["lse"].shape, dtype=torch.float64, device=DEV)
    first = _cumulative(st["drafts"])
    if sum(st["drafts"]) * H > 8192:
        return None
    for s in range(case["seqs"]):
        c, n, a, b = st["ctx"][s], st["lens"][s], int(first[s]), int(first[s + 1])
        pages = -(-n // bs)
        ids = st["table"][s, :pages].long()
        for h in range(H):
            k, v = (_exact_rows(st, name, s, h, n) for name in ("k", "v"))
            pad = pages * bs - n
            low = torch.nn.functional.pad(k, (0, 0, 0, pad), value=math.inf).view(pages, bs, D)
            top = torch.nn.functional.pad(k, (0, 0, 0, pad), value=-math.inf).view(pages, bs, D)
            box = torch.stack([low.min(1).values, top.max(1).values], 1)  # [pages, 2, D]
            big = box.abs().amax((1, 2))
            e = (torch.frexp(big).exponent.int() - 1 - 6).clamp(min=-127)
            e = torch.where(big < 2.0 ** -126, -127, e)
            code = torch.round(box * _pow2(-e, box.dtype)[:, None, None]).clamp(-127, 127)
            summary[ids, h] = code.to(torch.int8)
            exps[ids, h] = (e + 127).to(torch.uint8)
            allowed = torch.zeros((b - a, n), dtype=torch.bool, device=DEV)
            rank = torch.zeros((b - a, pages), dtype=torch.float64, device=DEV)
            for i in range(b - a):
                qc = _exact_codes(st["q"][a + i, h * G:(h + 1) * G].double())
                for g in range(G):
                    rank[i] += torch.maximum(qc[g] * code[:, 0], qc[g] * code[:, 1]).sum(-1)
            rank = (rank.float().double() * _pow2(e, rank.dtype)).cpu().numpy()
            for i in range(b - a):
                m = (c + i) // bs + 1
                r = rank[i, :m].copy()
                r[0] = r[m - 1] = np.inf
                best = np.sort(np.lexsort((np.arange(m), -r))[:topk])
                sel[a + i, h, :len(best)] = torch.from_numpy(best.astype(np.int32))
                grid = torch.zeros(pages, dtype=torch.bool)
                grid[torch.from_numpy(best)] = True
                live = grid.to(DEV).repeat_interleave(bs)[:n]
                live[c + i + 1:] = False
                allowed[i] = live
            qh = st["q"][a:b, h * G:(h + 1) * G].double()
            x = torch.matmul(qh.reshape(-1, D), k.t().contiguous()).view(b - a, G, n) * st["scale"]
            x.masked_fill_(~allowed[:, None], float("-inf"))
            z = torch.logsumexp(x, -1)
            lse[a:b, h * G:(h + 1) * G] = z
            out[a:b, h * G:(h + 1) * G] = torch.matmul(
                torch.exp(x - z[..., None]).view(-1, n), v).view(b - a, G, D)
    return summary, exps, sel.to(DEV), out, lse


def _exact_evict(case, st):
    bs, H = case["bs"], case["H"]
    score, pos = st["scores"].cpu().numpy(), st["positions"].cpu().numpy()
    s_out = np.zeros(score.shape)
    p_out = np.full(pos.shape, -1, np.int32)
    table = st["table"].cpu().numpy().astype(np.int64)
    moves = []
    for s, n in enumerate(st["lens"]):
        kept = min(n, case["budget"])
        for h in range(H):
            index = np.arange(n)
            guard = (pos[s, h, :n] < case["sinks"]) | (pos[s, h, :n] >= n - case["recent"])
            order = np.lexsort((index, np.where(guard, -np.inf, -score[s, h, :n].astype(float))))
            chosen = np.sort(order[:kept])
            holes = np.setdiff1d(index[:kept], chosen)
            source = index[:kept].copy()
            source[holes] = chosen[chosen >= kept]
            s_out[s, h, :kept] = score[s, h, source]
            p_out[s, h, :kept] = pos[s, h, source]
            for d, f in ((holes, source[holes]),):
                slot = [table[s, x // bs] * bs + x % bs for x in (d, f)]
                moves.append(np.stack([slot[0], slot[1], np.full(len(d), h)], 1))
    moves = torch.from_numpy(np.concatenate(moves)).to(DEV)
    kv = []
    for name in ("k", "v"):
        bufs = tuple(b.clone() for b in st[name])
        for b in bufs:
            b[moves[:, 0], moves[:, 2]] = b[moves[:, 1], moves[:, 2]]
        kv.append(bufs)
    lens = torch.tensor([min(n, case["budget"]) for n in st["lens"]], dtype=torch.int32)
    return _dev(s_out), _dev(p_out), lens.to(DEV), kv[0], kv[1]


def _exact_verify(case, st):
    W, H, D = case["W"], case["H"], case["D"]
    first = _cumulative(st["drafts"])
    index = st["state_idx"].tolist()
    T = sum(st["drafts"])
    source = torch.zeros((T, W), dtype=torch.long)  # rows of [new rows, state rows]
    bits = np.zeros(tuple(st["mask"].shape), np.uint64)
    where = []
    for s, t in enumerate(st["drafts"]):
        for i in range(t):
            path, j = [], i
            while j >= 0:
                path.append(int(first[s]) + j)
                bits[first[s] + i, j // 64] |= np.uint64(1 << (j % 64))
                j = st["parents"][int(first[s]) + j]
            past = [T + index[s] * (W - 1) + r for r in range(W - 1)]
            line = past + path[::-1]
            source[first[s] + i] = torch.tensor(line[len(line) - W:])
            where.append((s, i))
    where = torch.tensor(where, device=DEV)
    source = source.to(DEV)
    res = []
    snaps = []
    for i in range(2):
        rows = st["x"][i].double()
        if W > 1:
            rows = torch.cat([rows, st["state"][i].double().view(-1, H, D)])
        c = torch.zeros((T, H, D), dtype=torch.float64, device=DEV)
        for k in range(W):
            c += st["taps"][i][k].double() * rows[source[:, k]]
        norm = torch.rsqrt((c * c).sum(-1, keepdim=True) / D + EPS)
        cache = torch.zeros(st["cache"][i].shape, dtype=torch.float64, device=DEV)
        cache[st["slot"]] = c * norm * st["gamma"][i].double()
        res.append(cache)
        if W > 1:
            snap = torch.zeros(st["snap"][i].shape, dtype=torch.float64, device=DEV)
            snap[where[:, 0], where[:, 1]] = rows[source[:, 1:]]
            snaps.append(snap)
    return (*res, *snaps, _dev(bits.view(np.int64)))
