"""The cache operators' definitions in fp64 on the CPU, key by key and row by row, for the tests of
the HIP kernels. Inputs are CPU tensors; caches come as the values their rows stand for.

Error bounds. A logit is a sum of D products, accumulated in fp32: with u = 2^-24 its error is at
most (D + 2) u scale sum|q k| (twice that is allowed, for the scale folded into the base-2 exponent),
and exp of it adds |logit| u and a few u. A weight is off by that, relative, and so is the sum of
weights: `weight_error`. The sums over the keys add (L + 64) u. Weights that are rounded to bf16
for the product with V add 2^-8, and the output's own rounding 2^-8 of itself for bf16.
"""
import math

import numpy as np
import torch

U = 2.0 ** -24
HALF_STEP = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


def slot_of(table, s, p, bs, num_slots):
    """Cache row of position p, or -1."""
    if p >= table.shape[1] * bs:
        return -1
    page = int(table[s, p // bs])
    if page < 0 or page >= num_slots // bs:
        return -1
    return page * bs + p % bs


def mx_values(codes, scales):
    """fp64 values of MXFP8 rows [.., D] uint8, [.., D/32] uint8."""
    v = codes.view(torch.float8_e4m3fn).float().double()
    e = scales.double() - 127
    return v * torch.pow(2.0, e).repeat_interleave(32, -1)


def mx_encode(x):
    """fp32 rows to codes and scales (the format of shortconv.h)."""
    b = x.float().unflatten(-1, (-1, 32))
    top = b.abs().amax(-1, keepdim=True)
    e = ((top.contiguous().view(torch.int32) >> 23) - 135).clamp(min=-127)
    c = torch.ldexp(b.double(), -e).clamp(-448, 448).float().to(torch.float8_e4m3fn)
    return (c.flatten(-2).view(torch.uint8).contiguous(),
            (e + 127).to(torch.uint8).squeeze(-1).contiguous())


def seen_keys(i, c, t, cap, mask_row):
    """Positions token i of a sequence with c cached keys and t new tokens looks at."""
    c = min(max(c, 0), cap)
    keys = list(range(c))
    for j in range(t):
        if c + j >= cap:
            break
        if mask_row is None:
            ok = j <= i
        else:
            ok = j // 64 < len(mask_row) and (int(mask_row[j // 64]) >> (j % 64)) & 1
        if ok:
            keys.append(c + j)
    return keys


class Rows:
    """Expected rows with bounds: for each token and query head the output, its bound, the
    log-sum-exp, its bound; tokens of no sequence are NaN."""

    def __init__(self, T, Hq, D):
        self.out = np.full((T, Hq, D), np.nan)
        self.bound = np.full((T, Hq, D), np.nan)
        self.lse = np.full((T, Hq), np.nan)
        self.lse_bound = np.full((T, Hq), np.nan)


def weight_error(q, k, scale, logits):
    """Relative error allowed on a weight exp(logit - lse), for these rows."""
    D = q.shape[-1]
    cond = abs(scale) * (np.abs(q) @ np.abs(k).T).max() if len(k) else 0.0
    return 2 * (2 * (D + 2) * U * cond + (np.abs(logits).max() if logits.size else 0) * 2 * U) + 32 * U


def attend(r, t, h, G, q, k, v, scale, dtype):
    """One token's query heads of cache head h over keys k, v [L, D] (fp64 arrays)."""
    for g in range(G):
        hq = h * G + g
        x = (k @ q[hq]) * scale
        if len(k) == 0:
            r.out[t, hq] = 0
            r.bound[t, hq] = 0
            r.lse[t, hq] = -math.inf
            r.lse_bound[t, hq] = 0
            continue
        m = x.max()
        w = np.exp(x - m)
        l = w.sum()
        r.out[t, hq] = (w @ v) / l
        r.lse[t, hq] = m + math.log(l)
        err = weight_error(q[hq:hq + 1], k, scale, x) + (len(k) + 64) * U
        spread = (w @ np.abs(v)) / l
        half = HALF_STEP[dtype]
        rounded = 1.01 * half if dtype == torch.bfloat16 else 0.0
        r.bound[t, hq] = spread * (2 * err + rounded) * 1.02 + np.abs(r.out[t, hq]) * half * 1.02 + 1e-30
        r.lse_bound[t, hq] = 2 * err + 4 * U * abs(r.lse[t, hq])


def attention(q, cu, ctx, table, bs, k, v, num_slots, scale, dtype, mask=None, selected=None):
    """q [T,Hq,D], k/v [num_slots,H,D] fp64 arrays; cu, ctx, table, mask, selected int arrays."""
    T, Hq, D = q.shape
    H = k.shape[1]
    G = Hq // H
    r = Rows(T, Hq, D)
    cap = table.shape[1] * bs
    for s in range(len(cu) - 1):
        c, n = int(ctx[s]), int(cu[s + 1] - cu[s])
        for i in range(n):
            t = int(cu[s]) + i
            for h in range(H):
                if selected is None:
                    pos = seen_keys(i, c, n, cap, None if mask is None else mask[t])
                else:
                    last = min(min(max(c, 0), cap) + i, cap - 1)
                    pos = [p for pb in selected[t, h] if 0 <= pb < table.shape[1]
                           for p in range(pb * bs, (pb + 1) * bs) if p <= last]
                slots = [x for x in (slot_of(table, s, p, bs, num_slots) for p in pos) if x >= 0]
                attend(r, t, h, G, q[t], k[slots, h], v[slots, h], scale, dtype)
    return r


def scores(q, lse, cu, ctx, table, bs, k, num_slots, scale, capacity, scores_in, mask=None):
    """Expected accumulated weights and bounds [N,H,capacity]; NaN where nothing is written."""
    T, Hq, D = q.shape
    H = k.shape[1]
    G = Hq // H
    N = len(cu) - 1
    out = np.full((N, H, capacity), np.nan)
    bound = np.full((N, H, capacity), np.nan)
    cap = table.shape[1] * bs
    for s in range(N):
        c, n = min(max(int(ctx[s]), 0), cap), int(cu[s + 1] - cu[s])
        total = min(c + n, cap, capacity)
        for h in range(H):
            out[s, h, :total] = 0
            bound[s, h, :total] = 0
            if scores_in is not None:
                m = min(c, total)
                out[s, h, :m] = scores_in[s, h, :m]
                bound[s, h, :m] = np.abs(scores_in[s, h, :m]) * (n * G + 4) * U
            for i in range(n):
                t = int(cu[s]) + i
                pos = seen_keys(i, c, n, cap, None if mask is None else mask[t])
                for p in pos:
                    slot = slot_of(table, s, p, bs, num_slots)
                    if p >= total or slot < 0:
                        continue
                    for g in range(G):
                        z = float(lse[t, h * G + g])
                        if z == -math.inf:
                            continue
                        qq = q[t, h * G + g]
                        x = (k[slot, h] @ qq) * scale
                        w = math.exp(x - z)
                        err = weight_error(qq[None], k[slot, h][None], scale, np.array([x, z]))
                        out[s, h, p] += w
                        bound[s, h, p] += w * (err + (n * G + 8) * U)
    return out, bound


def exponent_of(top):
    return -127 if top < 2.0 ** -126 else max(-127, (math.frexp(top)[1] - 1 if math.isfinite(top)
                                                      else 128) - 6)


def codes_of(x, e):
    return np.clip(np.rint(np.ldexp(x, -e)), -127, 127)


def summary(k, cu, ctx, table, bs, num_slots, rebuild, summary_in, exponents_in):
    """Summaries after the call (int8, uint8 arrays)."""
    out, exps = summary_in.copy(), exponents_in.copy()
    H = k.shape[1]
    cap = table.shape[1] * bs
    for s in range(len(cu) - 1):
        c = min(max(int(ctx[s]), 0), cap)
        n = min(c + int(cu[s + 1] - cu[s]), cap)
        for pb in range(0 if rebuild else c // bs, -(-n // bs)):
            slot = slot_of(table, s, pb * bs, bs, num_slots)
            if slot < 0:
                continue
            rows = k[slot:slot + min(bs, n - pb * bs)]
            for h in range(H):
                x = rows[:, h]
                lo = np.where(np.isnan(x), np.inf, x).min(0)
                hi = np.where(np.isnan(x), -np.inf, x).max(0)
                none = lo > hi
                lo, hi = np.where(none, 0, lo), np.where(none, 0, hi)
                e = exponent_of(max(np.abs(lo).max(), np.abs(hi).max()))
                out[slot // bs, h, 0] = codes_of(lo, e)
                out[slot // bs, h, 1] = codes_of(hi, e)
                exps[slot // bs, h] = e + 127
    return out, exps


def select(q, cu, ctx, table, bs, num_slots, summ, exps, sinks, recents, topk):
    """Selected pages [T,H,topk]; -2 in rows that belong to no sequence."""
    T, Hq, D = q.shape
    H = summ.shape[1]
    G = Hq // H
    MB = table.shape[1]
    out = np.full((T, H, topk), -2, np.int32)
    for s in range(len(cu) - 1):
        c = min(max(int(ctx[s]), 0), MB * bs)
        for i in range(int(cu[s + 1] - cu[s])):
            t = int(cu[s]) + i
            P = min((c + i) // bs + 1, MB)
            for h in range(H):
                x = np.nan_to_num(q[t, h * G:(h + 1) * G], nan=0.0, posinf=np.inf, neginf=-np.inf)
                code = codes_of(x, exponent_of(np.abs(x).max()))
                order = []
                for pb in range(P):
                    page = int(table[s, pb])
                    if page < 0 or page >= num_slots // bs:
                        continue
                    if pb < sinks or pb >= P - recents:
                        order.append((-math.inf, pb))
                        continue
                    lo, hi = summ[page, h].astype(np.float64)
                    whole = np.maximum(code * lo, code * hi).sum()
                    score = np.float32(whole) * np.float64(2.0) ** (int(exps[page, h]) - 127)
                    order.append((-float(score), pb))
                picked = sorted(pb for _, pb in sorted(order)[:topk])
                out[t, h] = -1
                out[t, h, :len(picked)] = picked
    return out


def evict(scores_, positions, lens, seen, budget, sinks, recent, table, bs, num_slots, capacity):
    """Per (sequence, head): new length, source index of each kept entry, and the moves as
    (destination slot, source slot) pairs."""
    N, H, _ = scores_.shape
    plan = {}
    for s in range(N):
        n = min(max(int(lens[s]), 0), capacity, table.shape[1] * bs)
        kept = min(n, budget)
        for h in range(H):
            rank = []
            for j in range(n):
                guard = positions[s, h, j] < sinks or positions[s, h, j] >= int(seen[s]) - recent
                f = float(scores_[s, h, j])
                # protected, then numbers from the largest, then NaN; equal ones by index
                rank.append((0, 0, j) if guard else (2, 0, j) if math.isnan(f) else (1, -f, j))
            chosen = sorted(j for _, _, j in sorted(rank)[:kept])
            source = list(range(kept))
            holes = [j for j in range(kept) if j not in set(chosen)]
            for j, f in zip(holes, [x for x in chosen if x >= kept]):
                source[j] = f
            moves = []
            for j in holes:
                a = slot_of(table, s, j, bs, num_slots)
                b = slot_of(table, s, source[j], bs, num_slots)
                if a >= 0 and b >= 0:
                    moves.append((a, b))
            plan[s, h] = (kept, source, moves)
    return plan
