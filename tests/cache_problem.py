"""Random problems over a paged cache, on the CPU as fp64 values and on the GPU as tensors. Every
cache row that no sequence owns holds NaN (MXFP8: NaN codes and scales), so a read of a wrong row
shows in the result."""
import numpy as np
import torch

import cache_reference as ref
import causal_short_convolution_amd as sc

DEV = "cuda:0"
TORCH = {"f32": torch.float32, "bf16": torch.bfloat16}


class Problem:
    """ctx[s] cached keys and drafts[s] new tokens of each sequence, H cache heads read by G query
    heads each. mask: None (chain), "tree" (random trees), "random" (any bits, rows may be empty),
    or an int64 array. spare_blocks: page-table columns behind the used ones. bad: fraction of
    pages whose table entry is outside the pool. behind: query rows behind the last sequence."""

    def __init__(self, seed, dtype="bf16", mx=False, H=2, G=3, D=64, bs=16, ctx=(5,), drafts=(1,),
                 mask=None, words=None, spare_blocks=1, bad=0.0, behind=0, pad=0, scale=None,
                 q_scale=1.5):
        g = np.random.default_rng(seed)
        tg = torch.Generator().manual_seed(seed)
        self.H, self.G, self.D, self.bs, self.mx = H, G, D, bs, mx
        self.dt = TORCH[dtype]
        self.ctx = np.array(ctx, np.int32)
        self.drafts = list(drafts)
        self.N = len(ctx)
        self.cu = np.concatenate([[0], np.cumsum(drafts)]).astype(np.int32)
        self.T = int(self.cu[-1]) + behind
        self.scale = D ** -0.5 if scale is None else scale
        lens = [c + t for c, t in zip(ctx, drafts)]
        need = [-(-n // bs) for n in lens]
        self.pages = sum(need) + 4
        self.num_slots = self.pages * bs + (bs // 2 if bs > 1 else 0)  # a page that does not fit
        perm = g.permutation(self.pages).astype(np.int32)
        MB = max(need) + spare_blocks
        self.table = g.choice(np.array([-1, -7, self.pages, 2 ** 31 - 1], np.int32), (self.N, MB))
        at = 0
        owned = np.zeros(self.num_slots, bool)
        for s, n in enumerate(need):
            self.table[s, :n] = perm[at:at + n]
            at += n
            for p in range(lens[s]):
                owned[self.table[s, p // bs] * bs + p % bs] = True
            for b in range(n):
                if g.random() < bad:
                    self.table[s, b] = g.choice(np.array([-1, self.pages, 2 ** 31 - 1]))
        x = [torch.randn((self.num_slots, H, D), generator=tg) for _ in range(2)]
        own = torch.from_numpy(owned)
        if mx:
            self.stored = []
            for t in x:
                codes, scales = ref.mx_encode(t)
                codes[~own] = 0x7F
                scales[~own] = 0xFF
                self.stored.append((codes, scales))
            self.kv = [ref.mx_values(c, s).numpy() for c, s in self.stored]
            (kc, ks), (vc, vs) = self.stored
            self.dev_kv = [t.to(DEV) for t in (kc, vc, ks, vs)]
            self.key = [self.dev_kv[0], self.dev_kv[2]]
        else:
            self.stored = [t.to(self.dt) for t in x]
            for t in self.stored:
                t[~own] = float("nan")
            self.kv = [t.double().numpy() for t in self.stored]
            self.dev_kv = [t.to(DEV) for t in self.stored]
            self.key = self.dev_kv[:1]
        Hq = H * G
        base = torch.zeros((self.T, Hq * D + pad), dtype=self.dt)
        q = (torch.randn((self.T, Hq * D), generator=tg) * q_scale).to(self.dt)
        base[:, :Hq * D] = q
        self.q = q.double().view(self.T, Hq, D).numpy()
        self.dev_q = base.to(DEV)[:, :Hq * D].view(self.T, Hq, D)
        longest = max(self.drafts) if self.drafts else 1
        words = max(1, -(-longest // 64)) if words is None else words
        self.parents = np.full(self.T, -1, np.int32)
        if isinstance(mask, str):
            m = np.zeros((self.T, words), np.uint64)
            for s in range(self.N):
                for i in range(self.drafts[s]):
                    t = int(self.cu[s]) + i
                    if mask == "tree":
                        self.parents[t] = -1 if i == 0 or g.random() < 0.1 else g.integers(
                            max(0, i - 4), i)
                        p = self.parents[t]
                        if p >= 0:
                            m[t] = m[int(self.cu[s]) + p]
                        if i // 64 < words:
                            m[t, i // 64] |= np.uint64(1 << (i % 64))
                    else:
                        m[t] = g.integers(0, 2 ** 64, words, dtype=np.uint64)
                        if g.random() < 0.3:
                            m[t] = 0
            mask = m.view(np.int64)
        self.mask = mask
        d = lambda a: None if a is None else torch.from_numpy(np.ascontiguousarray(a)).to(DEV)
        self.dev = dict(cu=d(self.cu), ctx=d(self.ctx), table=d(self.table), mask=d(mask))
        self.where = (self.dev["cu"], self.dev["ctx"], self.dev["table"], bs)

    def fresh_out(self, fill=7.0):
        out = torch.full((self.T, self.H * self.G, self.D), fill, dtype=self.dt, device=DEV)
        return out, torch.full((self.T, self.H * self.G), fill, device=DEV)

    def tree_attention(self, out, lse, **kw):
        f = sc.shortconv_tree_attention_mxfp8 if self.mx else sc.shortconv_tree_attention
        f(self.dev_q, *self.where, *self.dev_kv, out, scale=self.scale, mask=self.dev["mask"],
          lse=lse, **kw)

    def block_attention(self, selected, out, lse, **kw):
        f = sc.shortconv_block_attention_mxfp8 if self.mx else sc.shortconv_block_attention
        f(self.dev_q, *self.where, selected, *self.dev_kv, out, scale=self.scale, lse=lse, **kw)

    def cache_scores(self, lse, scores_in, scores_out, **kw):
        f = sc.shortconv_cache_scores_mxfp8 if self.mx else sc.shortconv_cache_scores
        f(self.dev_q, lse, *self.where, *self.key, scores_in, scores_out, scale=self.scale,
          mask=self.dev["mask"], **kw)

    def expected(self, selected=None):
        mask = None if self.mask is None else self.mask.view(np.uint64)
        return ref.attention(self.q, self.cu, self.ctx, self.table, self.bs, *self.kv,
                             self.num_slots, self.scale, self.dt,
                             mask=None if selected is not None else mask, selected=selected)


def check_rows(r, out, lse, fill=7.0):
    """A result against the expected rows; rows of no sequence must hold `fill`."""
    got, z = out.double().cpu().numpy(), None if lse is None else lse.double().cpu().numpy()
    mine = ~np.isnan(r.lse[:, 0]) if len(r.lse) else np.zeros(0, bool)
    assert (got[~mine] == fill).all(), "rows behind the last sequence were written"
    if z is not None:
        assert (z[~mine] == fill).all()
    got, exp, bound = got[mine], r.out[mine], r.bound[mine]
    assert np.isfinite(got).all(), f"{(~np.isfinite(got)).sum()} values not finite"
    off = np.abs(got - exp)
    assert (off <= bound).all(), f"worst {np.nanmax(off / np.maximum(bound, 1e-300)):.3g} of the bound"
    if z is not None:
        z, e, b = z[mine], r.lse[mine], r.lse_bound[mine]
        empty = np.isinf(e)
        assert (z[empty] == e[empty]).all()
        assert (np.abs(z[~empty] - e[~empty]) <= b[~empty]).all(), \
            f"lse off by {np.max(np.abs(z[~empty] - e[~empty]) / b[~empty]):.3g} of the bound"
