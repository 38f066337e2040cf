"""Accumulated attention weight and eviction by it, against the definitions."""
import numpy as np
import pytest
import torch

import cache_reference as ref
import causal_short_convolution_amd as sc
from cache_problem import DEV, Problem

pytestmark = pytest.mark.gpu

KINDS = [("f32", False), ("bf16", False), ("bf16", True), ("f32", True)]


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def check_scores(p, capacity=None, start=True, in_place=False, lse=None):
    cap = p.table.shape[1] * p.bs + 3 if capacity is None else capacity
    r = p.expected()
    if lse is None:
        lse = torch.from_numpy(np.nan_to_num(r.lse, nan=0.0, neginf=-np.inf).astype(np.float32))
    g = np.random.default_rng(1)
    init = g.random((p.N, p.H, cap)).astype(np.float32)
    src = torch.from_numpy(init).to(DEV) if start else None
    out = src if in_place else torch.full((p.N, p.H, cap), -9.0, device=DEV)
    p.cache_scores(lse.to(DEV), src, out)
    torch.cuda.synchronize()
    mask = None if p.mask is None else p.mask.view(np.uint64)
    want, bound = ref.scores(p.q, lse.double().numpy(), p.cu, p.ctx, p.table, p.bs, p.kv[0],
                             p.num_slots, p.scale, cap, init if start else None, mask)
    got = out.double().cpu().numpy()
    left = np.isnan(want)
    keep = init if in_place else np.full_like(got, -9.0)
    assert (got[left] == keep[left]).all(), "entries behind the sequence were written"
    off = np.abs(got - want)[~left]
    assert (off <= bound[~left] + 1e-30).all(), \
        f"worst {np.max(off / (bound[~left] + 1e-30)):.3g} of the bound"
    return out


@pytest.mark.parametrize("dtype,mx", KINDS)
@pytest.mark.parametrize("H,G,D,bs", [(1, 1, 64, 16), (2, 4, 128, 16), (3, 2, 256, 8), (2, 20, 64, 1)])
def test_scores(dtype, mx, H, G, D, bs):
    check_scores(Problem(1, dtype, mx, H, G, D, bs, ctx=(40, 0, 129, 7), drafts=(3, 5, 1, 0),
                         mask="tree", behind=1))


@pytest.mark.parametrize("dtype,mx", KINDS)
@pytest.mark.parametrize("mask", [None, "random"])
def test_scores_masks(dtype, mx, mask):
    """Empty rows (lse -inf) add nothing; unseen drafts stay zero."""
    check_scores(Problem(2, dtype, mx, 2, 2, 64, 16, ctx=(0, 20, 33), drafts=(9, 70, 2), mask=mask,
                         bad=0.2))


def test_scores_without_a_start_in_place_and_short_capacity():
    p = Problem(3, "bf16", False, 2, 3, 64, 16, ctx=(50, 10), drafts=(4, 2))
    check_scores(p, start=False)
    check_scores(p, in_place=True)
    check_scores(p, capacity=20)


@pytest.mark.parametrize("rows", [1, 40, 200])
def test_scores_many_rows(rows):
    check_scores(Problem(4, "bf16", False, 1, 4, 128, 16, ctx=(60,), drafts=(rows,), mask="tree"))


def test_scores_sum_to_the_rows():
    """Each row spreads a weight of 1 over its keys: with the lse of the attention itself the sums
    over the positions count the rows."""
    p = Problem(5, "bf16", False, 2, 4, 128, 16, ctx=(1000, 77), drafts=(6, 1), mask="tree")
    out, lse = p.fresh_out()
    p.tree_attention(out, lse)
    cap = p.table.shape[1] * p.bs
    got = torch.zeros((2, 2, cap), device=DEV)
    p.cache_scores(lse, None, got)
    torch.cuda.synchronize()
    rows = torch.tensor([[24.0, 24.0], [4.0, 4.0]], dtype=torch.float64)
    # each weight is off by at most the relative error the bound of test_scores allows; 1e-4 covers
    # 2 (2 (D + 2) 2^-24 sum|q k| scale) for these inputs (sum|q k| scale < 60)
    assert (got.double().sum(-1).cpu() - rows).abs().max() < 24 * 1e-4


def test_scores_nan_in_masked_places_do_not_leak():
    p = Problem(6, "bf16", False, 1, 2, 64, 16, ctx=(10,), drafts=(4,), mask=np.array(
        [[1], [3], [5], [9]], np.int64))
    lse = torch.zeros((4, 2), device=DEV)
    clean = torch.zeros((1, 1, 32), device=DEV)
    p.cache_scores(lse, None, clean)
    slot = int(p.table[0, 0]) * 16 + 12  # draft 2: token 2 alone looks at it
    p.dev_kv[0][slot] = float("nan")
    out = torch.zeros((1, 1, 32), device=DEV)
    p.cache_scores(lse, None, out)
    torch.cuda.synchronize()
    keep = [i for i in range(32) if i != 12]
    assert torch.equal(out[..., keep], clean[..., keep]) and bool(out[0, 0, 12].isnan())


# ------------------------------------------------------------------------------------------------
# Eviction
# ------------------------------------------------------------------------------------------------
class Cut:
    """An eviction problem: scores with ties and special values, positions as they are after an
    earlier eviction."""

    def __init__(self, seed, dtype="bf16", mx=False, H=2, D=64, bs=16, lens=(40,), budget=16,
                 sinks=2, recent=4, cap_extra=5, bad=0.0, special=True, shuffled=True):
        g = np.random.default_rng(seed)
        self.p = Problem(seed, dtype, mx, H, 1, D, bs, ctx=lens, drafts=[0] * len(lens), bad=bad)
        self.N, self.H = len(lens), H
        self.cap = max(lens) + cap_extra
        self.lens = np.array(lens, np.int32)
        self.seen = self.lens + (7 if shuffled else 0)
        self.scores = (g.integers(0, 12, (self.N, H, self.cap)) / 4).astype(np.float32)
        if special:
            for v in (np.nan, np.inf, -np.inf, -0.0, -1.5):
                self.scores[g.random(self.scores.shape) < 0.05] = v
        self.positions = np.zeros((self.N, H, self.cap), np.int32)
        for s in range(self.N):
            for h in range(H):
                n = int(self.seen[s])
                pos = g.permutation(n)[:lens[s]] if shuffled else np.arange(lens[s])
                self.positions[s, h, :lens[s]] = pos
        self.budget, self.sinks, self.recent = budget, sinks, recent

    def run(self, in_place=False, **kw):
        d = lambda a: torch.from_numpy(a.copy()).to(DEV)
        sc_in, pos_in, lens_in = d(self.scores), d(self.positions), d(self.lens)
        outs = ((sc_in, pos_in, lens_in) if in_place else
                (torch.full_like(sc_in, -9.0), torch.full_like(pos_in, -9),
                 torch.full_like(lens_in, -9)))
        caches = [t.clone() for t in self.p.dev_kv]
        f = sc.shortconv_cache_evict_mxfp8 if self.p.mx else sc.shortconv_cache_evict
        f(sc_in, pos_in, lens_in, d(self.seen), self.budget, self.p.dev["table"], self.p.bs,
          *caches, *outs, sinks=self.sinks, recent=self.recent, **kw)
        torch.cuda.synchronize()
        return outs, caches

    def check(self, in_place=False, **kw):
        outs, caches = self.run(in_place, **kw)
        s_out, p_out, l_out = (t.cpu().numpy() for t in outs)
        plan = ref.evict(self.scores, self.positions, self.lens, self.seen, self.budget, self.sinks,
                         self.recent, self.p.table, self.p.bs, self.p.num_slots, self.cap)
        want_s = self.scores.copy() if in_place else np.full_like(self.scores, -9.0)
        want_p = self.positions.copy() if in_place else np.full_like(self.positions, -9)
        want_kv = [t.clone() for t in self.p.dev_kv]
        for (s, h), (kept, source, moves) in plan.items():
            want_s[s, h, :kept] = self.scores[s, h, source]
            want_p[s, h, :kept] = self.positions[s, h, source]
            assert l_out[s] == kept
            if moves:
                to, frm = torch.tensor(moves, device=DEV).t()
                for w, t in zip(want_kv, self.p.dev_kv):
                    w[to, h] = t[frm, h]
        assert np.array_equal(s_out.view(np.int32), want_s.view(np.int32))
        assert np.array_equal(p_out, want_p)
        for got, want in zip(caches, want_kv):
            bits = torch.int32 if got.dtype == torch.float32 else (
                torch.int16 if got.dtype == torch.bfloat16 else torch.uint8)
            assert torch.equal(got.view(bits), want.view(bits)), "cache rows"


@pytest.mark.parametrize("dtype,mx", KINDS)
@pytest.mark.parametrize("H,D,bs", [(1, 64, 16), (3, 128, 8), (2, 256, 1), (8, 128, 64)])
@pytest.mark.parametrize("in_place", [False, True])
def test_evict(dtype, mx, H, D, bs, in_place):
    Cut(1, dtype, mx, H, D, bs, lens=(40, 3, 16, 17, 0, 130)).check(in_place)


@pytest.mark.parametrize("budget", [0, 1, 2, 15, 16, 17, 39, 40, 41, 1000])
def test_budgets(budget):
    Cut(2, lens=(40, 16, 1), budget=budget).check()


@pytest.mark.parametrize("sinks,recent", [(0, 0), (1, 0), (0, 1), (100, 0), (0, 100), (30, 30)])
def test_protected_entries(sinks, recent):
    """None, some, and more protected entries than the budget holds."""
    Cut(3, lens=(60, 20), budget=12, sinks=sinks, recent=recent).check()


def test_all_scores_equal():
    c = Cut(4, lens=(300,), budget=100, special=False)
    c.scores[:] = 1.0
    c.check()


def test_all_scores_nan():
    c = Cut(5, lens=(300,), budget=100)
    c.scores[:] = np.nan
    c.check()


def test_pages_outside_the_pool():
    Cut(6, lens=(90, 64), budget=30, bs=8, bad=0.4).check()


def test_capacity_below_the_lengths():
    c = Cut(7, lens=(90, 20), budget=10, cap_extra=5)
    c.lens = np.array([200, -4], np.int32)  # clamped to the capacity and to zero
    c.check()


@pytest.mark.parametrize("lens,budget", [((2500, 1030), 1024), ((5000,), 4999), ((9000, 8191), 3),
                                         ((20000,), 9000), ((40000, 9), 3000)])
def test_long_rows(lens, budget):
    """More entries than a workgroup has threads; distinct scores."""
    c = Cut(8, lens=lens, budget=budget, H=2, recent=64, special=False, shuffled=False)
    g = np.random.default_rng(8)
    c.scores[:] = np.exp(2 * g.standard_normal(c.scores.shape)).astype(np.float32)
    c.scores[g.random(c.scores.shape) < 0.2] = 0.0
    c.check()


def test_more_entries_than_registers_hold():
    c = Cut(11, lens=(70000, 300), budget=900, H=1, recent=64, special=False, shuffled=False)
    c.scores[:] = np.random.default_rng(11).integers(0, 3000, c.scores.shape).astype(np.float32)
    c.check()


def test_evicting_twice():
    """A second eviction by the positions that the first one moved."""
    c = Cut(9, lens=(120,), budget=50, shuffled=False)
    (s1, p1, l1), caches = c.run()
    c2 = Cut(9, lens=(120,), budget=20, shuffled=False)
    c2.scores, c2.positions, c2.lens = s1.cpu().numpy(), p1.cpu().numpy(), l1.cpu().numpy()
    c2.seen = c.seen + 3
    c2.p.dev_kv = caches
    c2.check()


def test_graph_replays():
    """One captured eviction, replayed as scores and lengths change."""
    c = Cut(10, lens=(200, 90), budget=40)
    d = lambda a: torch.from_numpy(a.copy()).to(DEV)
    args = [d(c.scores), d(c.positions), d(c.lens), d(c.seen)]
    outs = [torch.empty_like(args[0]), torch.empty_like(args[1]), torch.empty_like(args[2])]
    caches = [t.clone() for t in c.p.dev_kv]

    def step():
        sc.shortconv_cache_evict(*args, 40, c.p.dev["table"], 16, *caches, *outs, sinks=2, recent=4)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(4):
        c.scores[:] = np.random.default_rng(i).random(c.scores.shape).astype(np.float32)
        c.lens[:] = [200 - 50 * i, 90 - 20 * i]
        args[0].copy_(torch.from_numpy(c.scores))
        args[2].copy_(torch.from_numpy(c.lens))
        for t, src in zip(caches, c.p.dev_kv):
            t.copy_(src)
        for o in outs:
            o.fill_(-9)
        graph.replay()
        torch.cuda.synchronize()
        (s, p, l), kv = c.run()
        assert torch.equal(outs[0].view(torch.int32), s.view(torch.int32))
        assert torch.equal(outs[1], p) and torch.equal(outs[2], l)
        assert all(torch.equal(a.view(torch.int16), b.view(torch.int16)) for a, b in zip(caches, kv))
        c.check()
