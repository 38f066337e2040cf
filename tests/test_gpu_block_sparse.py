"""Page summaries, page selection and attention over the selected pages: the whole numbers must be
those of the definition, the attention within its rounding bounds."""
import numpy as np
import pytest
import torch

import cache_reference as ref
import causal_short_convolution_amd as sc
from cache_problem import DEV, Problem, check_rows

pytestmark = pytest.mark.gpu

KINDS = [("f32", False), ("bf16", False), ("bf16", True), ("f32", True)]


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def summaries(p, rebuild=True, start=None):
    pages = p.num_slots // p.bs
    g = np.random.default_rng(3)
    s = g.integers(-128, 128, (pages, p.H, 2, p.D)).astype(np.int8) if start is None else start[0]
    e = g.integers(0, 256, (pages, p.H)).astype(np.uint8) if start is None else start[1]
    ds, de = torch.from_numpy(s).to(DEV), torch.from_numpy(e).to(DEV)
    f = sc.shortconv_block_summary_mxfp8 if p.mx else sc.shortconv_block_summary
    f(*p.key, *p.where, ds, de, rebuild=rebuild)
    torch.cuda.synchronize()
    want = ref.summary(p.kv[0], p.cu, p.ctx, p.table, p.bs, p.num_slots, rebuild, s, e)
    assert np.array_equal(ds.cpu().numpy(), want[0]) and np.array_equal(de.cpu().numpy(), want[1])
    return ds, de, want


def chosen(p, ds, de, topk, sinks=1, recents=1, q=None, **kw):
    sel = torch.full((p.T, p.H, topk), -2, dtype=torch.int32, device=DEV)
    sc.shortconv_block_select(p.dev_q if q is None else q, *p.where, ds, de, sel,
                              sink_blocks=sinks, recent_blocks=recents, **kw)
    torch.cuda.synchronize()
    return sel


def want_chosen(p, want, topk, sinks=1, recents=1):
    return ref.select(p.q, p.cu, p.ctx, p.table, p.bs, p.num_slots, *want, sinks, recents, topk)


@pytest.mark.parametrize("dtype,mx", KINDS)
@pytest.mark.parametrize("H,G,D,bs", [(1, 1, 64, 16), (2, 4, 128, 16), (3, 2, 256, 8), (5, 3, 64, 1),
                                      (8, 4, 128, 64)])
def test_summary_selection_attention(dtype, mx, H, G, D, bs):
    p = Problem(1, dtype, mx, H, G, D, bs, ctx=(37 * bs // 4, 0, 5 * bs + 3), drafts=(3, 2, 1),
                behind=2)
    ds, de, want = summaries(p)
    sel = chosen(p, ds, de, 4)
    exp = want_chosen(p, want, 4)
    assert np.array_equal(sel.cpu().numpy(), exp)
    out, lse = p.fresh_out()
    p.block_attention(sel, out, lse)
    check_rows(p.expected(selected=exp), out, lse)


@pytest.mark.parametrize("dtype,mx", KINDS)
def test_partial_summary_only_touches_the_new_pages(dtype, mx):
    p = Problem(2, dtype, mx, 2, 1, 64, 16, ctx=(40, 0, 64, 15), drafts=(5, 1, 33, 0))
    summaries(p, rebuild=False)


def test_summary_of_special_values():
    p = Problem(3, "f32", False, 2, 1, 64, 8, ctx=(48,), drafts=(0,))
    k = p.stored[0]
    slot = [int(p.table[0, b]) * 8 for b in range(6)]
    k[slot[0]:slot[0] + 8] = 0.0
    k[slot[1]:slot[1] + 8] = float("nan")
    k[slot[2] + 1, 0, 3] = float("inf")
    k[slot[3]:slot[3] + 8, 1] *= 1e-40
    k[slot[4] + 2, 1, 5] = float("nan")
    k[slot[5]:slot[5] + 8] = 0.49609375  # on a rounding tie
    p.dev_kv[0].copy_(k)
    p.kv[0] = k.double().numpy()
    summaries(p)


@pytest.mark.parametrize("topk", [1, 2, 3, 7, 40])
@pytest.mark.parametrize("sinks,recents", [(0, 0), (1, 1), (0, 3), (5, 0), (9, 9)])
def test_forced_pages_and_counts(topk, sinks, recents):
    p = Problem(4, "bf16", False, 2, 2, 64, 4, ctx=(50, 2, 0, 70), drafts=(2, 1, 1, 3), bad=0.2)
    ds, de, want = summaries(p)
    sel = chosen(p, ds, de, topk, sinks, recents)
    assert np.array_equal(sel.cpu().numpy(), want_chosen(p, want, topk, sinks, recents))


def test_equal_scores_go_to_the_lowest_page():
    p = Problem(5, "bf16", False, 1, 2, 64, 4, ctx=(400,), drafts=(2,))
    pages = p.num_slots // p.bs
    same = np.zeros((pages, 1, 2, 64), np.int8)
    same[:, :, 1] = 3
    same[::3, :, 1] = 5
    exps = np.full((pages, 1), 120, np.uint8)
    ds, de = torch.from_numpy(same).to(DEV), torch.from_numpy(exps).to(DEV)
    for topk in (5, 50, 90):
        sel = chosen(p, ds, de, topk, 0, 0)
        assert np.array_equal(sel.cpu().numpy(), want_chosen(p, (same, exps), topk, 0, 0))


def test_queries_with_special_values():
    p = Problem(6, "f32", False, 1, 3, 64, 4, ctx=(100,), drafts=(4,))
    p.q[0, 0, :5] = np.nan
    p.q[1] = 0.0
    p.q[2] *= 1e-41
    p.q[2] = p.q[2].astype(np.float32)
    p.q[3, 1, 7] = np.inf
    ds, de, want = summaries(p)
    sel = chosen(p, ds, de, 6, q=torch.from_numpy(p.q.astype(np.float32)).to(DEV))
    assert np.array_equal(sel.cpu().numpy(), want_chosen(p, want, 6))


@pytest.mark.parametrize("G,D", [(16, 128), (64, 64), (16, 256)])
def test_sums_beyond_24_bits(G, D):
    """Whole sums past 2^24 are rounded once to fp32; the largest codes reach them."""
    p = Problem(7, "f32", False, 1, G, D, 4, ctx=(200,), drafts=(2,))
    pages = p.num_slots // p.bs
    g = np.random.default_rng(1)
    s = g.integers(90, 128, (pages, 1, 2, D)).astype(np.int8)
    s[:, :, 0] *= -1
    e = np.full((pages, 1), 121, np.uint8)
    ds, de = torch.from_numpy(s).to(DEV), torch.from_numpy(e).to(DEV)
    p.q[:] = np.sign(p.q) * (1.9 + 0.05 * np.abs(p.q) / 8)
    p.q = p.q.astype(np.float32).astype(np.float64)
    sel = chosen(p, ds, de, 9, 0, 0, q=torch.from_numpy(p.q.astype(np.float32)).to(DEV))
    assert np.array_equal(sel.cpu().numpy(), want_chosen(p, (s, e), 9, 0, 0))


@pytest.mark.parametrize("pages", [300, 2500, 9000])
def test_many_pages(pages):
    p = Problem(8, "bf16", False, 1, 2, 64, 2, ctx=(2 * pages - 3, 40), drafts=(2, 1))
    ds, de, want = summaries(p)
    for topk in (3, 64, 257):
        sel = chosen(p, ds, de, topk)
        assert np.array_equal(sel.cpu().numpy(), want_chosen(p, want, topk))


@pytest.mark.parametrize("dtype,mx", KINDS)
def test_attention_skips_what_is_no_page(dtype, mx):
    """Ids outside the table, unordered ids, an id given twice, pages past the token's position,
    pages outside the pool, no id at all."""
    p = Problem(9, dtype, mx, 2, 3, 64, 8, ctx=(30, 0, 90), drafts=(4, 2, 1), bad=0.2)
    g = np.random.default_rng(2)
    MB = p.table.shape[1]
    sel = g.integers(-3, MB + 3, (p.T, 2, 7)).astype(np.int32)
    sel[0] = -1
    sel[1, 0] = [2, 2, -1, 0, MB, 2 ** 31 - 1, -2 ** 31]
    out, lse = p.fresh_out()
    p.block_attention(torch.from_numpy(sel).to(DEV), out, lse)
    check_rows(p.expected(selected=sel), out, lse)
    assert bool((out[0] == 0).all())
    out, lse = p.fresh_out()
    p.block_attention(torch.empty((p.T, 2, 0), dtype=torch.int32, device=DEV), out, lse)
    torch.cuda.synchronize()
    assert bool((out == 0).all()) and bool((lse == -float("inf")).all())


@pytest.mark.parametrize("dtype,mx", KINDS)
@pytest.mark.parametrize("G", [1, 4, 16, 40])
def test_attention_over_many_pages(dtype, mx, G):
    p = Problem(10, dtype, mx, 1, G, 128, 16, ctx=(1500, 33), drafts=(2, 1))
    g = np.random.default_rng(4)
    sel = np.full((p.T, 1, 70), -1, np.int32)
    for t in range(p.T):
        n = int(p.ctx[0 if t < 2 else 1]) // 16 + 1
        ids = np.sort(g.permutation(n)[:70])
        sel[t, 0, :len(ids)] = ids
    out, lse = p.fresh_out()
    p.block_attention(torch.from_numpy(sel).to(DEV), out, lse)
    check_rows(p.expected(selected=sel), out, lse)


def test_all_pages_equal_full_attention():
    """With every page selected the result is that of the attention over the whole cache."""
    p = Problem(11, "bf16", False, 2, 4, 128, 16, ctx=(300,), drafts=(5,))
    ds, de, want = summaries(p)
    sel = chosen(p, ds, de, 25)
    out, lse = p.fresh_out()
    p.block_attention(sel, out, lse)
    check_rows(p.expected(), out, lse)


def test_nan_behind_the_tokens_position_does_not_leak():
    p = Problem(12, "bf16", False, 1, 2, 64, 16, ctx=(20,), drafts=(6,))
    sel = torch.zeros((p.T, 1, 2), dtype=torch.int32, device=DEV)
    sel[:, :, 1] = 1
    clean, _ = p.fresh_out()
    p.block_attention(sel, clean, None)
    for pos in range(23, 26):  # the last three new tokens
        slot = int(p.table[0, pos // 16]) * 16 + pos % 16
        for t in p.dev_kv:
            t[slot] = float("nan")
    out, _ = p.fresh_out()
    p.block_attention(sel, out, None)
    torch.cuda.synchronize()
    assert torch.equal(out[:3], clean[:3]) and not bool(torch.isfinite(out[3:].float()).any())


def test_captured_step():
    """Summary, selection and attention of a decode step as one graph, replayed as the sequence
    grows."""
    p = Problem(13, "bf16", False, 2, 4, 64, 16, ctx=(200, 90), drafts=(1, 1))
    pages = p.num_slots // p.bs
    s = torch.zeros((pages, 2, 2, 64), dtype=torch.int8, device=DEV)
    e = torch.zeros((pages, 2), dtype=torch.uint8, device=DEV)
    sc.shortconv_block_summary(*p.key, *p.where, s, e, rebuild=True)
    sel = torch.zeros((2, 2, 5), dtype=torch.int32, device=DEV)
    out, lse = p.fresh_out()

    def step():
        sc.shortconv_block_summary(*p.key, *p.where, s, e)
        sc.shortconv_block_select(p.dev_q, *p.where, s, e, sel)
        p.block_attention(sel, out, lse)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for ctx in ((100, 3), (101, 4), (150, 89), (200, 90)):
        p.ctx[:] = ctx
        p.dev["ctx"].copy_(torch.from_numpy(p.ctx))
        before = (s.cpu().numpy(), e.cpu().numpy())
        graph.replay()
        torch.cuda.synchronize()
        want = ref.summary(p.kv[0], p.cu, p.ctx, p.table, p.bs, p.num_slots, False, *before)
        assert np.array_equal(s.cpu().numpy(), want[0]) and np.array_equal(e.cpu().numpy(), want[1])
        exp = want_chosen(p, want, 5)
        assert np.array_equal(sel.cpu().numpy(), exp)
        check_rows(p.expected(selected=exp), out, lse)
