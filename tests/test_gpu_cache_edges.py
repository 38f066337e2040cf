"""The cache operators where their launches change shape: keys split over every workgroup, pages and
entries around the sizes that the kernels hold in registers, scales of either sign, pools without
a whole page, side streams and captured steps."""
import numpy as np
import pytest
import torch

import cache_reference as ref
import causal_short_convolution_amd as sc
from cache_problem import DEV, Problem, check_rows
from test_gpu_block_sparse import chosen, summaries, want_chosen
from test_gpu_cache_evict import Cut, check_scores

pytestmark = pytest.mark.gpu

KINDS = [("f32", False), ("bf16", False), ("bf16", True), ("f32", True)]


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def check(p):
    out, lse = p.fresh_out()
    p.tree_attention(out, lse)
    torch.cuda.synchronize()
    check_rows(p.expected(), out, lse)


@pytest.mark.parametrize("scale", [-0.3, 0.0, -0.0, 1.7])
@pytest.mark.parametrize("dtype,mx", KINDS)
@pytest.mark.parametrize("G,drafts", [(2, (5, 3)), (6, (30, 9))])
def test_scales_of_either_sign(scale, dtype, mx, G, drafts):
    """Few rows and many; a scale of 0 weighs all keys alike."""
    p = Problem(1, dtype, mx, 2, G, 64, 16, ctx=(90, 0), drafts=drafts, mask="tree", scale=scale)
    check(p)
    check_scores(p)


@pytest.mark.parametrize("scale", [-0.3, 0.0])
def test_selected_pages_under_either_sign(scale):
    p = Problem(2, "bf16", True, 2, 4, 128, 16, ctx=(300, 10), drafts=(2, 3), scale=scale)
    sel = np.array([[[3, 0, -1], [1, 1000, 2]]] * 5, np.int32)
    out, lse = p.fresh_out()
    p.block_attention(torch.from_numpy(sel).to(DEV), out, lse)
    check_rows(p.expected(selected=sel), out, lse)


@pytest.mark.parametrize("dtype,mx", KINDS)
@pytest.mark.parametrize("G,drafts", [(1, 1), (4, 8), (8, 6), (8, 40)])
def test_one_unit_over_every_workgroup(dtype, mx, G, drafts):
    """One sequence and one cache head of many keys: each workgroup holds a few steps, and one row is
    joined from hundreds of parts."""
    check(Problem(3, dtype, mx, 1, G, 64, 64, ctx=(61001,), drafts=(drafts,), q_scale=0.7))


@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("parts", [15, 16, 17, 33])
def test_parts_around_a_round_of_the_join(D, parts):
    check(Problem(4, "bf16", False, 1, 2, D, 16, ctx=(128 * parts - 1,), drafts=(1,)))


def test_selected_pages_over_every_workgroup():
    p = Problem(5, "bf16", False, 1, 3, 64, 64, ctx=(70000,), drafts=(1,), q_scale=0.7)
    sel = np.random.default_rng(5).permutation(1094)[:1000].astype(np.int32).reshape(1, 1, 1000)
    out, lse = p.fresh_out()
    p.block_attention(torch.from_numpy(sel).to(DEV), out, lse)
    check_rows(p.expected(selected=sel), out, lse)


@pytest.mark.parametrize("dtype,mx", KINDS)
@pytest.mark.parametrize("D", [64, 128, 256])
def test_scores_of_ragged_lengths(dtype, mx, D):
    """Many sequences share the line of steps; some have no new token, some no key."""
    g = np.random.default_rng(6)
    ctx = g.integers(0, 700, 30)
    ctx[3], ctx[17] = 0, 5000
    drafts = g.integers(0, 4, 30)
    drafts[3] = 0
    check_scores(Problem(6, dtype, mx, 2, 3, D, 16, ctx=ctx, drafts=drafts, mask="tree", bad=0.05,
                         behind=1))


@pytest.mark.parametrize("bs", [1, 4, 16, 32])
def test_scores_of_pages_inside_and_past_a_tile(bs):
    check_scores(Problem(7, "bf16", True, 1, 2, 128, bs, ctx=(33, 127, 129), drafts=(2, 1, 200),
                         bad=0.1))


def test_scores_of_a_sequence_without_tokens_are_carried_over():
    p = Problem(8, "bf16", False, 2, 2, 64, 16, ctx=(70,), drafts=(0,), behind=2)
    start = torch.rand((1, 2, 90), device=DEV)
    out = torch.full((1, 2, 90), -3.0, device=DEV)
    p.cache_scores(torch.zeros((2, 4), device=DEV), start, out)
    torch.cuda.synchronize()
    assert torch.equal(out[..., :70], start[..., :70]) and bool((out[..., 70:] == -3.0).all())


@pytest.mark.parametrize("rows", [2, 60])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_pool_without_a_whole_page(dtype, rows):
    """Fewer rows than a page has: the pool holds no keys, whatever the table says."""
    H, G, D, bs = 2, 2, 64, 16
    dt = {"f32": torch.float32, "bf16": torch.bfloat16}[dtype]
    kv = [torch.full((bs - 1, H, D), float("nan"), dtype=dt, device=DEV) for _ in range(2)]
    q = torch.randn((rows, H * G, D), device=DEV).to(dt)
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device=DEV)
    where = (i32(0, rows), i32(40), torch.zeros((1, 9), dtype=torch.int32, device=DEV), bs)
    out = torch.full((rows, H * G, D), 3.0, dtype=dt, device=DEV)
    lse = torch.zeros((rows, H * G), device=DEV)
    sc.shortconv_tree_attention(q, *where, *kv, out, scale=0.1, lse=lse)
    torch.cuda.synchronize()
    assert bool((out == 0).all()) and bool((lse == -float("inf")).all())
    out.fill_(3.0)
    sel = torch.zeros((rows, H, 2), dtype=torch.int32, device=DEV)
    sc.shortconv_block_attention(q, *where, sel, *kv, out, scale=0.1, lse=lse)
    sums = torch.full((1, H, 100), 3.0, device=DEV)
    sc.shortconv_cache_scores(q, torch.zeros_like(lse), *where, kv[0], None, sums, scale=0.1)
    torch.cuda.synchronize()
    assert bool((out == 0).all()) and bool((lse == -float("inf")).all())
    assert bool((sums[..., :40 + rows] == 0).all()) and bool((sums[..., 40 + rows:] == 3.0).all())


@pytest.mark.parametrize("pages", [1, 63, 64, 65, 1023, 1025, 4097, 16383, 16385])
def test_pages_around_what_registers_hold(pages):
    """Table widths of every remainder of 4, and each way of picking."""
    p = Problem(9, "bf16", False, 1, 2, 64, 1, ctx=(pages - 1, 3), drafts=(1, 2), spare_blocks=0)
    ds, de, want = summaries(p)
    for topk in (1, 100):
        sel = chosen(p, ds, de, topk)
        assert np.array_equal(sel.cpu().numpy(), want_chosen(p, want, topk))


@pytest.mark.parametrize("H,G,D", [(1, 65, 64), (2, 130, 64), (1, 70, 256)])
def test_selection_of_many_heads_in_a_group(H, G, D):
    """Sums of codes past 13 bits are cut into three planes."""
    p = Problem(10, "bf16", False, H, G, D, 4, ctx=(300, 50), drafts=(3, 1))
    ds, de, want = summaries(p)
    sel = chosen(p, ds, de, 12)
    assert np.array_equal(sel.cpu().numpy(), want_chosen(p, want, 12))


def test_selection_tiles_end_with_their_sequences():
    p = Problem(11, "f32", False, 2, 3, 128, 8, ctx=(200, 0, 64, 5, 90, 1000),
                drafts=(15, 16, 0, 17, 1, 33), behind=5, pad=8)
    ds, de, want = summaries(p)
    sel = chosen(p, ds, de, 5)
    assert np.array_equal(sel.cpu().numpy(), want_chosen(p, want, 5))


@pytest.mark.parametrize("n", [2047, 2048, 2049, 5119, 5121, 16384, 16385, 32769, 65536])
def test_entries_around_what_registers_hold(n):
    c = Cut(12, lens=(n, 7), budget=n - 1 if n % 2 else n // 3, H=1, recent=16, cap_extra=0, bs=1,
            special=False, shuffled=False)
    g = np.random.default_rng(n)
    c.scores[:] = np.exp(3 * g.standard_normal(c.scores.shape)).astype(np.float32)
    c.check()


@pytest.mark.parametrize("kind", ["two values", "one differs", "denormal", "both signs", "infinite",
                                  "mostly nan"])
def test_scores_that_are_hard_to_rank(kind):
    g = np.random.default_rng(13)
    c = Cut(13, lens=(3500, 1200), budget=1100, H=2, special=False, shuffled=False)
    shape = c.scores.shape
    if kind == "two values":
        c.scores[:] = np.where(g.random(shape) < 0.6, 1.0, np.nextafter(np.float32(1), np.float32(2)))
    elif kind == "one differs":
        c.scores[:] = 0.25
        c.scores[:, :, 600] = 0.125
    elif kind == "denormal":
        c.scores[:] = g.integers(0, 50, shape).astype(np.float32) * np.float32(1.4e-45)
    elif kind == "both signs":
        c.scores[:] = g.standard_normal(shape) * np.exp(20 * g.standard_normal(shape))
        c.scores[g.random(shape) < 0.1] = -0.0
    elif kind == "infinite":
        c.scores[:] = g.choice(np.array([np.inf, -np.inf, 3e38, -3e38], np.float32), shape)
    else:
        c.scores[:] = np.where(g.random(shape) < 0.9, np.nan, 1.0)
    c.check()


def decode_step(p, selected, stream=None):
    """Scores of one step, a selection and attention over it, all on `stream`."""
    pages = p.num_slots // p.bs
    summ = torch.zeros((pages, p.H, 2, p.D), dtype=torch.int8, device=DEV)
    exps = torch.zeros((pages, p.H), dtype=torch.uint8, device=DEV)
    out, lse = p.fresh_out()
    sums = torch.zeros((p.N, p.H, p.table.shape[1] * p.bs), device=DEV)
    torch.cuda.synchronize()
    kw = {} if stream is None else {"stream": stream}
    f = sc.shortconv_block_summary_mxfp8 if p.mx else sc.shortconv_block_summary
    f(*p.key, *p.where, summ, exps, rebuild=True, **kw)
    sc.shortconv_block_select(p.dev_q, *p.where, summ, exps, selected, **kw)
    p.block_attention(selected, out, lse, **kw)
    p.cache_scores(lse, None, sums, **kw)
    return out, lse, sums


@pytest.mark.parametrize("mx", [False, True])
def test_a_step_on_side_streams(mx):
    """The same bits on the current stream, on another, and on two at once."""
    ps = [Problem(20 + i, "bf16", mx, 2, 4, 128, 16, ctx=(900, 40), drafts=(1, 1)) for i in range(2)]
    sels = [torch.full((p.T, p.H, 6), -2, dtype=torch.int32, device=DEV) for p in ps]
    want = [decode_step(p, s) for p, s in zip(ps, sels)]
    torch.cuda.synchronize()
    want_sel = [s.clone() for s in sels]
    streams = [torch.cuda.Stream() for _ in ps]
    for _ in range(3):
        for s in sels:
            s.fill_(-2)
        torch.cuda.synchronize()
        got = [decode_step(p, s, st) for p, s, st in zip(ps, sels, streams)]
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            assert all(torch.equal(x, y) for x, y in zip(a, b))
        assert all(torch.equal(x, y) for x, y in zip(want_sel, sels))


def test_captured_step_with_eviction_replays():
    """Attention, the weights of its keys and the eviction by them in one graph, replayed with eager
    work between, against the eager calls each time."""
    p = Problem(30, "bf16", False, 2, 4, 64, 16, ctx=(300, 120), drafts=(1, 1))
    cap, budget = 320, 100
    g = torch.Generator().manual_seed(1)
    start = torch.rand((2, 2, cap), generator=g).to(DEV)
    pos = torch.arange(cap, dtype=torch.int32, device=DEV).expand(2, 2, cap).contiguous()
    lens = torch.tensor([301, 121], dtype=torch.int32, device=DEV)
    first = [t.clone() for t in p.dev_kv]

    def step():
        out, lse = p.fresh_out()
        sums, s_out = torch.zeros_like(start), torch.zeros_like(start)
        p_out, l_out = torch.zeros_like(pos), torch.zeros_like(lens)
        p.tree_attention(out, lse)
        p.cache_scores(lse, start, sums)
        sc.shortconv_cache_evict(sums, pos, lens, lens, budget, p.dev["table"], p.bs, *p.dev_kv,
                                 s_out, p_out, l_out, sinks=2, recent=8)
        return out, lse, s_out, p_out, l_out

    def reset():
        for t, f in zip(p.dev_kv, first):
            t.copy_(f)

    same = lambda a, b: torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    reset()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for i in range(4):
        p.dev_q.copy_(torch.randn(p.dev_q.shape, generator=g).to(p.dev_q))
        reset()
        want = step()
        torch.cuda.synchronize()
        want_kv = [t.clone() for t in p.dev_kv]
        reset()
        graph.replay()
        torch.cuda.synchronize()
        assert all(same(a, b) for a, b in zip(want, got)), i
        assert all(same(a, b) for a, b in zip(want_kv, p.dev_kv)), i
