"""shortconv_tree_attention against the definition in fp64: types, head layouts, lengths, masks,
pages, and what a serving program does with it (streams, graphs, workspaces)."""
import numpy as np
import pytest
import torch

import causal_short_convolution_amd as sc
from cache_problem import DEV, Problem, check_rows

pytestmark = pytest.mark.gpu

KINDS = [("f32", False), ("bf16", False), ("bf16", True), ("f32", True)]


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def run(p, **kw):
    out, lse = p.fresh_out()
    p.tree_attention(out, lse, **kw)
    torch.cuda.synchronize()
    return out, lse


def check(p):
    out, lse = run(p)
    check_rows(p.expected(), out, lse)


@pytest.mark.parametrize("dtype,mx", KINDS)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("H,G", [(1, 1), (2, 3), (1, 16), (3, 20)])
def test_types_and_heads(dtype, mx, D, H, G):
    check(Problem(1, dtype, mx, H, G, D, 16, ctx=(37, 0, 130), drafts=(5, 3, 1), mask="tree"))


@pytest.mark.parametrize("dtype,mx", KINDS)
@pytest.mark.parametrize("bs", [1, 2, 8, 64, 128])
def test_page_sizes(dtype, mx, bs):
    check(Problem(2, dtype, mx, 2, 4, 128, bs, ctx=(1, 63, 200, 129), drafts=(1, 2, 17, 4),
                  mask="tree"))


@pytest.mark.parametrize("dtype,mx", KINDS)
def test_lengths_around_tiles(dtype, mx):
    """Every number of keys near the multiples of 16, 32, 64 and 128, one token each."""
    lens = [0, 1, 2, 15, 16, 17, 30, 31, 32, 33, 47, 62, 63, 64, 65, 95, 126, 127, 128, 129, 255,
            256, 257, 511]
    check(Problem(3, dtype, mx, 1, 2, 64, 16, ctx=lens, drafts=[1] * len(lens)))


@pytest.mark.parametrize("dtype,mx", KINDS)
@pytest.mark.parametrize("mask", [None, "tree", "random"])
def test_masks(dtype, mx, mask):
    """Chains, trees and arbitrary masks with empty rows; sequences with no new token, rows behind
    the last sequence, a context of zero (rows for which nothing is left)."""
    check(Problem(4, dtype, mx, 2, 2, 64, 16, ctx=(0, 9, 40, 0, 16), drafts=(7, 0, 70, 1, 16),
                  mask=mask, behind=3))


def test_empty_rows_are_zero():
    mask = np.zeros((6, 1), np.int64)
    mask[2] = 4
    p = Problem(5, "bf16", False, 2, 2, 64, 16, ctx=(0,), drafts=(6,), mask=mask)
    out, lse = run(p)
    check_rows(p.expected(), out, lse)
    assert bool((out[[0, 1, 3, 4, 5]] == 0).all()) and bool(torch.isinf(lse[0]).all())


@pytest.mark.parametrize("dtype,mx", KINDS)
def test_fewer_mask_words_than_drafts(dtype, mx):
    check(Problem(6, dtype, mx, 1, 2, 64, 16, ctx=(20,), drafts=(100,), mask="random", words=1))


@pytest.mark.parametrize("dtype,mx", KINDS)
def test_pages_outside_the_pool_hold_no_keys(dtype, mx):
    p = Problem(7, dtype, mx, 2, 2, 64, 8, ctx=(100, 64, 3), drafts=(9, 4, 2), mask="tree", bad=0.4)
    check(p)
    p.table[:] = -1
    p.dev["table"].fill_(-1)
    out, lse = run(p)
    assert bool((out == 0).all()) and bool((lse == -float("inf")).all())


def test_table_shorter_than_the_sequence():
    """Keys past max_blocks * block_size do not exist."""
    p = Problem(8, "bf16", False, 2, 2, 64, 16, ctx=(60, 10), drafts=(9, 3), spare_blocks=0)
    p.table = p.table[:, :2].copy()
    p.dev["table"] = torch.from_numpy(p.table).to(DEV)
    p.where = (p.dev["cu"], p.dev["ctx"], p.dev["table"], 16)
    check(p)


def test_strided_queries_and_no_lse():
    p = Problem(9, "bf16", False, 2, 4, 128, 16, ctx=(50, 3), drafts=(4, 6), mask="tree", pad=40)
    out, _ = p.fresh_out()
    p.tree_attention(out, None)
    check_rows(p.expected(), out, None)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("what", [float("nan"), float("inf"), -float("inf"), "lowest"])
def test_masked_drafts_never_leak(dtype, what):
    """Drafts that only some rows look at hold NaN, infinities or the type's lowest value: the rows
    that do not look at them stay exactly what they are without them."""
    mask = np.zeros((8, 1), np.int64)
    for i in range(8):
        mask[i] = (1 << i) | 1 if i != 3 else 0b1001
    p = Problem(10, dtype, False, 2, 3, 64, 16, ctx=(21,), drafts=(8,), mask=mask)
    clean, clean_lse = run(p)
    bad_key = 21 + 3  # draft 3, which only token 3 looks at
    slot = int(p.table[0, bad_key // 16]) * 16 + bad_key % 16
    value = torch.finfo(p.dt).min if what == "lowest" else what
    for t in p.dev_kv:
        t[slot] = value
    out, lse = run(p)
    rest = [0, 1, 2, 4, 5, 6, 7]
    assert torch.equal(out[rest], clean[rest]) and torch.equal(lse[rest], clean_lse[rest])
    if what != "lowest":
        assert not bool(torch.isfinite(out[3].float()).any())


def test_large_logits_keep_the_softmax_finite():
    p = Problem(11, "f32", False, 1, 2, 64, 16, ctx=(70,), drafts=(3,), scale=40.0)
    out, lse = run(p)
    assert bool(torch.isfinite(out).all()) and bool(torch.isfinite(lse).all())
    check_rows(p.expected(), out, lse)


@pytest.mark.parametrize("dtype,mx,D", [("bf16", False, 128), ("bf16", True, 128),
                                        ("f32", False, 64)])
def test_long_ragged_batch(dtype, mx, D):
    """Contexts long and short enough that the keys of one sequence are split and joined."""
    check(Problem(12, dtype, mx, 2, 4, D, 16, ctx=(4000, 1, 700, 2500, 0), drafts=(2, 1, 1, 3, 2),
                  mask="tree"))


def test_many_short_sequences():
    n = 300
    check(Problem(13, "bf16", False, 2, 2, 64, 16, ctx=[(7 * i) % 40 for i in range(n)],
                  drafts=[i % 3 for i in range(n)]))


@pytest.mark.parametrize("dtype,mx", KINDS)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("G,drafts", [(3, (11, 0, 15)), (4, (16, 9)), (5, (20, 24)), (8, (33, 30)),
                                      (16, (31, 1)), (7, (45, 60)), (20, (30,))])
def test_rows_per_sequence(dtype, mx, D, G, drafts):
    """From 33 to 600 query rows per sequence and cache head, over short and long contexts."""
    check(Problem(14, dtype, mx, 2, G, D, 16, ctx=(150, 70, 1000)[:len(drafts)], drafts=drafts,
                  mask="tree"))


@pytest.mark.parametrize("bs", [1, 8, 64])
@pytest.mark.parametrize("mask", [None, "random"])
def test_many_rows_masks_and_pages(bs, mask):
    check(Problem(22, "bf16", False, 1, 4, 128, bs, ctx=(150, 0, 63, 64), drafts=(20, 70, 9, 33),
                  mask=mask, bad=0.2, behind=2))


@pytest.mark.parametrize("what", [float("nan"), float("inf"), -float("inf")])
def test_many_rows_masked_drafts_never_leak(what):
    n = 24
    mask = np.array([[(1 << i) | 1] if i != 3 else [0b1001] for i in range(n)], np.int64)
    p = Problem(23, "bf16", False, 2, 4, 128, 16, ctx=(21,), drafts=(n,), mask=mask)
    clean, clean_lse = run(p)
    slot = int(p.table[0, 24 // 16]) * 16 + 24 % 16
    for t in p.dev_kv:
        t[slot] = what
    out, lse = run(p)
    rest = [i for i in range(n) if i != 3]
    assert torch.equal(out[rest], clean[rest]) and torch.equal(lse[rest], clean_lse[rest])
    assert not bool(torch.isfinite(out[3].float()).any())
    p.dev_kv[0][slot] = 0.5  # a finite logit: what V holds is what comes out
    out, lse = run(p)
    assert torch.equal(out[rest], clean[rest])
    got = out[3].float()
    assert bool(got.isnan().all()) if what != what else bool((got == what).all())


def test_cache_beyond_32_bit_offsets():
    """Rows whose byte and element offsets pass 2^32."""
    H, D, bs = 16, 256, 16
    slots = (1 << 32) // (H * D) + 4096
    p = Problem(15, "bf16", False, H, 2, D, bs, ctx=(40,), drafts=(2,))
    first = slots // bs - p.pages
    big = []
    for t in p.dev_kv:
        b = torch.empty((slots, H, D), dtype=t.dtype, device=DEV)
        b[first * bs:(first + p.pages) * bs] = t[:p.pages * bs]
        big.append(b)
    table = torch.where((p.dev["table"] >= 0) & (p.dev["table"] < p.pages), p.dev["table"] + first,
                        -1).to(torch.int32)
    out, lse = p.fresh_out()
    sc.shortconv_tree_attention(p.dev_q, p.dev["cu"], p.dev["ctx"], table, bs, *big, out,
                                scale=p.scale, lse=lse)
    check_rows(p.expected(), out, lse)


def test_no_tokens_and_no_sequences():
    p = Problem(16, "bf16", False, 2, 2, 64, 16, ctx=(5, 6), drafts=(0, 0))
    run(p)
    cu = torch.zeros(1, dtype=torch.int32, device=DEV)
    empty = torch.zeros((0, 3), dtype=torch.int32, device=DEV)
    q = torch.zeros((2, 4, 64), dtype=torch.bfloat16, device=DEV)
    out = torch.full_like(q, 7.0)
    sc.shortconv_tree_attention(q, cu, empty[:, 0].contiguous(), empty, 16, *p.dev_kv, out)
    assert bool((out == 7.0).all())


def test_same_bits_every_time_and_on_another_stream():
    p = Problem(17, "bf16", False, 2, 4, 128, 16, ctx=(900, 31), drafts=(3, 5), mask="tree")
    out, lse = run(p)
    side = torch.cuda.Stream()
    for _ in range(3):
        again, again_lse = p.fresh_out()
        side.wait_stream(torch.cuda.current_stream())
        p.tree_attention(again, again_lse, stream=side)
        torch.cuda.synchronize()
        assert torch.equal(out, again) and torch.equal(lse, again_lse)


def test_two_streams_at_once():
    ps = [Problem(18 + i, "bf16", False, 2, 4, 128, 16, ctx=(1500, 3), drafts=(2, 4), mask="tree")
          for i in range(2)]
    want = [run(p) for p in ps]
    streams = [torch.cuda.Stream() for _ in ps]
    for _ in range(5):
        got = [p.fresh_out() for p in ps]
        torch.cuda.synchronize()
        for p, (o, l), st in zip(ps, got, streams):
            p.tree_attention(o, l, stream=st)
        torch.cuda.synchronize()
        for (o, l), (wo, wl) in zip(got, want):
            assert torch.equal(o, wo) and torch.equal(l, wl)


def test_graph_replays_follow_the_lengths():
    """One captured call, replayed after the lengths, the table's rows and the queries changed."""
    p = Problem(20, "bf16", False, 2, 2, 64, 16, ctx=(700, 20), drafts=(2, 3))
    out, lse = p.fresh_out()
    p.tree_attention(out, lse)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        p.tree_attention(out, lse)
    for ctx in ((700, 20), (1, 0), (333, 19), (700, 20)):
        p.ctx[:] = ctx
        p.dev["ctx"].copy_(torch.from_numpy(p.ctx))
        out.fill_(7.0)
        lse.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        check_rows(p.expected(), out, lse)
        eager, eager_lse = run(p)
        assert torch.equal(out, eager) and torch.equal(lse, eager_lse)


def test_workspace_too_small_is_refused():
    p = Problem(21, "bf16", False, 2, 2, 64, 16, ctx=(700, 20), drafts=(2, 3))
    need = sc.shortconv_tree_attention_workspace_size(p.T, p.N, 4, 2, 64, p.dt)
    if need == 0:
        pytest.skip("no workspace needed")
    out, lse = p.fresh_out()
    with pytest.raises(sc.ShortConvError, match="workspace"):
        p.tree_attention(out, lse,
                         workspace=torch.empty(need - 1, dtype=torch.uint8, device=DEV))
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device=DEV)  # contents do not matter
    p.tree_attention(out, lse, workspace=ws)
    check_rows(p.expected(), out, lse)


@pytest.mark.parametrize("seed", range(8))
def test_random(seed):
    g = np.random.default_rng(900 + seed)
    dtype, mx = KINDS[seed % 4]
    n = int(g.integers(1, 6))
    check(Problem(1000 + seed, dtype, mx, int(g.integers(1, 5)), int(g.integers(1, 10)),
                  int(g.choice([64, 128, 256])), int(g.choice([1, 4, 16, 32, 64])),
                  ctx=[int(x) for x in g.integers(0, 300, n)],
                  drafts=[int(x) for x in g.integers(0, 20, n)],
                  mask=[None, "tree", "random"][seed % 3], bad=0.1, behind=int(g.integers(0, 3)),
                  pad=8 * int(g.integers(0, 4))))
