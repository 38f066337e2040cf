"""The torch binding of the cache operators rejects malformed tensor arguments before the library
is loaded or called (on host tensors, the library loader replaced by one that fails the test): a
well-formed argument set stops only at "must be on a GPU", each malformed variant at the argument
it breaks."""
import pytest
import torch

from causal_short_convolution_amd import _cache as c

T, N, H, G, D, W, S, SLOTS, MB, BS, M, K = 12, 3, 2, 3, 64, 4, 5, 64, 5, 8, 6, 4
CAP = 40
BF, F32, I32, I64, U8, I8 = (torch.bfloat16, torch.float32, torch.int32, torch.int64, torch.uint8,
                             torch.int8)


@pytest.fixture(autouse=True)
def no_library(monkeypatch):
    def refuse(*_a, **_k):
        raise AssertionError("the binding reached the library with arguments it should reject")
    monkeypatch.setattr(c, "load_cache_library", refuse)


def z(*shape, dt=BF):
    return torch.zeros(shape, dtype=dt)


def plain(names=("k_cache", "v_cache")):
    return {n: z(SLOTS, H, D) for n in names}


def mx(names=("k", "v")):
    return {**{f"{n}_codes": z(SLOTS, H, D, dt=U8) for n in names},
            **{f"{n}_scales": z(SLOTS, H, D // 32, dt=U8) for n in names}}


def batch():
    return dict(cu_seqlens=z(N + 1, dt=I32), context_lens=z(N, dt=I32),
                block_table=z(N, MB, dt=I32), block_size=BS)


def verify(cache):
    return dict(k=z(T, H, D), v=z(T, H, D), cu_seqlens=z(N + 1, dt=I32), parents=z(T, dt=I32),
                k_taps=z(W, H, D, dt=F32), v_taps=z(W, H, D, dt=F32), k_gamma=z(D, dt=F32),
                v_gamma=z(D, dt=F32), eps=1e-6, k_state=z(S, W - 1, H, D),
                v_state=z(S, W - 1, H, D), state_idx=z(N, dt=I32), k_snap=z(N, M, W - 1, H, D),
                v_snap=z(N, M, W - 1, H, D), slot_mapping=z(T, dt=I64), **cache,
                mask=z(T, 1, dt=I64))


def attn(cache, **extra):
    return dict(q=z(T, G * H, D), **batch(), **extra, **cache, out=z(T, G * H, D),
                lse=z(T, G * H, dt=F32), workspace=z(64, dt=U8))


def scores(cache):
    return dict(q=z(T, G * H, D), lse=z(T, G * H, dt=F32), **batch(), **cache,
                scores=z(N, H, CAP, dt=F32), scores_out=z(N, H, CAP, dt=F32), mask=z(T, 1, dt=I64))


def evict(cache):
    return dict(scores=z(N, H, CAP, dt=F32), positions=z(N, H, CAP, dt=I32), lens=z(N, dt=I32),
                seen=z(N, dt=I32), budget=20, block_table=z(N, MB, dt=I32), block_size=BS, **cache,
                scores_out=z(N, H, CAP, dt=F32), positions_out=z(N, H, CAP, dt=I32),
                lens_out=z(N, dt=I32), workspace=z(64, dt=U8))


SUM = dict(summary=z(SLOTS // BS, H, 2, D, dt=I8), exponents=z(SLOTS // BS, H, dt=U8))
SEL = dict(selected=z(T, H, K, dt=I32))
ENTRY = {
    "verify_tree": (c.shortconv_kv_verify_tree, lambda: verify(plain())),
    "verify_tree_mx": (c.shortconv_kv_verify_tree_mxfp8, lambda: verify(mx())),
    "tree": (c.shortconv_tree_attention, lambda: attn(plain(), mask=z(T, 1, dt=I64))),
    "tree_mx": (c.shortconv_tree_attention_mxfp8, lambda: attn(mx())),
    "summary": (c.shortconv_block_summary, lambda: dict(k_cache=z(SLOTS, H, D), **batch(), **SUM)),
    "summary_mx": (c.shortconv_block_summary_mxfp8, lambda: dict(**mx(("k",)), **batch(), **SUM)),
    "select": (c.shortconv_block_select,
               lambda: dict(q=z(T, G * H, D), **batch(), **SUM, **SEL, workspace=z(64, dt=U8))),
    "block": (c.shortconv_block_attention, lambda: attn(plain(), **SEL)),
    "block_mx": (c.shortconv_block_attention_mxfp8, lambda: attn(mx(), **SEL)),
    "scores": (c.shortconv_cache_scores, lambda: scores(plain(("k_cache",)))),
    "scores_mx": (c.shortconv_cache_scores_mxfp8, lambda: scores(mx(("k",)))),
    "evict": (c.shortconv_cache_evict, lambda: evict(plain())),
    "evict_mx": (c.shortconv_cache_evict_mxfp8, lambda: evict(mx())),
}


@pytest.mark.parametrize("entry", sorted(ENTRY))
def test_well_formed_arguments_reach_the_device_check(entry):
    fn, make = ENTRY[entry]
    with pytest.raises(ValueError, match="must be on a GPU"):
        fn(**make())


def strided(t):
    return torch.zeros(t.shape[:-1] + (2 * t.shape[-1],), dtype=t.dtype)[..., ::2]


ALL_BATCH = ("tree", "tree_mx", "summary", "summary_mx", "select", "block", "block_mx", "scores",
             "scores_mx")
BAD = [(e, a, f, m) for e in ALL_BATCH for a, f, m in (
    ("cu_seqlens", lambda t: t.to(I64), "cu_seqlens must be torch.int32"),
    ("context_lens", lambda t: z(N + 1, dt=I32), "context_lens must have shape"),
    ("context_lens", lambda t: t.to(I64), "context_lens must be torch.int32"),
    ("block_table", lambda t: z(N - 1, MB, dt=I32), "block_table must have shape"),
    ("block_table", lambda t: t.to(I64), "block_table must be torch.int32"),
    ("block_table", strided, "block_table must be contiguous"),
    ("block_size", lambda t: 12, "power of two"))]
BAD += [(e, a, f, m) for e in ("tree", "tree_mx", "block", "block_mx", "scores", "select")
        for a, f, m in (
    ("q", lambda t: z(T, G * H + 1, D), "multiple of the cache's"),
    ("q", lambda t: z(T, G * H, D, dt=torch.float16), "q must be"),
    ("q", lambda t: z(T, G * H, D // 2), "q must have shape"),
    ("q", lambda t: z(T, D, G * H).transpose(1, 2), "contiguous heads"))]
BAD += [(e, a, f, m) for e in ("tree", "tree_mx", "block", "block_mx") for a, f, m in (
    ("out", lambda t: z(T, G * H, D, dt=F32), "out must be torch.bfloat16"),
    ("out", lambda t: z(T + 1, G * H, D), "out must have shape"),
    ("out", strided, "out must be contiguous"),
    ("lse", lambda t: z(T, H, dt=F32), "lse must have shape"),
    ("lse", lambda t: z(T, G * H), "lse must be torch.float32"),
    ("workspace", lambda t: z(4, dt=F32), "workspace must be torch.uint8"))]
BAD += [
    ("tree", "q", lambda t: t.float(), "q must be torch.bfloat16 as the caches are"),
    ("block", "q", lambda t: t.float(), "q must be torch.bfloat16 as the caches are"),
    ("scores", "q", lambda t: t.float(), "q must be torch.bfloat16"),
    ("tree", "k_cache", lambda t: z(SLOTS, H, 96), "head_dim 64, 128 or 256"),
    ("tree", "k_cache", lambda t: z(SLOTS, H, D, dt=torch.float16), "k_cache must be"),
    ("tree", "v_cache", lambda t: z(SLOTS - 1, H, D), "v_cache must have shape"),
    ("tree", "v_cache", strided, "v_cache must be contiguous"),
    ("tree", "mask", lambda t: z(T, 1, dt=I32), "mask must be torch.int64"),
    ("tree", "mask", lambda t: z(T - 1, 1, dt=I64), "mask must have shape"),
    ("tree_mx", "k_codes", lambda t: z(SLOTS, H, D), "k_codes must be torch.uint8"),
    ("tree_mx", "v_scales", lambda t: z(SLOTS, H, D, dt=U8), "v_scales must have shape"),
    ("block", "selected", lambda t: t.to(I64), "selected must be torch.int32"),
    ("block", "selected", lambda t: z(T, H + 1, K, dt=I32), "selected must have shape"),
    ("select", "selected", lambda t: z(T - 1, H, K, dt=I32), "selected must have shape"),
    ("select", "summary", lambda t: z(SLOTS // BS, H, 2, D, dt=U8), "summary must be torch.int8"),
    ("select", "exponents", lambda t: z(SLOTS // BS, H + 1, dt=U8), "exponents must have shape"),
    ("summary", "summary", lambda t: z(SLOTS // BS - 1, H, 2, D, dt=I8), "summary must have shape"),
    ("summary", "exponents", lambda t: z(SLOTS // BS, H, dt=I8), "exponents must be torch.uint8"),
    ("summary_mx", "k_scales", lambda t: z(SLOTS, H, dt=U8), "k_scales must have shape"),
    ("scores", "scores", lambda t: z(N, H, CAP - 1, dt=F32), "scores must have shape"),
    ("scores", "scores_out", lambda t: z(N, H, CAP), "scores_out must be torch.float32"),
    ("scores", "lse", lambda t: None, "lse is required"),
    ("scores_mx", "k_scales", lambda t: z(SLOTS, H, D, dt=U8), "k_scales must have shape"),
    ("evict", "positions", lambda t: t.to(I64), "positions must be torch.int32"),
    ("evict", "positions", lambda t: z(N, H, CAP - 1, dt=I32), "positions must have shape"),
    ("evict", "lens", lambda t: z(N + 1, dt=I32), "lens must have shape"),
    ("evict", "seen", lambda t: t.to(I64), "seen must be torch.int32"),
    ("evict", "scores", lambda t: z(N, H + 1, CAP, dt=F32), "scores must have shape"),
    ("evict", "scores_out", strided, "scores_out must be contiguous"),
    ("evict", "lens_out", lambda t: None, "lens_out is required"),
    ("evict", "block_size", lambda t: 0, "power of two"),
    ("evict", "v_cache", lambda t: z(SLOTS, H, D, dt=F32), "v_cache must be torch.bfloat16"),
    ("evict_mx", "k_scales", lambda t: z(SLOTS, H, dt=U8), "k_scales must have shape"),
    ("verify_tree", "parents", lambda t: t.to(I64), "parents must be torch.int32"),
    ("verify_tree", "parents", lambda t: z(T + 1, dt=I32), "parents must have shape"),
    ("verify_tree", "mask", lambda t: z(T, 1, dt=I32), "mask must be torch.int64"),
    ("verify_tree", "k_snap", lambda t: z(N, M, W, H, D), "k_snap must have shape"),
    ("verify_tree", "v_snap", lambda t: z(N, M + 1, W - 1, H, D), "v_snap must have shape"),
    ("verify_tree", "slot_mapping", lambda t: t.to(I32), "slot_mapping must be torch.int64"),
    ("verify_tree", "v_cache", lambda t: z(SLOTS, H, D, dt=F32), "v_cache must be torch.bfloat16"),
    ("verify_tree_mx", "v_codes", lambda t: z(SLOTS, H, D), "v_codes must be torch.uint8"),
]


@pytest.mark.parametrize("entry,arg,make,msg", BAD,
                         ids=[f"{e}-{a}-{i}" for i, (e, a, _, _) in enumerate(BAD)])
def test_malformed_argument_is_rejected_before_the_library(entry, arg, make, msg):
    fn, good = ENTRY[entry]
    args = good()
    args[arg] = make(args[arg])
    with pytest.raises(ValueError, match=msg):
        fn(**args)


def test_tensors_on_different_devices_are_rejected():
    args = ENTRY["tree"][1]()
    args["block_table"] = args["block_table"].to("meta")
    with pytest.raises(ValueError, match="block_table is on meta"):
        c.shortconv_tree_attention(**args)
