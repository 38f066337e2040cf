"""The cache operators' C-ABI library on the host (no GPU): it loads, exports every symbol
include/shortconv_cache.h declares and nothing else, and rejects bad arguments before anything
reaches the HIP runtime. Pointers are fake integers that no call dereferences: every call either
fails validation or returns SC_OK without launching.
"""
import ctypes
import os
import re
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "shortconv_cache.h")
FAKE = 0x100000
INVALID, UNSUPPORTED = -1, -2


@pytest.fixture(scope="module")
def lib():
    from causal_short_convolution_amd import _cache
    if not os.path.exists(_cache.CACHE_LIBRARY_PATH):
        from causal_short_convolution_amd import build
        build.build()
    return _cache.load_cache_library()


def declared():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    return set(re.findall(r"\b(shortconv_\w+)\s*\(", text))


def test_library_exports_the_header_and_nothing_else(lib):
    from causal_short_convolution_amd import _cache
    out = subprocess.run(["nm", "-D", "--defined-only", _cache.CACHE_LIBRARY_PATH], check=True,
                         capture_output=True, text=True).stdout
    assert {line.split()[-1] for line in out.splitlines() if " T " in line} == declared()
    assert len(declared()) == 19


def test_abi_version(lib):
    v = int(re.search(r"#define SHORTCONV_CACHE_ABI_VERSION (\d+)", open(HEADER).read()).group(1))
    assert lib.shortconv_cache_abi_version() == v


P = FAKE
VERIFY = dict(k=P, v=P, ks=1024, vs=1024, cu=P, n=2, T=10, par=P, kt=P, vt=P, kg=P, vg=P, eps=1e-6,
              kst=P, vst=P, S=2, sidx=P, ksn=P, vsn=P, M=8, mask=P, words=1, slot=P, kc=P, vc=P,
              slots=100, H=8, D=128, W=4, dtype=1, stream=None)
VERIFY_MX = {**{k: v for k, v in list(VERIFY.items())[:25]}, "kcs": P, "vcs": P,
             **{k: v for k, v in list(VERIFY.items())[25:]}}
QUERY = dict(q=P, qs=4096, cu=P, ctx=P, n=2, T=10, table=P, mb=8, bs=16)
TAIL = dict(Hq=32, H=8, D=128, dtype=1, stream=None)
ATTN = dict(scale=0.1, out=P, lse=P, ws=P, wsb=1 << 62)
TREE = {**QUERY, "mask": P, "words": 1, "kc": P, "vc": P, "slots": 128, **ATTN, **TAIL}
TREE_MX = {**QUERY, "mask": P, "words": 1, "kc": P, "vc": P, "ksc": P, "vsc": P, "slots": 128,
           **ATTN, **TAIL}
BLOCK = {**QUERY, "sel": P, "topk": 4, "kc": P, "vc": P, "slots": 128, **ATTN, **TAIL}
BLOCK_MX = {**QUERY, "sel": P, "topk": 4, "kc": P, "vc": P, "ksc": P, "vsc": P, "slots": 128,
            **ATTN, **TAIL}
SUMMARY = dict(kc=P, cu=P, ctx=P, n=2, table=P, mb=8, bs=16, slots=128, rebuild=0, sum=P, exps=P,
               H=8, D=128, dtype=1, stream=None)
SUMMARY_MX = dict(kc=P, ksc=P, cu=P, ctx=P, n=2, table=P, mb=8, bs=16, slots=128, rebuild=0, sum=P,
                  exps=P, H=8, D=128, stream=None)
SELECT = {**QUERY, "slots": 128, "sum": P, "exps": P, "sinks": 1, "recents": 1, "sel": P,
          "topk": 4, "ws": P, "wsb": 1 << 62, **TAIL}
SCORES = dict(q=P, qs=4096, lse=P, cu=P, ctx=P, n=2, T=10, table=P, mb=8, bs=16, mask=P, words=1,
              kc=P, slots=128, scale=0.1, sin=P, sout=P, cap=128, **TAIL)
SCORES_MX = dict(q=P, qs=4096, lse=P, cu=P, ctx=P, n=2, T=10, table=P, mb=8, bs=16, mask=P,
                 words=1, kc=P, ksc=P, slots=128, scale=0.1, sin=P, sout=P, cap=128, **TAIL)
EVICT = dict(sc=P, pos=P, lens=P, seen=P, n=2, cap=128, budget=64, sinks=1, recent=4, table=P, mb=8,
             bs=16, kc=P, vc=P, slots=128, so=P, po=P, lo=P, ws=P, wsb=1 << 62, H=8, D=128, dtype=1,
             stream=None)
EVICT_MX = dict(sc=P, pos=P, lens=P, seen=P, n=2, cap=128, budget=64, sinks=1, recent=4, table=P,
                mb=8, bs=16, kc=P, vc=P, ksc=P, vsc=P, slots=128, so=P, po=P, lo=P, ws=P,
                wsb=1 << 62, H=8, D=128, stream=None)

SHAPES = [(dict(dtype=7), UNSUPPORTED, "dtype"), (dict(D=96), UNSUPPORTED, "head_dim"),
          (dict(H=0), INVALID, "num_heads"), (dict(H=1 << 20), UNSUPPORTED, "num_heads too large")]
PAGES = [(dict(bs=0), UNSUPPORTED, "block_size"), (dict(bs=24), UNSUPPORTED, "block_size"),
         (dict(bs=1 << 17), UNSUPPORTED, "block_size"), (dict(mb=-1), INVALID, "negative"),
         (dict(mb=1 << 28), UNSUPPORTED, "max_blocks"), (dict(slots=-1), INVALID, "negative"),
         (dict(slots=1 << 31), UNSUPPORTED, "num_slots"), (dict(table=None), INVALID, "block_table")]
BATCH = [(dict(n=-1), INVALID, "num_seqs"), (dict(n=70000), UNSUPPORTED, "65535"),
         (dict(cu=None), INVALID, "cu_seqlens"), (dict(ctx=None), INVALID, "context_lens")]
TOKENS = [(dict(T=-1), INVALID, "total_tokens"), (dict(T=1 << 31), INVALID, "total_tokens")]
HEADS = [(dict(Hq=12), INVALID, "multiple"), (dict(Hq=4), INVALID, "multiple"),
         (dict(Hq=1 << 20), UNSUPPORTED, "num_q_heads"), (dict(q=None), INVALID, "null q"),
         (dict(qs=100), INVALID, "stride"), (dict(qs=4097), INVALID, "16 bytes"),
         (dict(q=P + 8), INVALID, "aligned")]
KV = [(dict(kc=None), INVALID, "cache"), (dict(vc=None), INVALID, "cache"),
      (dict(kc=P + 4), INVALID, "aligned")]
SCALES = [(dict(ksc=None), INVALID, "cache")]
COMMON = SHAPES + PAGES + BATCH + TOKENS + HEADS
ATT = COMMON + KV + [(dict(scale=float("nan")), INVALID, "scale"),
                     (dict(scale=float("inf")), INVALID, "scale"),
                     (dict(out=None), INVALID, "out"), (dict(out=P + 8), INVALID, "aligned")]
WORDS = [(dict(words=-1), INVALID, "mask_words")]
NO_TYPE = [c for c in SHAPES if "dtype" not in c[0]]

CASES = {
    "shortconv_kv_verify_tree": (VERIFY, SHAPES + TOKENS + WORDS + [
        (dict(W=0), UNSUPPORTED, "width"), (dict(W=9), UNSUPPORTED, "width"),
        (dict(n=-1), INVALID, "num_seqs"), (dict(M=0), INVALID, "max_tokens"),
        (dict(S=-1), INVALID, "num_state_slots"), (dict(slots=-1), INVALID, "num_slots"),
        (dict(eps=-1.0), INVALID, "eps"), (dict(eps=float("nan")), INVALID, "eps"),
        (dict(kt=None), INVALID, "taps"), (dict(vst=None), INVALID, "conv state"),
        (dict(cu=None), INVALID, "cu_seqlens"), (dict(par=None), INVALID, "parents"),
        (dict(slot=None), INVALID, "slot_mapping"), (dict(kc=None), INVALID, "cache"),
        (dict(ksn=None), INVALID, "snapshot"), (dict(k=None), INVALID, "null K"),
        (dict(vs=8), INVALID, "stride"), (dict(ks=1028), INVALID, "16 bytes"),
        (dict(v=P + 8), INVALID, "aligned")]),
    "shortconv_kv_verify_tree_mxfp8": (VERIFY_MX, SHAPES + [(dict(kcs=None), INVALID, "cache")]),
    "shortconv_tree_attention": (TREE, ATT + WORDS),
    "shortconv_tree_attention_mxfp8": (TREE_MX, ATT + WORDS + SCALES +
                                       [(dict(vsc=None), INVALID, "cache")]),
    "shortconv_block_attention": (BLOCK, ATT + [(dict(topk=-1), INVALID, "topk"),
                                                (dict(sel=None), INVALID, "selected")]),
    "shortconv_block_attention_mxfp8": (BLOCK_MX, ATT + SCALES),
    "shortconv_block_summary": (SUMMARY, SHAPES + PAGES + BATCH + [
        (dict(kc=None), INVALID, "cache"), (dict(sum=None), INVALID, "summary"),
        (dict(exps=None), INVALID, "summary or exponents"), (dict(sum=P + 4), INVALID, "aligned")]),
    "shortconv_block_summary_mxfp8": (SUMMARY_MX, NO_TYPE + PAGES + SCALES),
    "shortconv_block_select": (SELECT, COMMON + [
        (dict(topk=-1), INVALID, "topk"), (dict(sinks=-1), INVALID, "sink_blocks"),
        (dict(recents=-1), INVALID, "recent_blocks"), (dict(sel=None), INVALID, "selected"),
        (dict(sum=None), INVALID, "summary"),
        (dict(H=1, Hq=2048, qs=1 << 20), UNSUPPORTED, "query heads per cache head")]),
    "shortconv_cache_scores": (SCORES, COMMON + WORDS + [
        (dict(kc=None), INVALID, "cache"), (dict(lse=None), INVALID, "lse"),
        (dict(sout=None), INVALID, "scores_out"), (dict(cap=-1), INVALID, "capacity"),
        (dict(scale=float("nan")), INVALID, "scale")]),
    "shortconv_cache_scores_mxfp8": (SCORES_MX, COMMON + SCALES),
    "shortconv_cache_evict": (EVICT, SHAPES + PAGES + KV + [
        (dict(budget=-1), INVALID, "negative"), (dict(sinks=-1), INVALID, "negative"),
        (dict(recent=-1), INVALID, "negative"), (dict(n=-1), INVALID, "negative"),
        (dict(n=70000), UNSUPPORTED, "65535"), (dict(cap=1 << 31), UNSUPPORTED, "capacity"),
        (dict(lens=None), INVALID, "lens"), (dict(seen=None), INVALID, "seen"),
        (dict(lo=None), INVALID, "lens_out"), (dict(sc=None), INVALID, "scores"),
        (dict(po=None), INVALID, "positions"), (dict(ws=None), INVALID, "workspace"),
        (dict(wsb=16), INVALID, "workspace"), (dict(ws=P + 4), INVALID, "aligned")]),
    "shortconv_cache_evict_mxfp8": (EVICT_MX, NO_TYPE + PAGES + KV + SCALES),
}
FLAT = [(fn, over, code, msg) for fn, (_, cases) in CASES.items() for over, code, msg in cases]


@pytest.mark.parametrize("fn,over,code,msg", FLAT,
                         ids=[f"{f[10:]}-{'-'.join(o)}-{i}" for i, (f, o, _, _) in enumerate(FLAT)])
def test_rejects(lib, fn, over, code, msg):
    args = {**CASES[fn][0], **over}
    rc = getattr(lib, fn)(*args.values())
    err = lib.shortconv_cache_last_error().decode()
    assert rc == code, err
    assert err.startswith(fn + ":") and msg in err, err


@pytest.mark.parametrize("fn,over", [
    ("shortconv_kv_verify_tree", dict(n=0)), ("shortconv_kv_verify_tree", dict(T=0, k=None)),
    ("shortconv_tree_attention", dict(n=0, cu=None, ctx=None, table=None)),
    ("shortconv_tree_attention", dict(T=0, q=None, out=None)),
    ("shortconv_block_attention", dict(n=0)), ("shortconv_block_summary", dict(n=0)),
    ("shortconv_block_summary", dict(slots=15, kc=None)),
    ("shortconv_block_select", dict(topk=0, sel=None)), ("shortconv_block_select", dict(T=0)),
    ("shortconv_cache_scores", dict(n=0)), ("shortconv_cache_scores", dict(cap=0, sout=None)),
    ("shortconv_cache_evict", dict(n=0)),
])
def test_nothing_to_do(lib, fn, over):
    args = {**CASES[fn][0], **over}
    assert getattr(lib, fn)(*args.values()) == 0, lib.shortconv_cache_last_error()
    assert lib.shortconv_cache_last_error() == b""


def test_workspace_sizes(lib):
    bad = ctypes.c_size_t(-1).value
    f = lib.shortconv_cache_evict_workspace_size
    assert f(2, 128, 64, 8) == 2 * 8 * (1 + 2 * 64) * 4
    assert f(2, 128, 100, 8) == 2 * 8 * (1 + 2 * 28) * 4   # at most the entries past the budget
    assert f(2, 64, 64, 8) == 2 * 8 * 4
    assert f(-1, 64, 64, 8) == bad and f(1, 64, -1, 8) == bad and f(1, 64, 1, 0) == bad
    f = lib.shortconv_tree_attention_workspace_size
    assert f(0, 0, 8, 8, 128, 1) != bad
    assert f(-1, 1, 8, 8, 128, 1) == bad and f(1, 1, 9, 8, 128, 1) == bad
    assert f(1, 1, 8, 8, 96, 1) == bad and f(1, 1, 8, 8, 128, 2) == bad
    f = lib.shortconv_block_attention_workspace_size
    assert f(1, 4, 16, 8, 8, 128, 1) != bad and f(1, -4, 16, 8, 8, 128, 1) == bad
    f = lib.shortconv_block_select_workspace_size
    assert f(-1, 4, 8) == bad and f(4, 4, 0) == bad and f(4, 4, 8) != bad
