"""ctypes binding of libshortconv_cache.so: the operators on the paged KV cache that the fused step
writes (include/shortconv_cache.h). Argument marshalling only, as in ``_binding``; there is no
fallback path of any kind.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

import torch

from ._binding import (SC_DTYPE, ShortConvError, _Args, _caches, _F32, _HERE, _I32, _I64,
                       _mx_caches, _ptr, _state_pools, _step_common, _stream_handle, _U8)

CACHE_LIBRARY_PATH = os.path.join(_HERE, "libshortconv_cache.so")

_lib = None


def load_cache_library(path: str = CACHE_LIBRARY_PATH):
    """Load the built library (raises if it is missing: there is no other implementation)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise ImportError(
            f"{path} is not built; run `python -m causal_short_convolution_amd.build` "
            "(the cache operators have no implementation other than this HIP library)")
    lib = ctypes.CDLL(path)
    P, I32, I64, F, Z = (ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float,
                         ctypes.c_size_t)
    verify = [P, P, I64, I64, P, I32, I64, P, P, P, P, P, F, P, P, I64, P, P, P, I32, P, I32, P]
    query = [P, I64, P, P, I32, I64, P, I32, I32]  # q .. block_size
    tail = [I32, I32, I32, I32, P]                 # num_q_heads, num_heads, head_dim, dtype, stream
    attn = [F, P, P, P, Z]                         # scale, out, lse, workspace, bytes
    summary = [P, P, I32, P, I32, I32, I64, I32, P, P, I32, I32]
    scores = [P, I64, P, P, P, I32, I64, P, I32, I32, P, I32]
    evict = [P, P, P, P, I32, I64, I32, I32, I32, P, I32, I32]
    evict_tail = [I64, P, P, P, P, Z, I32, I32]
    signatures = {
        "shortconv_kv_verify_tree": verify + [P, P, I64, I32, I32, I32, I32, P],
        "shortconv_kv_verify_tree_mxfp8": verify + [P, P, P, P, I64, I32, I32, I32, I32, P],
        "shortconv_tree_attention": query + [P, I32, P, P, I64] + attn + tail,
        "shortconv_tree_attention_mxfp8": query + [P, I32, P, P, P, P, I64] + attn + tail,
        "shortconv_block_summary": [P] + summary + [I32, P],
        "shortconv_block_summary_mxfp8": [P, P] + summary + [P],
        "shortconv_block_select": query + [I64, P, P, I32, I32, P, I32, P, Z] + tail,
        "shortconv_block_attention": query + [P, I32, P, P, I64] + attn + tail,
        "shortconv_block_attention_mxfp8": query + [P, I32, P, P, P, P, I64] + attn + tail,
        "shortconv_cache_scores": scores + [P, I64, F, P, P, I64] + tail,
        "shortconv_cache_scores_mxfp8": scores + [P, P, I64, F, P, P, I64] + tail,
        "shortconv_cache_evict": evict + [P, P] + evict_tail + [I32, P],
        "shortconv_cache_evict_mxfp8": evict + [P, P, P, P] + evict_tail + [P],
        "shortconv_cache_abi_version": [],
    }
    for name, argtypes in signatures.items():
        getattr(lib, name).restype = ctypes.c_int
        getattr(lib, name).argtypes = argtypes
    sizes = {
        "shortconv_tree_attention_workspace_size": [I64, I32, I32, I32, I32, I32],
        "shortconv_block_select_workspace_size": [I64, I32, I32],
        "shortconv_block_attention_workspace_size": [I64, I32, I32, I32, I32, I32, I32],
        "shortconv_cache_evict_workspace_size": [I32, I64, I32, I32],
    }
    for name, argtypes in sizes.items():
        getattr(lib, name).restype = ctypes.c_size_t
        getattr(lib, name).argtypes = argtypes
    lib.shortconv_cache_last_error.restype = ctypes.c_char_p
    lib.shortconv_cache_last_error.argtypes = []
    _lib = lib
    return lib


def cache_last_error() -> str:
    return load_cache_library().shortconv_cache_last_error().decode()


def cache_abi_version() -> int:
    return int(load_cache_library().shortconv_cache_abi_version())


def _check(rc: int):
    if rc != 0:
        raise ShortConvError(rc, cache_last_error())


def _size(n: int) -> int:
    if n == ctypes.c_size_t(-1).value:
        raise ShortConvError(-1, cache_last_error())
    return int(n)


def _code(dtype) -> int:
    return SC_DTYPE[dtype] if isinstance(dtype, torch.dtype) else int(dtype)


def _workspace(a: _Args, workspace, need: int, device, stream):
    """The caller's workspace, or one allocated here for the stream that the call runs on."""
    a.tensor(workspace, "workspace", _U8, (None,), optional=True)
    if workspace is None:
        if need == 0:
            return None
        workspace = torch.empty(need, dtype=torch.uint8, device=device)
        if stream is not None:  # allocated on the current stream, used on another
            stream.wait_stream(torch.cuda.current_stream(device))
            workspace.record_stream(stream)
    return workspace


def _nbytes(workspace) -> int:
    return 0 if workspace is None else workspace.numel()


def _tables(a: _Args, block_table, block_size, num_seqs):
    """block_table int32 [num_seqs, max_blocks]; returns (max_blocks, block_size)."""
    a.tensor(block_table, "block_table", _I32, (num_seqs, None))
    bs = int(block_size)
    if bs < 1 or bs > 65536 or bs & (bs - 1):
        a.fail(f"block_size must be a power of two in [1, 65536], got {block_size}")
    return block_table.shape[1], bs


def _batch(a: _Args, cu_seqlens, context_lens, block_table, block_size):
    """The batch and paging arguments; returns (num_seqs, max_blocks, block_size)."""
    a.tensor(cu_seqlens, "cu_seqlens", _I32, (None,))
    N = cu_seqlens.shape[0] - 1
    if N < 0:
        a.fail("cu_seqlens must hold at least one entry (num_seqs + 1)")
    a.tensor(context_lens, "context_lens", _I32, (N,))
    return (N, *_tables(a, block_table, block_size, N))


def _queries(a: _Args, q, H, D, dtypes=(torch.float32, torch.bfloat16)):
    """q [T, Hq, D] rows with Hq a multiple of H; returns (token stride, Hq)."""
    qs = a.rows(q, "q", None, D, dtypes)
    if q.shape[1] < 1 or q.shape[1] % H:
        a.fail(f"q must have a multiple of the cache's {H} heads, got {q.shape[1]}")
    return qs, q.shape[1]


def _mask(a: _Args, mask, T):
    a.tensor(mask, "mask", _I64, (T, None), optional=True)
    return 0 if mask is None else mask.shape[1]


def _cache_shape(a: _Args, k, name, dtypes):
    """Heads and head_dim of a cache tensor [num_slots, H, D]."""
    a.tensor(k, name, dtypes, (None, None, None))
    if k.shape[1] < 1 or k.shape[2] not in (64, 128, 256):
        a.fail(f"{name} must be [num_slots, heads, head_dim] with head_dim 64, 128 or 256, "
               f"got {list(k.shape)}")
    return k.shape[1], k.shape[2]


_ROWS = (torch.float32, torch.bfloat16)


# ------------------------------------------------------------------------------------------------
# The step over a tree of drafted tokens
# ------------------------------------------------------------------------------------------------
def _verify_tree(fn, k, v, cu_seqlens, parents, k_taps, v_taps, k_gamma, v_gamma, eps, k_state,
                 v_state, state_idx, k_snap, v_snap, slot_mapping, caches, mask, stream):
    a = _Args(fn)
    W, H, D, ks, vs, S = _step_common(a, k, v, k_taps, v_taps, k_gamma, v_gamma, k_state, v_state)
    T = k.shape[0]
    a.tensor(cu_seqlens, "cu_seqlens", _I32, (None,))
    N = cu_seqlens.shape[0] - 1
    if N < 0:
        a.fail("cu_seqlens must hold at least one entry (num_seqs + 1)")
    a.tensor(parents, "parents", _I32, (T,))
    a.tensor(state_idx, "state_idx", _I32, (N,), optional=True)
    a.tensor(slot_mapping, "slot_mapping", _I64, (T,))
    if W > 1 or k_snap is not None or v_snap is not None:
        a.tensor(k_snap, "k_snap", (k.dtype,), (N, None, W - 1, H, D))
        a.tensor(v_snap, "v_snap", (k.dtype,), (N, k_snap.shape[1], W - 1, H, D))
    max_tokens = k_snap.shape[1] if k_snap is not None else 1
    words = _mask(a, mask, T)
    nslots = _caches(a, *caches, H, D, k.dtype) if len(caches) == 2 else _mx_caches(a, *caches, H,
                                                                                  D)
    a.on_gpu()
    lib = load_cache_library()
    with torch.cuda.device(k.device):
        rc = getattr(lib, fn)(
            _ptr(k), _ptr(v), ks, vs, _ptr(cu_seqlens), N, T, _ptr(parents), _ptr(k_taps),
            _ptr(v_taps), _ptr(k_gamma), _ptr(v_gamma), float(eps), _ptr(k_state), _ptr(v_state),
            S, _ptr(state_idx), _ptr(k_snap), _ptr(v_snap), max_tokens, _ptr(mask), words,
            _ptr(slot_mapping), *map(_ptr, caches), nslots, H, D, W, SC_DTYPE[k.dtype],
            _stream_handle(k.device, stream))
    _check(rc)


def shortconv_kv_verify_tree(k, v, cu_seqlens, parents, k_taps, v_taps, k_gamma, v_gamma, eps,
                             k_state, v_state, state_idx, k_snap, v_snap, slot_mapping, k_cache,
                             v_cache, *, mask: Optional[torch.Tensor] = None,
                             stream: Optional[torch.cuda.Stream] = None) -> None:
    """``shortconv_kv_verify`` for drafted tokens that form a tree (see
    include/shortconv_cache.h): parents int32 [T], the index within its sequence of the token each
    one follows (less than its own; -1 for a root). mask int64 [T, words], written when given: the
    ancestors of each token and itself, for ``shortconv_tree_attention``. The other arguments are
    those of ``shortconv_kv_verify``."""
    _verify_tree("shortconv_kv_verify_tree", k, v, cu_seqlens, parents, k_taps, v_taps, k_gamma,
                 v_gamma, eps, k_state, v_state, state_idx, k_snap, v_snap, slot_mapping,
                 (k_cache, v_cache), mask, stream)


def shortconv_kv_verify_tree_mxfp8(k, v, cu_seqlens, parents, k_taps, v_taps, k_gamma, v_gamma,
                                   eps, k_state, v_state, state_idx, k_snap, v_snap, slot_mapping,
                                   k_codes, v_codes, k_scales, v_scales, *,
                                   mask: Optional[torch.Tensor] = None,
                                   stream: Optional[torch.cuda.Stream] = None) -> None:
    """``shortconv_kv_verify_tree`` writing MXFP8 cache rows."""
    _verify_tree("shortconv_kv_verify_tree_mxfp8", k, v, cu_seqlens, parents, k_taps, v_taps,
                 k_gamma, v_gamma, eps, k_state, v_state, state_idx, k_snap, v_snap, slot_mapping,
                 (k_codes, v_codes, k_scales, v_scales), mask, stream)


# ------------------------------------------------------------------------------------------------
# Attention over the cache
# ------------------------------------------------------------------------------------------------
def _kv(a: _Args, caches, q):
    """Checks the caches; returns (H, D, num_slots)."""
    if len(caches) == 2:
        H, D = _cache_shape(a, caches[0], "k_cache", _ROWS)
        n = _caches(a, *caches, H, D, caches[0].dtype)
        if isinstance(q, torch.Tensor) and q.dtype != caches[0].dtype:
            a.fail(f"q must be {caches[0].dtype} as the caches are, got {q.dtype}")
    else:
        H, D = _cache_shape(a, caches[0], "k_codes", _U8)
        n = _mx_caches(a, *caches, H, D)
    return H, D, n


def _outputs(a: _Args, out, lse, q):
    a.tensor(out, "out", (q.dtype,), tuple(q.shape))
    a.tensor(lse, "lse", _F32, tuple(q.shape[:2]), optional=True)


def shortconv_tree_attention_workspace_size(total_tokens, num_seqs, num_q_heads, num_heads,
                                            head_dim, dtype) -> int:
    """Bytes of workspace ``shortconv_tree_attention`` needs (dtype: the queries')."""
    return _size(load_cache_library().shortconv_tree_attention_workspace_size(
        int(total_tokens), int(num_seqs), int(num_q_heads), int(num_heads), int(head_dim),
        _code(dtype)))


def _tree_attention(fn, q, cu_seqlens, context_lens, block_table, block_size, caches, out, scale,
                    mask, lse, workspace, stream):
    a = _Args(fn)
    H, D, nslots = _kv(a, caches, q)
    qs, Hq = _queries(a, q, H, D)
    T = q.shape[0]
    N, MB, bs = _batch(a, cu_seqlens, context_lens, block_table, block_size)
    words = _mask(a, mask, T)
    _outputs(a, out, lse, q)
    a.tensor(workspace, "workspace", _U8, (None,), optional=True)
    a.on_gpu()
    lib = load_cache_library()
    need = shortconv_tree_attention_workspace_size(T, N, Hq, H, D, q.dtype)
    with torch.cuda.device(q.device):
        workspace = _workspace(a, workspace, need, q.device, stream)
        rc = getattr(lib, fn)(
            _ptr(q), qs, _ptr(cu_seqlens), _ptr(context_lens), N, T, _ptr(block_table), MB, bs,
            _ptr(mask), words, *map(_ptr, caches), nslots,
            float(D ** -0.5 if scale is None else scale), _ptr(out), _ptr(lse), _ptr(workspace),
            _nbytes(workspace), Hq, H, D, SC_DTYPE[q.dtype], _stream_handle(q.device, stream))
    _check(rc)


def shortconv_tree_attention(q, cu_seqlens, context_lens, block_table, block_size, k_cache,
                             v_cache, out, *, scale: Optional[float] = None,
                             mask: Optional[torch.Tensor] = None,
                             lse: Optional[torch.Tensor] = None,
                             workspace: Optional[torch.Tensor] = None,
                             stream: Optional[torch.cuda.Stream] = None) -> None:
    """Attention of the new tokens of each sequence over its cached keys and the new tokens that
    ``mask`` names (see include/shortconv_cache.h).

    q, out [T,Hq,D] of the caches' dtype (q: any token stride); cu_seqlens int32 [N+1];
    context_lens int32 [N], the keys cached before the new tokens (whose rows are in the cache
    too); block_table int32 [N,max_blocks]; caches [num_slots,H,D] with Hq a multiple of H; scale
    defaults to D**-0.5; mask int64 [T,words] or None (a chain); lse fp32 [T,Hq], written when
    given. ``workspace`` (a uint8 device tensor) is allocated here when not given.
    """
    _tree_attention("shortconv_tree_attention", q, cu_seqlens, context_lens, block_table,
                    block_size, (k_cache, v_cache), out, scale, mask, lse, workspace, stream)


def shortconv_tree_attention_mxfp8(q, cu_seqlens, context_lens, block_table, block_size, k_codes,
                                   v_codes, k_scales, v_scales, out, *,
                                   scale: Optional[float] = None,
                                   mask: Optional[torch.Tensor] = None,
                                   lse: Optional[torch.Tensor] = None,
                                   workspace: Optional[torch.Tensor] = None,
                                   stream: Optional[torch.cuda.Stream] = None) -> None:
    """``shortconv_tree_attention`` over MXFP8 cache rows; q and out fp32 or bf16."""
    _tree_attention("shortconv_tree_attention_mxfp8", q, cu_seqlens, context_lens, block_table,
                    block_size, (k_codes, v_codes, k_scales, v_scales), out, scale, mask, lse,
                    workspace, stream)


# ------------------------------------------------------------------------------------------------
# Attention over selected pages
# ------------------------------------------------------------------------------------------------
def _summary(a: _Args, summary, exponents, H, D, num_slots, block_size):
    pages = num_slots // block_size
    a.tensor(summary, "summary", (torch.int8,), (pages, H, 2, D))
    a.tensor(exponents, "exponents", _U8, (pages, H))


def _block_summary(fn, cache, cu_seqlens, context_lens, block_table, block_size, summary,
                   exponents, rebuild, stream):
    a = _Args(fn)
    mx = len(cache) == 2
    H, D = _cache_shape(a, cache[0], "k_codes" if mx else "k_cache", _U8 if mx else _ROWS)
    nslots = cache[0].shape[0]
    if mx:
        a.tensor(cache[1], "k_scales", _U8, (nslots, H, D // 32))
    N, MB, bs = _batch(a, cu_seqlens, context_lens, block_table, block_size)
    _summary(a, summary, exponents, H, D, nslots, bs)
    a.on_gpu()
    lib = load_cache_library()
    dev = summary.device
    with torch.cuda.device(dev):
        rc = getattr(lib, fn)(
            *map(_ptr, cache), _ptr(cu_seqlens), _ptr(context_lens), N, _ptr(block_table), MB, bs, nslots, int(bool(rebuild)), _ptr(summary),
            _ptr(exponents), H, D, *([] if mx else [SC_DTYPE[cache[0].dtype]]),
            _stream_handle(dev, stream))
    _check(rc)


def shortconv_block_summary(k_cache, cu_seqlens, context_lens, block_table, block_size, summary,
                            exponents, *, rebuild: bool = False,
                            stream: Optional[torch.cuda.Stream] = None) -> None:
    """Minimum and maximum of each page's keys per head and channel, as int8 codes with one
    power of two per page and head (see include/shortconv_cache.h): summary int8
    [num_slots // block_size, H, 2, D], exponents uint8 [num_slots // block_size, H]. Only the
    pages that the new tokens touch are written, with ``rebuild`` every page of every sequence."""
    _block_summary("shortconv_block_summary", (k_cache,), cu_seqlens, context_lens, block_table,
                   block_size, summary, exponents, rebuild, stream)


def shortconv_block_summary_mxfp8(k_codes, k_scales, cu_seqlens, context_lens, block_table,
                                  block_size, summary, exponents, *, rebuild: bool = False,
                                  stream: Optional[torch.cuda.Stream] = None) -> None:
    """``shortconv_block_summary`` of MXFP8 keys."""
    _block_summary("shortconv_block_summary_mxfp8", (k_codes, k_scales), cu_seqlens, context_lens,
                   block_table, block_size, summary, exponents, rebuild, stream)


def shortconv_block_select_workspace_size(total_tokens, max_blocks, num_heads) -> int:
    """Bytes of workspace ``shortconv_block_select`` needs."""
    return _size(load_cache_library().shortconv_block_select_workspace_size(
        int(total_tokens), int(max_blocks), int(num_heads)))


def shortconv_block_select(q, cu_seqlens, context_lens, block_table, block_size, summary,
                           exponents, selected, *, sink_blocks: int = 1, recent_blocks: int = 1,
                           workspace: Optional[torch.Tensor] = None,
                           stream: Optional[torch.cuda.Stream] = None) -> None:
    """The pages each new token reads, per cache head (see include/shortconv_cache.h): the first
    ``sink_blocks`` and the last ``recent_blocks`` of its pages and those with the largest scores
    against ``summary``. selected int32 [T,H,topk], written: ascending indexes into the sequence's
    block_table row, -1 behind them."""
    a = _Args("shortconv_block_select")
    a.tensor(summary, "summary", (torch.int8,), (None, None, 2, None))
    pages, H, _, D = summary.shape
    a.tensor(exponents, "exponents", _U8, (pages, H))
    if H < 1:
        a.fail("summary must have at least one head")
    qs, Hq = _queries(a, q, H, D)
    T = q.shape[0]
    N, MB, bs = _batch(a, cu_seqlens, context_lens, block_table, block_size)
    a.tensor(selected, "selected", _I32, (T, H, None))
    a.tensor(workspace, "workspace", _U8, (None,), optional=True)
    a.on_gpu()
    lib = load_cache_library()
    need = shortconv_block_select_workspace_size(T, MB, H)
    with torch.cuda.device(q.device):
        workspace = _workspace(a, workspace, need, q.device, stream)
        rc = lib.shortconv_block_select(
            _ptr(q), qs, _ptr(cu_seqlens), _ptr(context_lens), N, T, _ptr(block_table), MB, bs,
            pages * bs, _ptr(summary), _ptr(exponents), int(sink_blocks), int(recent_blocks),
            _ptr(selected), selected.shape[2], _ptr(workspace), _nbytes(workspace), Hq, H, D,
            SC_DTYPE[q.dtype], _stream_handle(q.device, stream))
    _check(rc)


def shortconv_block_attention_workspace_size(total_tokens, topk, block_size, num_q_heads,
                                             num_heads, head_dim, dtype) -> int:
    """Bytes of workspace ``shortconv_block_attention`` needs (dtype: the queries')."""
    return _size(load_cache_library().shortconv_block_attention_workspace_size(
        int(total_tokens), int(topk), int(block_size), int(num_q_heads), int(num_heads),
        int(head_dim), _code(dtype)))


def _block_attention(fn, q, cu_seqlens, context_lens, block_table, block_size, selected, caches,
                     out, scale, lse, workspace, stream):
    a = _Args(fn)
    H, D, nslots = _kv(a, caches, q)
    qs, Hq = _queries(a, q, H, D)
    T = q.shape[0]
    N, MB, bs = _batch(a, cu_seqlens, context_lens, block_table, block_size)
    a.tensor(selected, "selected", _I32, (T, H, None))
    topk = selected.shape[2]
    _outputs(a, out, lse, q)
    a.tensor(workspace, "workspace", _U8, (None,), optional=True)
    a.on_gpu()
    lib = load_cache_library()
    need = shortconv_block_attention_workspace_size(T, topk, bs, Hq, H, D, q.dtype)
    with torch.cuda.device(q.device):
        workspace = _workspace(a, workspace, need, q.device, stream)
        rc = getattr(lib, fn)(
            _ptr(q), qs, _ptr(cu_seqlens), _ptr(context_lens), N, T, _ptr(block_table), MB, bs,
            _ptr(selected), topk, *map(_ptr, caches), nslots,
            float(D ** -0.5 if scale is None else scale), _ptr(out), _ptr(lse), _ptr(workspace),
            _nbytes(workspace), Hq, H, D, SC_DTYPE[q.dtype], _stream_handle(q.device, stream))
    _check(rc)


def shortconv_block_attention(q, cu_seqlens, context_lens, block_table, block_size, selected,
                              k_cache, v_cache, out, *, scale: Optional[float] = None,
                              lse: Optional[torch.Tensor] = None,
                              workspace: Optional[torch.Tensor] = None,
                              stream: Optional[torch.cuda.Stream] = None) -> None:
    """Attention of each new token over the keys of its selected pages, up to its own position (see
    include/shortconv_cache.h). selected int32 [T,H,topk] as ``shortconv_block_select`` writes
    it; the other arguments are those of ``shortconv_tree_attention``."""
    _block_attention("shortconv_block_attention", q, cu_seqlens, context_lens, block_table,
                     block_size, selected, (k_cache, v_cache), out, scale, lse, workspace, stream)


def shortconv_block_attention_mxfp8(q, cu_seqlens, context_lens, block_table, block_size, selected,
                                    k_codes, v_codes, k_scales, v_scales, out, *,
                                    scale: Optional[float] = None,
                                    lse: Optional[torch.Tensor] = None,
                                    workspace: Optional[torch.Tensor] = None,
                                    stream: Optional[torch.cuda.Stream] = None) -> None:
    """``shortconv_block_attention`` over MXFP8 cache rows; q and out fp32 or bf16."""
    _block_attention("shortconv_block_attention_mxfp8", q, cu_seqlens, context_lens, block_table,
                     block_size, selected, (k_codes, v_codes, k_scales, v_scales), out, scale, lse,
                     workspace, stream)


# ------------------------------------------------------------------------------------------------
# Accumulated attention weight and eviction by it
# ------------------------------------------------------------------------------------------------
def _cache_scores(fn, q, lse, cu_seqlens, context_lens, block_table, block_size, cache, scores,
                  scores_out, scale, mask, stream):
    a = _Args(fn)
    mx = len(cache) == 2
    H, D = _cache_shape(a, cache[0], "k_codes" if mx else "k_cache", _U8 if mx else _ROWS)
    nslots = cache[0].shape[0]
    if mx:
        a.tensor(cache[1], "k_scales", _U8, (nslots, H, D // 32))
    qs, Hq = _queries(a, q, H, D, _ROWS if mx else (cache[0].dtype,))
    T = q.shape[0]
    a.tensor(lse, "lse", _F32, (T, Hq))
    N, MB, bs = _batch(a, cu_seqlens, context_lens, block_table, block_size)
    words = _mask(a, mask, T)
    a.tensor(scores_out, "scores_out", _F32, (N, H, None))
    a.tensor(scores, "scores", _F32, tuple(scores_out.shape), optional=True)
    a.on_gpu()
    lib = load_cache_library()
    with torch.cuda.device(q.device):
        rc = getattr(lib, fn)(
            _ptr(q), qs, _ptr(lse), _ptr(cu_seqlens), _ptr(context_lens), N, T, _ptr(block_table),
            MB, bs, _ptr(mask), words, *map(_ptr, cache), nslots,
            float(D ** -0.5 if scale is None else scale), _ptr(scores), _ptr(scores_out),
            scores_out.shape[2], Hq, H, D, SC_DTYPE[q.dtype], _stream_handle(q.device, stream))
    _check(rc)


def shortconv_cache_scores(q, lse, cu_seqlens, context_lens, block_table, block_size, k_cache,
                           scores, scores_out, *, scale: Optional[float] = None,
                           mask: Optional[torch.Tensor] = None,
                           stream: Optional[torch.cuda.Stream] = None) -> None:
    """Adds the attention weight that each key receives from the queries to ``scores`` (fp32
    [N,H,capacity], or None for zeros; new tokens start from zero), into ``scores_out`` (which may
    be ``scores``). lse fp32 [T,Hq] as the attention returned it; scale and mask as it was given
    them (see include/shortconv_cache.h)."""
    _cache_scores("shortconv_cache_scores", q, lse, cu_seqlens, context_lens, block_table,
                  block_size, (k_cache,), scores, scores_out, scale, mask, stream)


def shortconv_cache_scores_mxfp8(q, lse, cu_seqlens, context_lens, block_table, block_size,
                                 k_codes, k_scales, scores, scores_out, *,
                                 scale: Optional[float] = None,
                                 mask: Optional[torch.Tensor] = None,
                                 stream: Optional[torch.cuda.Stream] = None) -> None:
    """``shortconv_cache_scores`` over MXFP8 keys; q fp32 or bf16."""
    _cache_scores("shortconv_cache_scores_mxfp8", q, lse, cu_seqlens, context_lens, block_table,
                  block_size, (k_codes, k_scales), scores, scores_out, scale, mask, stream)


def shortconv_cache_evict_workspace_size(num_seqs, capacity, budget, num_heads) -> int:
    """Bytes of workspace ``shortconv_cache_evict`` needs."""
    return _size(load_cache_library().shortconv_cache_evict_workspace_size(
        int(num_seqs), int(capacity), int(budget), int(num_heads)))


def _cache_evict(fn, scores, positions, lens, seen, budget, block_table, block_size, caches,
                 scores_out, positions_out, lens_out, sinks, recent, workspace, stream):
    a = _Args(fn)
    mx = len(caches) == 4
    H, D = _cache_shape(a, caches[0], "k_codes" if mx else "k_cache", _U8 if mx else _ROWS)
    nslots = _mx_caches(a, *caches, H, D) if mx else _caches(a, *caches, H, D, caches[0].dtype)
    a.tensor(scores, "scores", _F32, (None, H, None))
    N, _, cap = scores.shape
    a.tensor(positions, "positions", _I32, (N, H, cap))
    a.tensor(lens, "lens", _I32, (N,))
    a.tensor(seen, "seen", _I32, (N,))
    a.tensor(scores_out, "scores_out", _F32, (N, H, cap))
    a.tensor(positions_out, "positions_out", _I32, (N, H, cap))
    a.tensor(lens_out, "lens_out", _I32, (N,))
    MB, bs = _tables(a, block_table, block_size, N)
    a.tensor(workspace, "workspace", _U8, (None,), optional=True)
    a.on_gpu()
    lib = load_cache_library()
    dev = scores.device
    need = shortconv_cache_evict_workspace_size(N, cap, budget, H)
    with torch.cuda.device(dev):
        workspace = _workspace(a, workspace, need, dev, stream)
        rc = getattr(lib, fn)(
            _ptr(scores), _ptr(positions), _ptr(lens), _ptr(seen), N, cap, int(budget), int(sinks),
            int(recent), _ptr(block_table), MB, bs, *map(_ptr, caches), nslots, _ptr(scores_out),
            _ptr(positions_out), _ptr(lens_out), _ptr(workspace), _nbytes(workspace), H, D,
            *([] if mx else [SC_DTYPE[caches[0].dtype]]), _stream_handle(dev, stream))
    _check(rc)


def shortconv_cache_evict(scores, positions, lens, seen, budget, block_table, block_size, k_cache,
                          v_cache, scores_out, positions_out, lens_out, *, sinks: int = 0,
                          recent: int = 0, workspace: Optional[torch.Tensor] = None,
                          stream: Optional[torch.cuda.Stream] = None) -> None:
    """Keeps at most ``budget`` entries per sequence and head (see include/shortconv_cache.h):
    those at positions below ``sinks`` or among the last ``recent`` of ``seen``, then the ones with
    the largest scores. Kept entries past the budget move into the holes below it, in the caches,
    in scores_out and in positions_out; lens_out gets the new lengths. scores, scores_out fp32
    and positions, positions_out int32 [N,H,capacity]; lens, seen, lens_out int32 [N]. An output
    may be its input."""
    _cache_evict("shortconv_cache_evict", scores, positions, lens, seen, budget, block_table,
                 block_size, (k_cache, v_cache), scores_out, positions_out, lens_out, sinks,
                 recent, workspace, stream)


def shortconv_cache_evict_mxfp8(scores, positions, lens, seen, budget, block_table, block_size,
                                k_codes, v_codes, k_scales, v_scales, scores_out, positions_out,
                                lens_out, *, sinks: int = 0, recent: int = 0,
                                workspace: Optional[torch.Tensor] = None,
                                stream: Optional[torch.cuda.Stream] = None) -> None:
    """``shortconv_cache_evict`` of MXFP8 cache rows."""
    _cache_evict("shortconv_cache_evict_mxfp8", scores, positions, lens, seen, budget, block_table,
                 block_size, (k_codes, v_codes, k_scales, v_scales), scores_out, positions_out,
                 lens_out, sinks, recent, workspace, stream)
