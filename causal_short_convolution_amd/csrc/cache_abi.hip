// C ABI of the cache operators: host-side validation, problem geometry and launch. The operations,
// layouts and error behaviour are specified in include/shortconv_cache.h.
#include <stdarg.h>
#include <stdio.h>

#include "cache_internal.h"
#include "shortconv_cache.h"

#define SC_API extern "C" __attribute__((visibility("default")))

namespace {

thread_local char g_err[512] = "";

int fail(int code, const char* fmt, ...) {
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(g_err, sizeof g_err, fmt, ap);
    va_end(ap);
    return code;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int element_bytes(int32_t dtype) { return dtype == SC_DTYPE_F32 ? 4 : 2; }

int launched(const char* fn, hipError_t e) {
    if (e != hipSuccess) return fail(SC_ERR_HIP, "%s: launch failed: %s", fn, hipGetErrorString(e));
    return SC_OK;
}

int check_shape(const char* fn, int32_t heads, int32_t D, int32_t dtype) {
    if (dtype != SC_DTYPE_F32 && dtype != SC_DTYPE_BF16)
        return fail(SC_ERR_UNSUPPORTED, "%s: unknown dtype %d", fn, dtype);
    if (D != 64 && D != 128 && D != 256)
        return fail(SC_ERR_UNSUPPORTED, "%s: head_dim %d not in {64, 128, 256}", fn, D);
    if (heads < 1) return fail(SC_ERR_INVALID, "%s: num_heads %d < 1", fn, heads);
    if ((int64_t)heads * D > (int64_t)1 << 20)
        return fail(SC_ERR_UNSUPPORTED, "%s: num_heads too large", fn);
    return SC_OK;
}

int check_queries(const char* fn, int32_t q_heads, int32_t heads, int32_t D) {
    if (q_heads < heads || q_heads % heads)
        return fail(SC_ERR_INVALID, "%s: num_q_heads %d is not a multiple of num_heads %d", fn,
                    q_heads, heads);
    if ((int64_t)q_heads * D > (int64_t)1 << 20)
        return fail(SC_ERR_UNSUPPORTED, "%s: num_q_heads too large", fn);
    return SC_OK;
}

int check_paging(const char* fn, const int32_t* table, int32_t max_blocks, int32_t block_size,
                 int64_t num_slots, int32_t num_seqs) {
    if (block_size < 1 || block_size > 65536 || (block_size & (block_size - 1)))
        return fail(SC_ERR_UNSUPPORTED, "%s: block_size %d is not a power of two in [1, 65536]", fn,
                    block_size);
    if (max_blocks < 0 || num_slots < 0) return fail(SC_ERR_INVALID, "%s: negative size", fn);
    if ((int64_t)max_blocks * block_size > INT32_MAX)
        return fail(SC_ERR_UNSUPPORTED, "%s: max_blocks * block_size must be below 2^31", fn);
    if (num_slots > INT32_MAX)
        return fail(SC_ERR_UNSUPPORTED, "%s: num_slots must be below 2^31", fn);
    if (num_seqs > 0 && max_blocks > 0 && !table)
        return fail(SC_ERR_INVALID, "%s: null block_table", fn);
    return SC_OK;
}

int check_batch(const char* fn, const int32_t* cu, const int32_t* ctx, int32_t num_seqs,
                int64_t tokens) {
    if (num_seqs < 0) return fail(SC_ERR_INVALID, "%s: num_seqs < 0", fn);
    if (num_seqs > 65535) return fail(SC_ERR_UNSUPPORTED, "%s: more than 65535 sequences", fn);
    if (tokens < 0 || tokens > INT32_MAX)
        return fail(SC_ERR_INVALID, "%s: total_tokens must be in [0, 2^31)", fn);
    if (num_seqs > 0 && (!cu || !ctx))
        return fail(SC_ERR_INVALID, "%s: null cu_seqlens or context_lens", fn);
    return SC_OK;
}

int check_rows(const char* fn, const char* name, const void* x, int64_t stride, int64_t row,
               int32_t dtype) {
    if (!x) return fail(SC_ERR_INVALID, "%s: null %s", fn, name);
    if (stride < row)
        return fail(SC_ERR_INVALID, "%s: %s token stride smaller than its row", fn, name);
    if ((stride * element_bytes(dtype)) % 16)
        return fail(SC_ERR_INVALID, "%s: %s token stride must be a multiple of 16 bytes", fn, name);
    return SC_OK;
}

int check_aligned(const char* fn, const void* const* ptrs, int n) {
    for (int i = 0; i < n; ++i)
        if (!aligned16(ptrs[i]))
            return fail(SC_ERR_INVALID, "%s: pointers must be 16-byte aligned", fn);
    return SC_OK;
}

sc::Paging paging(const int32_t* table, int32_t max_blocks, int32_t block_size, int64_t num_slots) {
    sc::Paging p = {};
    p.table = table;
    p.max_blocks = max_blocks;
    while ((1 << p.shift) < block_size) ++p.shift;
    p.num_pages = (int32_t)(num_slots >> p.shift);
    return p;
}

sc::Batch batch(const int32_t* cu, const int32_t* ctx, int32_t num_seqs, int64_t tokens) {
    sc::Batch b = {};
    b.cu = cu;
    b.ctx = ctx;
    b.num_seqs = num_seqs;
    b.tokens = tokens;
    return b;
}

#define SC_TRY(call)                       \
    do {                                   \
        const int rc_ = (call);            \
        if (rc_ != SC_OK) return rc_;      \
    } while (0)

// ------------------------------------------------------------------------------------------------
// The step over a tree
// ------------------------------------------------------------------------------------------------
int verify_tree(const char* fn, bool mx, const void* k, const void* v, int64_t k_tok_stride,
                int64_t v_tok_stride, const int32_t* cu, int32_t num_seqs, int64_t tokens,
                const int32_t* parents, const float* k_taps, const float* v_taps,
                const float* k_gamma, const float* v_gamma, float eps, const void* k_state,
                const void* v_state, int64_t state_slots, const int32_t* state_idx, void* k_snap,
                void* v_snap, int32_t max_tokens, int64_t* mask, int32_t words,
                const int64_t* slot, void* k_cache, void* v_cache, void* k_scales, void* v_scales,
                int64_t num_slots, int32_t heads, int32_t D, int32_t W, int32_t dtype,
                void* stream) {
    g_err[0] = 0;
    SC_TRY(check_shape(fn, heads, D, dtype));
    if (W < 1 || W > 8) return fail(SC_ERR_UNSUPPORTED, "%s: width %d not in [1, 8]", fn, W);
    if (num_seqs < 0) return fail(SC_ERR_INVALID, "%s: num_seqs < 0", fn);
    if (tokens < 0 || tokens > INT32_MAX)
        return fail(SC_ERR_INVALID, "%s: total_tokens must be in [0, 2^31)", fn);
    if (max_tokens < 1) return fail(SC_ERR_INVALID, "%s: max_tokens < 1", fn);
    if (words < 0) return fail(SC_ERR_INVALID, "%s: mask_words < 0", fn);
    if (state_slots < 0) return fail(SC_ERR_INVALID, "%s: num_state_slots < 0", fn);
    if (num_slots < 0) return fail(SC_ERR_INVALID, "%s: num_slots < 0", fn);
    if (!(eps >= 0.0f) || eps > 3.0e38f)
        return fail(SC_ERR_INVALID, "%s: eps must be finite and >= 0", fn);
    if (!k_taps || !v_taps || !k_gamma || !v_gamma)
        return fail(SC_ERR_INVALID, "%s: null taps or gamma", fn);
    if (W > 1 && state_slots > 0 && (!k_state || !v_state))
        return fail(SC_ERR_INVALID, "%s: null conv state with width %d > 1", fn, W);
    if (num_seqs == 0 || tokens == 0) return SC_OK;  // nothing to compute or snapshot
    if (!cu) return fail(SC_ERR_INVALID, "%s: null cu_seqlens", fn);
    if (!parents) return fail(SC_ERR_INVALID, "%s: null parents", fn);
    if (!slot) return fail(SC_ERR_INVALID, "%s: null slot_mapping", fn);
    if (num_slots > 0 && (!k_cache || !v_cache || (mx && (!k_scales || !v_scales))))
        return fail(SC_ERR_INVALID, "%s: null cache", fn);
    if (W > 1 && (!k_snap || !v_snap))
        return fail(SC_ERR_INVALID, "%s: null snapshot buffer with width %d > 1", fn, W);
    const int64_t row = (int64_t)heads * D;
    SC_TRY(check_rows(fn, "K", k, k_tok_stride, row, dtype));
    SC_TRY(check_rows(fn, "V", v, v_tok_stride, row, dtype));
    const void* ptrs[] = {k, v, k_taps, v_taps, k_gamma, v_gamma, k_state, v_state, k_snap, v_snap,
                          k_cache, v_cache};
    SC_TRY(check_aligned(fn, ptrs, 12));
    sc::StepArgs a = {};
    a.x[0] = k;
    a.x[1] = v;
    a.x_stride[0] = k_tok_stride;
    a.x_stride[1] = v_tok_stride;
    a.taps[0] = k_taps;
    a.taps[1] = v_taps;
    a.gamma[0] = k_gamma;
    a.gamma[1] = v_gamma;
    a.state[0] = W > 1 && state_slots > 0 ? const_cast<void*>(k_state) : nullptr;
    a.state[1] = W > 1 && state_slots > 0 ? const_cast<void*>(v_state) : nullptr;
    a.cache[0] = k_cache;
    a.cache[1] = v_cache;
    a.scales[0] = k_scales;
    a.scales[1] = v_scales;
    a.cu = cu;
    a.state_idx = state_idx;
    a.slot = slot;
    a.tokens = tokens;
    a.num_slots = num_slots;
    a.num_state_slots = state_slots;
    a.num_seqs = num_seqs;
    a.heads = heads;
    a.lanes_per_tensor = (int32_t)(row / (16 / element_bytes(dtype)));
    a.lane_blocks = (int32_t)((2 * (int64_t)a.lanes_per_tensor + 255) / 256);
    a.eps = eps;
    sc::VerifyArgs va = {};
    va.snap[0] = W > 1 ? k_snap : nullptr;
    va.snap[1] = W > 1 ? v_snap : nullptr;
    va.max_tokens = max_tokens;
    sc::TreeArgs ta = {};
    ta.parents = parents;
    ta.mask = words > 0 ? mask : nullptr;
    ta.words = words;
    return launched(fn, sc::launch_verify_tree(a, va, ta, mx, dtype, D, W, (hipStream_t)stream));
}

// ------------------------------------------------------------------------------------------------
// Attention and its weights
// ------------------------------------------------------------------------------------------------
enum Kind { TREE, BLOCKS, SCORES };

// The units' shape, from the query rows of an average sequence, or of one token.
sc::AttnShape unit_shape(Kind kind, int64_t tokens, int32_t num_seqs, int32_t q_heads,
                         int32_t heads, int32_t D, int32_t dtype) {
    const int64_t group = q_heads / heads;
    const int64_t each = kind == TREE && num_seqs > 0 ? (tokens + num_seqs - 1) / num_seqs : 1;
    return sc::attention_shape(kind == TREE, each * group, element_bytes(dtype), D);
}

int64_t part_offset(int32_t num_seqs) { return ((int64_t)num_seqs + 1) * 8 / 256 * 256 + 256; }

// The prefix sums of the sequences' steps (tree), and two parts per worker: rows of D sums, then
// the rows' maxima and sums.
size_t attention_workspace(Kind kind, int64_t tokens, int32_t num_seqs, int32_t q_heads,
                           int32_t heads, int32_t D, int32_t dtype) {
    const sc::AttnShape shape = unit_shape(kind, tokens, num_seqs, q_heads, heads, D, dtype);
    return part_offset(kind == TREE ? num_seqs : 0) +
           (size_t)shape.worker_count(D) * 2 * shape.rows() * (D + 2) * sizeof(float);
}

int attention(const char* fn, Kind kind, bool mx, const void* q, int64_t q_stride,
              const int32_t* cu, const int32_t* ctx, int32_t num_seqs, int64_t tokens,
              const int32_t* table, int32_t max_blocks, int32_t block_size, const int64_t* mask,
              int32_t words, const int32_t* selected, int32_t topk, const void* k, const void* v,
              const void* ks, const void* vs, int64_t num_slots, float scale, void* out,
              float* lse, const float* scores_in, float* scores_out, int64_t capacity, void* ws,
              size_t ws_bytes, int32_t q_heads, int32_t heads, int32_t D, int32_t dtype,
              void* stream) {
    g_err[0] = 0;
    SC_TRY(check_shape(fn, heads, D, dtype));
    SC_TRY(check_queries(fn, q_heads, heads, D));
    SC_TRY(check_paging(fn, table, max_blocks, block_size, num_slots, num_seqs));
    SC_TRY(check_batch(fn, cu, ctx, num_seqs, tokens));
    if (!(scale > -3.0e38f && scale < 3.0e38f))
        return fail(SC_ERR_INVALID, "%s: scale must be finite", fn);
    if (words < 0) return fail(SC_ERR_INVALID, "%s: mask_words < 0", fn);
    if (topk < 0) return fail(SC_ERR_INVALID, "%s: topk < 0", fn);
    if (capacity < 0) return fail(SC_ERR_INVALID, "%s: capacity < 0", fn);
    if (num_seqs == 0 || (kind != SCORES && tokens == 0)) return SC_OK;
    const int64_t row = (int64_t)q_heads * D;
    if (tokens > 0) SC_TRY(check_rows(fn, "q", q, q_stride, row, dtype));
    const bool empty = num_slots == 0 || max_blocks == 0;
    if (!empty && (!k || (kind != SCORES && !v) || (mx && (!ks || (kind != SCORES && !vs)))))
        return fail(SC_ERR_INVALID, "%s: null cache", fn);
    if (kind != SCORES && !out) return fail(SC_ERR_INVALID, "%s: null out", fn);
    if (kind == BLOCKS && topk > 0 && !selected)
        return fail(SC_ERR_INVALID, "%s: null selected", fn);
    if (kind == SCORES) {
        if (tokens > 0 && !lse) return fail(SC_ERR_INVALID, "%s: null lse", fn);
        if (capacity > 0 && !scores_out) return fail(SC_ERR_INVALID, "%s: null scores_out", fn);
        if (capacity == 0 || max_blocks == 0) return SC_OK;
    }
    const void* ptrs[] = {q, k, v, out, ws};
    SC_TRY(check_aligned(fn, ptrs, 5));
    const size_t need = kind == SCORES ? 0
                                       : attention_workspace(kind, tokens, num_seqs, q_heads,
                                                             heads, D, dtype);
    if (need > 0 && (!ws || ws_bytes < need))
        return fail(SC_ERR_INVALID, "%s: workspace of %zu bytes needed, %zu given", fn, need,
                    ws ? ws_bytes : (size_t)0);
    sc::AttnArgs a = {};
    a.b = batch(cu, ctx, num_seqs, tokens);
    a.pg = paging(table, max_blocks, block_size, num_slots);
    a.q = q;
    a.q_stride = q_stride;
    a.cache[0] = k;
    a.cache[1] = v;
    a.scales[0] = ks;
    a.scales[1] = vs;
    a.mask = mask;
    a.words = words;
    a.selected = selected;
    a.topk = topk;
    a.out = out;
    a.lse = lse;
    a.scores_in = scores_in;
    a.scores_out = scores_out;
    a.capacity = capacity;
    a.ws = ws;
    a.part_offset = part_offset(kind == TREE ? num_seqs : 0);
    a.heads = heads;
    a.group = q_heads / heads;
    a.scale = scale;
    const hipStream_t st = (hipStream_t)stream;
    if (kind == SCORES) return launched(fn, sc::launch_cache_scores(a, mx, dtype, D, st));
    const sc::AttnShape shape = unit_shape(kind, tokens, num_seqs, q_heads, heads, D, dtype);
    return launched(fn, shape.waves ? sc::launch_wide_attention(a, mx, D, shape, st)
                                    : sc::launch_attention(a, kind == BLOCKS, mx, dtype, D,
                                                           shape.tiles, st));
}

size_t bad_size(const char* fn, const char* why) {
    fail(SC_ERR_INVALID, "%s: %s", fn, why);
    return SIZE_MAX;
}

int summary(const char* fn, bool mx, const void* k, const void* ks, const int32_t* cu,
            const int32_t* ctx, int32_t num_seqs, const int32_t* table, int32_t max_blocks,
            int32_t block_size, int64_t num_slots, int32_t rebuild, void* sum,
            void* exps, int32_t heads, int32_t D, int32_t dtype, void* stream) {
    g_err[0] = 0;
    SC_TRY(check_shape(fn, heads, D, dtype));
    SC_TRY(check_paging(fn, table, max_blocks, block_size, num_slots, num_seqs));
    SC_TRY(check_batch(fn, cu, ctx, num_seqs, 0));
    if (num_seqs == 0 || max_blocks == 0 || num_slots < block_size) return SC_OK;
    if (!k || (mx && !ks)) return fail(SC_ERR_INVALID, "%s: null cache", fn);
    if (!sum || !exps) return fail(SC_ERR_INVALID, "%s: null summary or exponents", fn);
    const void* ptrs[] = {k, sum};
    SC_TRY(check_aligned(fn, ptrs, 2));
    sc::SummaryArgs a = {};
    a.b = batch(cu, ctx, num_seqs, INT32_MAX);  // only lengths are taken from cu_seqlens
    a.pg = paging(table, max_blocks, block_size, num_slots);
    a.cache = k;
    a.scales = ks;
    a.summary = static_cast<int8_t*>(sum);
    a.exponents = static_cast<uint8_t*>(exps);
    a.heads = heads;
    a.rebuild = rebuild;
    return launched(fn, sc::launch_block_summary(a, mx, dtype, D, (hipStream_t)stream));
}

int64_t key_stride(int32_t max_blocks) { return ((int64_t)max_blocks + 3) / 4 * 4; }

// Rows that can have to move for one head: none unless an entry lies past the budget.
int64_t most_moves(int64_t capacity, int32_t budget) {
    const int64_t past = capacity > budget ? capacity - budget : 0;
    return past < budget ? past : budget;
}

int evict(const char* fn, bool mx, const float* scores, const int32_t* positions,
          const int32_t* lens, const int32_t* seen, int32_t num_seqs, int64_t capacity,
          int32_t budget, int32_t sinks, int32_t recent, const int32_t* table, int32_t max_blocks,
          int32_t block_size, void* k, void* v, void* ks, void* vs, int64_t num_slots,
          float* scores_out, int32_t* positions_out, int32_t* lens_out, void* ws, size_t ws_bytes,
          int32_t heads, int32_t D, int32_t dtype, void* stream) {
    g_err[0] = 0;
    SC_TRY(check_shape(fn, heads, D, dtype));
    SC_TRY(check_paging(fn, table, max_blocks, block_size, num_slots, num_seqs));
    if (num_seqs < 0 || capacity < 0 || budget < 0 || sinks < 0 || recent < 0)
        return fail(SC_ERR_INVALID, "%s: negative size", fn);
    if (num_seqs > 65535 || heads > 65535)
        return fail(SC_ERR_UNSUPPORTED, "%s: more than 65535 sequences or heads", fn);
    if (capacity > INT32_MAX) return fail(SC_ERR_UNSUPPORTED, "%s: capacity must be below 2^31", fn);
    if (num_seqs == 0) return SC_OK;
    if (!lens || !seen || !lens_out)
        return fail(SC_ERR_INVALID, "%s: null lens, seen or lens_out", fn);
    if (capacity > 0 && (!scores || !positions || !scores_out || !positions_out))
        return fail(SC_ERR_INVALID, "%s: null scores or positions", fn);
    if (num_slots > 0 && max_blocks > 0 && (!k || !v || (mx && (!ks || !vs))))
        return fail(SC_ERR_INVALID, "%s: null cache", fn);
    const void* ptrs[] = {k, v, ws};
    SC_TRY(check_aligned(fn, ptrs, 3));
    const int64_t moves = most_moves(capacity, budget);
    const size_t units = (size_t)num_seqs * heads;
    const size_t need = units * (1 + 2 * (size_t)moves) * sizeof(int32_t);
    if (!ws || ws_bytes < need)
        return fail(SC_ERR_INVALID, "%s: workspace of %zu bytes needed, %zu given", fn, need,
                    ws ? ws_bytes : (size_t)0);
    sc::EvictArgs a = {};
    a.pg = paging(table, max_blocks, block_size, num_slots);
    a.scores = scores;
    a.positions = positions;
    a.lens = lens;
    a.seen = seen;
    a.scores_out = scores_out;
    a.positions_out = positions_out;
    a.lens_out = lens_out;
    a.cache[0] = k;
    a.cache[1] = v;
    a.scales[0] = ks;
    a.scales[1] = vs;
    a.count = static_cast<int32_t*>(ws);
    a.dst = a.count + units;
    a.src = a.dst + units * moves;
    a.capacity = capacity;
    a.max_moves = (int32_t)moves;
    a.num_seqs = num_seqs;
    a.heads = heads;
    a.budget = budget;
    a.sinks = sinks;
    a.recent = recent;
    return launched(fn, sc::launch_cache_evict(a, mx, dtype, D, (hipStream_t)stream));
}

}  // namespace

SC_API int shortconv_kv_verify_tree(const void* k, const void* v, int64_t k_tok_stride,
                                    int64_t v_tok_stride, const int32_t* cu_seqlens,
                                    int32_t num_seqs, int64_t total_tokens, const int32_t* parents,
                                    const float* k_taps, const float* v_taps, const float* k_gamma,
                                    const float* v_gamma, float eps, const void* k_state,
                                    const void* v_state, int64_t num_state_slots,
                                    const int32_t* state_idx, void* k_snap, void* v_snap,
                                    int32_t max_tokens, int64_t* mask, int32_t mask_words,
                                    const int64_t* slot_mapping, void* k_cache, void* v_cache,
                                    int64_t num_slots, int32_t num_heads, int32_t head_dim,
                                    int32_t width, int32_t dtype, void* stream) {
    return verify_tree("shortconv_kv_verify_tree", false, k, v, k_tok_stride, v_tok_stride,
                       cu_seqlens, num_seqs, total_tokens, parents, k_taps, v_taps, k_gamma,
                       v_gamma, eps, k_state, v_state, num_state_slots, state_idx, k_snap, v_snap,
                       max_tokens, mask, mask_words, slot_mapping, k_cache, v_cache, nullptr,
                       nullptr, num_slots, num_heads, head_dim, width, dtype, stream);
}

SC_API int shortconv_kv_verify_tree_mxfp8(
    const void* k, const void* v, int64_t k_tok_stride, int64_t v_tok_stride,
    const int32_t* cu_seqlens, int32_t num_seqs, int64_t total_tokens, const int32_t* parents,
    const float* k_taps, const float* v_taps, const float* k_gamma, const float* v_gamma,
    float eps, const void* k_state, const void* v_state, int64_t num_state_slots,
    const int32_t* state_idx, void* k_snap, void* v_snap, int32_t max_tokens, int64_t* mask,
    int32_t mask_words, const int64_t* slot_mapping, void* k_codes, void* v_codes, void* k_scales,
    void* v_scales, int64_t num_slots, int32_t num_heads, int32_t head_dim, int32_t width,
    int32_t dtype, void* stream) {
    return verify_tree("shortconv_kv_verify_tree_mxfp8", true, k, v, k_tok_stride, v_tok_stride,
                       cu_seqlens, num_seqs, total_tokens, parents, k_taps, v_taps, k_gamma,
                       v_gamma, eps, k_state, v_state, num_state_slots, state_idx, k_snap, v_snap,
                       max_tokens, mask, mask_words, slot_mapping, k_codes, v_codes, k_scales,
                       v_scales, num_slots, num_heads, head_dim, width, dtype, stream);
}

SC_API int shortconv_tree_attention(const void* q, int64_t q_tok_stride, const int32_t* cu_seqlens,
                                    const int32_t* context_lens, int32_t num_seqs,
                                    int64_t total_tokens, const int32_t* block_table,
                                    int32_t max_blocks, int32_t block_size, const int64_t* mask,
                                    int32_t mask_words, const void* k_cache, const void* v_cache,
                                    int64_t num_slots, float scale, void* out, float* lse,
                                    void* workspace, size_t workspace_bytes, int32_t num_q_heads,
                                    int32_t num_heads, int32_t head_dim, int32_t dtype,
                                    void* stream) {
    return attention("shortconv_tree_attention", TREE, false, q, q_tok_stride, cu_seqlens,
                     context_lens, num_seqs, total_tokens, block_table, max_blocks, block_size,
                     mask, mask_words, nullptr, 0, k_cache, v_cache, nullptr, nullptr, num_slots,
                     scale, out, lse, nullptr, nullptr, 0, workspace, workspace_bytes, num_q_heads,
                     num_heads, head_dim, dtype, stream);
}

SC_API int shortconv_tree_attention_mxfp8(
    const void* q, int64_t q_tok_stride, const int32_t* cu_seqlens, const int32_t* context_lens,
    int32_t num_seqs, int64_t total_tokens, const int32_t* block_table, int32_t max_blocks,
    int32_t block_size, const int64_t* mask, int32_t mask_words, const void* k_codes,
    const void* v_codes, const void* k_scales, const void* v_scales, int64_t num_slots,
    float scale, void* out, float* lse, void* workspace, size_t workspace_bytes,
    int32_t num_q_heads, int32_t num_heads, int32_t head_dim, int32_t dtype, void* stream) {
    return attention("shortconv_tree_attention_mxfp8", TREE, true, q, q_tok_stride, cu_seqlens,
                     context_lens, num_seqs, total_tokens, block_table, max_blocks, block_size,
                     mask, mask_words, nullptr, 0, k_codes, v_codes, k_scales, v_scales, num_slots,
                     scale, out, lse, nullptr, nullptr, 0, workspace, workspace_bytes, num_q_heads,
                     num_heads, head_dim, dtype, stream);
}

SC_API size_t shortconv_tree_attention_workspace_size(int64_t total_tokens, int32_t num_seqs,
                                                      int32_t num_q_heads, int32_t num_heads,
                                                      int32_t head_dim, int32_t dtype) {
    const char* fn = "shortconv_tree_attention_workspace_size";
    g_err[0] = 0;
    if (check_shape(fn, num_heads, head_dim, dtype) != SC_OK ||
        check_queries(fn, num_q_heads, num_heads, head_dim) != SC_OK)
        return SIZE_MAX;
    if (total_tokens < 0 || total_tokens > INT32_MAX || num_seqs < 0)
        return bad_size(fn, "bad total_tokens or num_seqs");
    return attention_workspace(TREE, total_tokens, num_seqs, num_q_heads, num_heads, head_dim,
                               dtype);
}

SC_API int shortconv_block_summary(const void* k_cache, const int32_t* cu_seqlens,
                                   const int32_t* context_lens, int32_t num_seqs,
                                   const int32_t* block_table, int32_t max_blocks,
                                   int32_t block_size, int64_t num_slots, int32_t rebuild, void* summary_, void* exponents,
                                   int32_t num_heads, int32_t head_dim, int32_t dtype,
                                   void* stream) {
    return summary("shortconv_block_summary", false, k_cache, nullptr, cu_seqlens, context_lens,
                   num_seqs, block_table, max_blocks, block_size, num_slots, rebuild, summary_,
                   exponents, num_heads, head_dim, dtype, stream);
}

SC_API int shortconv_block_summary_mxfp8(const void* k_codes, const void* k_scales,
                                         const int32_t* cu_seqlens, const int32_t* context_lens,
                                         int32_t num_seqs, const int32_t* block_table,
                                         int32_t max_blocks, int32_t block_size,
                                         int64_t num_slots, int32_t rebuild,
                                         void* summary_, void* exponents, int32_t num_heads,
                                         int32_t head_dim, void* stream) {
    return summary("shortconv_block_summary_mxfp8", true, k_codes, k_scales, cu_seqlens,
                   context_lens, num_seqs, block_table, max_blocks, block_size, num_slots, rebuild,
                   summary_, exponents, num_heads, head_dim, SC_DTYPE_BF16, stream);
}

SC_API size_t shortconv_block_select_workspace_size(int64_t total_tokens, int32_t max_blocks,
                                                    int32_t num_heads) {
    const char* fn = "shortconv_block_select_workspace_size";
    g_err[0] = 0;
    if (total_tokens < 0 || total_tokens > INT32_MAX || max_blocks < 0 || num_heads < 1)
        return bad_size(fn, "bad total_tokens, max_blocks or num_heads");
    return (size_t)total_tokens * num_heads * key_stride(max_blocks) * sizeof(uint32_t);
}

SC_API int shortconv_block_select(const void* q, int64_t q_tok_stride, const int32_t* cu_seqlens,
                                  const int32_t* context_lens, int32_t num_seqs,
                                  int64_t total_tokens, const int32_t* block_table,
                                  int32_t max_blocks, int32_t block_size, int64_t num_slots,
                                  const void* summary_, const void* exponents, int32_t sink_blocks,
                                  int32_t recent_blocks, int32_t* selected, int32_t topk,
                                  void* workspace, size_t workspace_bytes, int32_t num_q_heads,
                                  int32_t num_heads, int32_t head_dim, int32_t dtype,
                                  void* stream) {
    const char* fn = "shortconv_block_select";
    g_err[0] = 0;
    SC_TRY(check_shape(fn, num_heads, head_dim, dtype));
    SC_TRY(check_queries(fn, num_q_heads, num_heads, head_dim));
    SC_TRY(check_paging(fn, block_table, max_blocks, block_size, num_slots, num_seqs));
    SC_TRY(check_batch(fn, cu_seqlens, context_lens, num_seqs, total_tokens));
    if (topk < 0 || sink_blocks < 0 || recent_blocks < 0)
        return fail(SC_ERR_INVALID, "%s: negative topk, sink_blocks or recent_blocks", fn);
    // The sum of G * D products of two codes has to fit 32 bits.
    if ((int64_t)num_q_heads / num_heads * head_dim > INT32_MAX / (127 * 127))
        return fail(SC_ERR_UNSUPPORTED, "%s: too many query heads per cache head", fn);
    if (num_seqs == 0 || total_tokens == 0 || topk == 0) return SC_OK;
    SC_TRY(check_rows(fn, "q", q, q_tok_stride, (int64_t)num_q_heads * head_dim, dtype));
    if (!selected) return fail(SC_ERR_INVALID, "%s: null selected", fn);
    if (num_slots >= block_size && max_blocks > 0 && (!summary_ || !exponents))
        return fail(SC_ERR_INVALID, "%s: null summary or exponents", fn);
    const void* ptrs[] = {q, summary_, workspace};
    SC_TRY(check_aligned(fn, ptrs, 3));
    const size_t need =
        (size_t)total_tokens * num_heads * key_stride(max_blocks) * sizeof(uint32_t);
    if (need > 0 && (!workspace || workspace_bytes < need))
        return fail(SC_ERR_INVALID, "%s: workspace of %zu bytes needed, %zu given", fn, need,
                    workspace ? workspace_bytes : (size_t)0);
    sc::SelectArgs a = {};
    a.b = batch(cu_seqlens, context_lens, num_seqs, total_tokens);
    a.pg = paging(block_table, max_blocks, block_size, num_slots);
    a.q = q;
    a.q_stride = q_tok_stride;
    a.summary = static_cast<const int8_t*>(summary_);
    a.exponents = static_cast<const uint8_t*>(exponents);
    a.selected = selected;
    a.keys = static_cast<uint32_t*>(workspace);
    a.key_stride = key_stride(max_blocks);
    a.topk = topk;
    a.sinks = sink_blocks;
    a.recents = recent_blocks;
    a.heads = num_heads;
    a.group = num_q_heads / num_heads;
    return launched(fn, sc::launch_block_select(a, dtype, head_dim, (hipStream_t)stream));
}

SC_API int shortconv_block_attention(const void* q, int64_t q_tok_stride,
                                     const int32_t* cu_seqlens, const int32_t* context_lens,
                                     int32_t num_seqs, int64_t total_tokens,
                                     const int32_t* block_table, int32_t max_blocks,
                                     int32_t block_size, const int32_t* selected, int32_t topk,
                                     const void* k_cache, const void* v_cache, int64_t num_slots,
                                     float scale, void* out, float* lse, void* workspace,
                                     size_t workspace_bytes, int32_t num_q_heads,
                                     int32_t num_heads, int32_t head_dim, int32_t dtype,
                                     void* stream) {
    return attention("shortconv_block_attention", BLOCKS, false, q, q_tok_stride, cu_seqlens,
                     context_lens, num_seqs, total_tokens, block_table, max_blocks, block_size,
                     nullptr, 0, selected, topk, k_cache, v_cache, nullptr, nullptr, num_slots,
                     scale, out, lse, nullptr, nullptr, 0, workspace, workspace_bytes, num_q_heads,
                     num_heads, head_dim, dtype, stream);
}

SC_API int shortconv_block_attention_mxfp8(
    const void* q, int64_t q_tok_stride, const int32_t* cu_seqlens, const int32_t* context_lens,
    int32_t num_seqs, int64_t total_tokens, const int32_t* block_table, int32_t max_blocks,
    int32_t block_size, const int32_t* selected, int32_t topk, const void* k_codes,
    const void* v_codes, const void* k_scales, const void* v_scales, int64_t num_slots,
    float scale, void* out, float* lse, void* workspace, size_t workspace_bytes,
    int32_t num_q_heads, int32_t num_heads, int32_t head_dim, int32_t dtype, void* stream) {
    return attention("shortconv_block_attention_mxfp8", BLOCKS, true, q, q_tok_stride, cu_seqlens,
                     context_lens, num_seqs, total_tokens, block_table, max_blocks, block_size,
                     nullptr, 0, selected, topk, k_codes, v_codes, k_scales, v_scales, num_slots,
                     scale, out, lse, nullptr, nullptr, 0, workspace, workspace_bytes, num_q_heads,
                     num_heads, head_dim, dtype, stream);
}

SC_API size_t shortconv_block_attention_workspace_size(int64_t total_tokens, int32_t topk,
                                                       int32_t block_size, int32_t num_q_heads,
                                                       int32_t num_heads, int32_t head_dim,
                                                       int32_t dtype) {
    const char* fn = "shortconv_block_attention_workspace_size";
    g_err[0] = 0;
    if (check_shape(fn, num_heads, head_dim, dtype) != SC_OK ||
        check_queries(fn, num_q_heads, num_heads, head_dim) != SC_OK)
        return SIZE_MAX;
    if (total_tokens < 0 || total_tokens > INT32_MAX || topk < 0 || block_size < 1)
        return bad_size(fn, "bad total_tokens, topk or block_size");
    return attention_workspace(BLOCKS, total_tokens, 0, num_q_heads, num_heads, head_dim, dtype);
}

SC_API int shortconv_cache_scores(const void* q, int64_t q_tok_stride, const float* lse,
                                  const int32_t* cu_seqlens, const int32_t* context_lens,
                                  int32_t num_seqs, int64_t total_tokens,
                                  const int32_t* block_table, int32_t max_blocks,
                                  int32_t block_size, const int64_t* mask, int32_t mask_words,
                                  const void* k_cache, int64_t num_slots, float scale,
                                  const float* scores, float* scores_out, int64_t capacity,
                                  int32_t num_q_heads, int32_t num_heads, int32_t head_dim,
                                  int32_t dtype, void* stream) {
    return attention("shortconv_cache_scores", SCORES, false, q, q_tok_stride, cu_seqlens,
                     context_lens, num_seqs, total_tokens, block_table, max_blocks, block_size,
                     mask, mask_words, nullptr, 0, k_cache, nullptr, nullptr, nullptr, num_slots,
                     scale, nullptr, const_cast<float*>(lse), scores, scores_out, capacity,
                     nullptr, 0, num_q_heads, num_heads, head_dim, dtype, stream);
}

SC_API int shortconv_cache_scores_mxfp8(const void* q, int64_t q_tok_stride, const float* lse,
                                        const int32_t* cu_seqlens, const int32_t* context_lens,
                                        int32_t num_seqs, int64_t total_tokens,
                                        const int32_t* block_table, int32_t max_blocks,
                                        int32_t block_size, const int64_t* mask,
                                        int32_t mask_words, const void* k_codes,
                                        const void* k_scales, int64_t num_slots, float scale,
                                        const float* scores, float* scores_out, int64_t capacity,
                                        int32_t num_q_heads, int32_t num_heads, int32_t head_dim,
                                        int32_t dtype, void* stream) {
    return attention("shortconv_cache_scores_mxfp8", SCORES, true, q, q_tok_stride, cu_seqlens,
                     context_lens, num_seqs, total_tokens, block_table, max_blocks, block_size,
                     mask, mask_words, nullptr, 0, k_codes, nullptr, k_scales, nullptr, num_slots,
                     scale, nullptr, const_cast<float*>(lse), scores, scores_out, capacity,
                     nullptr, 0, num_q_heads, num_heads, head_dim, dtype, stream);
}

SC_API size_t shortconv_cache_evict_workspace_size(int32_t num_seqs, int64_t capacity,
                                                   int32_t budget, int32_t num_heads) {
    const char* fn = "shortconv_cache_evict_workspace_size";
    g_err[0] = 0;
    if (num_seqs < 0 || capacity < 0 || capacity > INT32_MAX || budget < 0 || num_heads < 1)
        return bad_size(fn, "bad num_seqs, capacity, budget or num_heads");
    return (size_t)num_seqs * num_heads * (1 + 2 * (size_t)most_moves(capacity, budget)) *
           sizeof(int32_t);
}

SC_API int shortconv_cache_evict(const float* scores, const int32_t* positions,
                                 const int32_t* lens, const int32_t* seen, int32_t num_seqs,
                                 int64_t capacity, int32_t budget, int32_t sinks, int32_t recent,
                                 const int32_t* block_table, int32_t max_blocks,
                                 int32_t block_size, void* k_cache, void* v_cache,
                                 int64_t num_slots, float* scores_out, int32_t* positions_out,
                                 int32_t* lens_out, void* workspace, size_t workspace_bytes,
                                 int32_t num_heads, int32_t head_dim, int32_t dtype,
                                 void* stream) {
    return evict("shortconv_cache_evict", false, scores, positions, lens, seen, num_seqs, capacity,
                 budget, sinks, recent, block_table, max_blocks, block_size, k_cache, v_cache,
                 nullptr, nullptr, num_slots, scores_out, positions_out, lens_out, workspace,
                 workspace_bytes, num_heads, head_dim, dtype, stream);
}

SC_API int shortconv_cache_evict_mxfp8(const float* scores, const int32_t* positions,
                                       const int32_t* lens, const int32_t* seen, int32_t num_seqs,
                                       int64_t capacity, int32_t budget, int32_t sinks,
                                       int32_t recent, const int32_t* block_table,
                                       int32_t max_blocks, int32_t block_size, void* k_codes,
                                       void* v_codes, void* k_scales, void* v_scales,
                                       int64_t num_slots, float* scores_out,
                                       int32_t* positions_out, int32_t* lens_out, void* workspace,
                                       size_t workspace_bytes, int32_t num_heads,
                                       int32_t head_dim, void* stream) {
    return evict("shortconv_cache_evict_mxfp8", true, scores, positions, lens, seen, num_seqs,
                 capacity, budget, sinks, recent, block_table, max_blocks, block_size, k_codes,
                 v_codes, k_scales, v_scales, num_slots, scores_out, positions_out, lens_out,
                 workspace, workspace_bytes, num_heads, head_dim, SC_DTYPE_BF16, stream);
}

SC_API const char* shortconv_cache_last_error(void) { return g_err; }

SC_API int shortconv_cache_abi_version(void) { return SHORTCONV_CACHE_ABI_VERSION; }
