/*
 * shortconv_cache.h -- C ABI of the operators that read and tend the paged KV cache which the
 * fused ShortConv K/V step (shortconv.h) writes, for AMD Instinct MI355X (gfx950):
 *
 *   shortconv_kv_verify_tree    the step for a tree of drafted tokens
 *   shortconv_tree_attention    attention of drafted (or single new) tokens over the cache
 *   shortconv_block_summary     per page and head an 8-bit bounding box of its keys
 *   shortconv_block_select      the pages worth reading, chosen per query by that box
 *   shortconv_block_attention   attention over the selected pages
 *   shortconv_cache_scores      attention weight each cached key received, accumulated
 *   shortconv_cache_evict       the cache cut down to a budget of entries per sequence and head
 *
 * The `_mxfp8` form of each reads (or writes) MXFP8 cache rows as laid out in shortconv.h.
 *
 * Conventions beyond those of shortconv.h (dtype, rows, ownership, streams, return values, no
 * allocation, arguments checked on the host before anything is launched):
 *  - Paging. Position p of sequence s lives in cache row
 *      block_table[s][p / block_size] * block_size + p % block_size,
 *    block_table int32 [num_seqs][max_blocks] contiguous, block_size a power of two in
 *    [1, 65536], max_blocks * block_size < 2^31, num_slots < 2^31. A page whose rows are not all
 *    inside [0, num_slots) (e.g. a table entry of -1) holds no keys: it is never read or written,
 *    and its positions count as masked.
 *  - A batch of new tokens is packed as in shortconv_kv_prefill: cu_seqlens int32 [num_seqs+1],
 *    sequence s owns tokens [cu_seqlens[s], cu_seqlens[s+1]). context_lens int32 [num_seqs]: the
 *    keys cached before those tokens. The rows of the new tokens are in the cache already, token i
 *    of sequence s at position context_lens[s] + i. Positions at or past max_blocks * block_size
 *    do not exist. Tokens at or behind cu_seqlens[num_seqs] belong to no sequence and every output
 *    row of theirs is left as it was.
 *  - Queries q [total_tokens][num_q_heads][D], token stride in elements; num_q_heads is a multiple
 *    of num_heads (the cache's), and query head j reads cache head j / (num_q_heads/num_heads).
 *  - mask: int64 [total_tokens][mask_words] or NULL. Bit j % 64 of word j / 64 in token i's row
 *    says that i may look at new token j of its own sequence; new tokens at or past 64 *
 *    mask_words are not looked at. NULL: token i looks at new tokens 0..i. Cached keys are always
 *    looked at.
 *  - A query row that nothing is left for gives zeros, and -inf as its log-sum-exp. Keys and
 *    values that a row does not look at never change it, whatever they hold (NaN, infinities).
 *  - Logits are scale * (q . k) and statistics are fp32. With bf16 queries the softmax weights are
 *    rounded to bf16 for the product with V; with fp32 queries nothing is rounded.
 *  - Workspaces are device memory, 16-byte aligned, of at least the bytes that the operator's
 *    *_workspace_size gives; contents on entry do not matter. Calls that may overlap must not
 *    share one (this includes replays of two captured graphs).
 */
#ifndef SHORTCONV_CACHE_H
#define SHORTCONV_CACHE_H

#include "shortconv.h"

#ifdef __cplusplus
extern "C" {
#endif

#define SHORTCONV_CACHE_ABI_VERSION 1

/*
 * shortconv_kv_verify_tree: shortconv_kv_verify for candidates that form a tree. The window of a
 * token is the token and its W-1 nearest ancestors; where the path to the root is shorter, the
 * sequence's conv state supplies the older rows (newest first). The state pools are only read.
 *  parents    int32 [total_tokens]: index, within its sequence, of the token each one follows. It
 *             must be less than the token's own index; any other value makes the token a root (it
 *             follows the sequence's last committed token).
 *  k/v_snap   as for shortconv_kv_verify: snapshot (s, i) is the conv state after the path from
 *             the root to token i. shortconv_state_commit with accepted[s] = i + 1 installs it.
 *  mask       int64 [total_tokens][mask_words] out, or NULL: the ancestors of each token and
 *             itself, as shortconv_tree_attention takes them (bits past 64 * mask_words dropped).
 * Other arguments and results are those of shortconv_kv_verify; with parents[i] = i - 1 the cache
 * rows and the snapshots are the same bit for bit.
 */
int shortconv_kv_verify_tree(const void* k, const void* v, int64_t k_tok_stride,
                             int64_t v_tok_stride, const int32_t* cu_seqlens, int32_t num_seqs,
                             int64_t total_tokens, const int32_t* parents, const float* k_taps,
                             const float* v_taps, const float* k_gamma, const float* v_gamma,
                             float eps, const void* k_state, const void* v_state,
                             int64_t num_state_slots, const int32_t* state_idx, void* k_snap,
                             void* v_snap, int32_t max_tokens, int64_t* mask, int32_t mask_words,
                             const int64_t* slot_mapping, void* k_cache, void* v_cache,
                             int64_t num_slots, int32_t num_heads, int32_t head_dim,
                             int32_t width, int32_t dtype, void* stream);

int shortconv_kv_verify_tree_mxfp8(
    const void* k, const void* v, int64_t k_tok_stride, int64_t v_tok_stride,
    const int32_t* cu_seqlens, int32_t num_seqs, int64_t total_tokens, const int32_t* parents,
    const float* k_taps, const float* v_taps, const float* k_gamma, const float* v_gamma,
    float eps, const void* k_state, const void* v_state, int64_t num_state_slots,
    const int32_t* state_idx, void* k_snap, void* v_snap, int32_t max_tokens, int64_t* mask,
    int32_t mask_words, const int64_t* slot_mapping, void* k_codes, void* v_codes, void* k_scales,
    void* v_scales, int64_t num_slots, int32_t num_heads, int32_t head_dim, int32_t width,
    int32_t dtype, void* stream);

/*
 * shortconv_tree_attention: out[t] = softmax over the keys that token t looks at, times V.
 *  q, out   [total_tokens][num_q_heads][D] of type `dtype`; out contiguous. With plain caches
 *           `dtype` is the caches' type too.
 *  lse      fp32 [total_tokens][num_q_heads] or NULL: natural log of the sum of exp(logit).
 * One token per sequence and no mask is plain decode.
 */
int shortconv_tree_attention(const void* q, int64_t q_tok_stride, const int32_t* cu_seqlens,
                             const int32_t* context_lens, int32_t num_seqs, int64_t total_tokens,
                             const int32_t* block_table, int32_t max_blocks, int32_t block_size,
                             const int64_t* mask, int32_t mask_words, const void* k_cache,
                             const void* v_cache, int64_t num_slots, float scale, void* out,
                             float* lse, void* workspace, size_t workspace_bytes,
                             int32_t num_q_heads, int32_t num_heads, int32_t head_dim,
                             int32_t dtype, void* stream);

int shortconv_tree_attention_mxfp8(
    const void* q, int64_t q_tok_stride, const int32_t* cu_seqlens, const int32_t* context_lens,
    int32_t num_seqs, int64_t total_tokens, const int32_t* block_table, int32_t max_blocks,
    int32_t block_size, const int64_t* mask, int32_t mask_words, const void* k_codes,
    const void* v_codes, const void* k_scales, const void* v_scales, int64_t num_slots,
    float scale, void* out, float* lse, void* workspace, size_t workspace_bytes,
    int32_t num_q_heads, int32_t num_heads, int32_t head_dim, int32_t dtype, void* stream);

/* Bytes of workspace for these sizes (host only); SIZE_MAX when they are invalid. */
size_t shortconv_tree_attention_workspace_size(int64_t total_tokens, int32_t num_seqs,
                                               int32_t num_q_heads, int32_t num_heads,
                                               int32_t head_dim, int32_t dtype);

/*
 * shortconv_block_summary: for each page of each sequence and each head, the minimum and the
 * maximum of its keys in every channel, over the positions below context_lens[s] + T_s.
 *  summary    int8 [num_slots / block_size][num_heads][2][D]: row 0 the minima, row 1 the maxima,
 *             as codes; indexed by the page id that block_table holds.
 *  exponents  uint8 [num_slots / block_size][num_heads]: one power of two per page and head. With
 *             m the largest magnitude of the page's minima and maxima, E = floor(log2 m) - 6,
 *             at least -127, is stored as E + 127, and a code is its value * 2^-E rounded to
 *             nearest even, within +-127. (-127 and codes of 0 when every value is 0.)
 *  rebuild    0: only the pages that the new tokens touch, i.e. those from
 *             context_lens[s] / block_size on. Otherwise every page of every sequence.
 * A NaN key element is passed over; a channel with nothing else counts as 0. Pages of no sequence
 * keep what they held. `dtype` is the cache's type; the `_mxfp8` form takes none.
 */
int shortconv_block_summary(const void* k_cache, const int32_t* cu_seqlens,
                            const int32_t* context_lens, int32_t num_seqs,
                            const int32_t* block_table, int32_t max_blocks, int32_t block_size,
                            int64_t num_slots, int32_t rebuild, void* summary, void* exponents,
                            int32_t num_heads, int32_t head_dim, int32_t dtype, void* stream);

int shortconv_block_summary_mxfp8(const void* k_codes, const void* k_scales,
                                  const int32_t* cu_seqlens, const int32_t* context_lens,
                                  int32_t num_seqs, const int32_t* block_table,
                                  int32_t max_blocks, int32_t block_size, int64_t num_slots,
                                  int32_t rebuild, void* summary, void* exponents, int32_t num_heads,
                                  int32_t head_dim, void* stream);

/*
 * shortconv_block_select: the pages that each new token reads, one choice per token and cache head
 * (its query heads read together). Token i of sequence s has the pages 0..P-1 with
 * P = (context_lens[s] + i) / block_size + 1, at most max_blocks.
 *  Score of page b: the query heads' values, divided by one power of two so that the largest
 *  magnitude of the token's heads lies in [64, 128) and rounded to nearest even within +-127, are
 *  codes c; I_b = sum over heads and channels of max(c * min_b, c * max_b), a whole number; the
 *  score is float(I_b) * 2^E_b (I_b rounded once to fp32). Two devices, or a CPU, agree on it bit
 *  for bit. A NaN element of q counts as 0.
 *  Order: the first sink_blocks and the last recent_blocks of the P pages, ascending, then the
 *  others by score, equal ones by the lower page. Pages outside the pool are never chosen.
 *  selected   int32 [total_tokens][num_heads][topk] out: the first topk pages of that order as
 *             indexes into the sequence's block_table row, ascending, -1 behind them.
 */
int shortconv_block_select(const void* q, int64_t q_tok_stride, const int32_t* cu_seqlens,
                           const int32_t* context_lens, int32_t num_seqs, int64_t total_tokens,
                           const int32_t* block_table, int32_t max_blocks, int32_t block_size,
                           int64_t num_slots, const void* summary, const void* exponents,
                           int32_t sink_blocks, int32_t recent_blocks, int32_t* selected,
                           int32_t topk, void* workspace, size_t workspace_bytes,
                           int32_t num_q_heads, int32_t num_heads, int32_t head_dim,
                           int32_t dtype, void* stream);

size_t shortconv_block_select_workspace_size(int64_t total_tokens, int32_t max_blocks,
                                             int32_t num_heads);

/*
 * shortconv_block_attention: attention of each new token over the keys of its selected pages at
 * positions up to its own (token i of sequence s: context_lens[s] + i). Entries of `selected`
 * outside the token's pages are passed over; one given twice counts twice. Otherwise as
 * shortconv_tree_attention.
 */
int shortconv_block_attention(const void* q, int64_t q_tok_stride, const int32_t* cu_seqlens,
                              const int32_t* context_lens, int32_t num_seqs, int64_t total_tokens,
                              const int32_t* block_table, int32_t max_blocks, int32_t block_size,
                              const int32_t* selected, int32_t topk, const void* k_cache,
                              const void* v_cache, int64_t num_slots, float scale, void* out,
                              float* lse, void* workspace, size_t workspace_bytes,
                              int32_t num_q_heads, int32_t num_heads, int32_t head_dim,
                              int32_t dtype, void* stream);

int shortconv_block_attention_mxfp8(
    const void* q, int64_t q_tok_stride, const int32_t* cu_seqlens, const int32_t* context_lens,
    int32_t num_seqs, int64_t total_tokens, const int32_t* block_table, int32_t max_blocks,
    int32_t block_size, const int32_t* selected, int32_t topk, const void* k_codes,
    const void* v_codes, const void* k_scales, const void* v_scales, int64_t num_slots,
    float scale, void* out, float* lse, void* workspace, size_t workspace_bytes,
    int32_t num_q_heads, int32_t num_heads, int32_t head_dim, int32_t dtype, void* stream);

size_t shortconv_block_attention_workspace_size(int64_t total_tokens, int32_t topk,
                                                int32_t block_size, int32_t num_q_heads,
                                                int32_t num_heads, int32_t head_dim,
                                                int32_t dtype);

/*
 * shortconv_cache_scores: the attention weight that each key received from a batch of queries,
 * summed over the queries and over the query heads of its cache head:
 *   scores_out[s][h][p] = scores[s][h][p] (0 for p >= context_lens[s], or when scores is NULL)
 *                         + sum of exp(scale * (q . k_p) - lse) over the rows that look at p
 *  lse         fp32 [total_tokens][num_q_heads], as the attention returned it; rows of -inf add
 *              nothing.
 *  scores      fp32 [num_seqs][num_heads][capacity] or NULL;  scores_out the same shape, may be
 *              the same memory. Written for p < min(context_lens[s] + T_s, capacity); other
 *              entries are left. A masked position's key adds nothing to it.
 * The sums are fp32 in a fixed order (deterministic).
 */
int shortconv_cache_scores(const void* q, int64_t q_tok_stride, const float* lse,
                           const int32_t* cu_seqlens, const int32_t* context_lens,
                           int32_t num_seqs, int64_t total_tokens, const int32_t* block_table,
                           int32_t max_blocks, int32_t block_size, const int64_t* mask,
                           int32_t mask_words, const void* k_cache, int64_t num_slots, float scale,
                           const float* scores, float* scores_out, int64_t capacity,
                           int32_t num_q_heads, int32_t num_heads, int32_t head_dim,
                           int32_t dtype, void* stream);

int shortconv_cache_scores_mxfp8(const void* q, int64_t q_tok_stride, const float* lse,
                                 const int32_t* cu_seqlens, const int32_t* context_lens,
                                 int32_t num_seqs, int64_t total_tokens,
                                 const int32_t* block_table, int32_t max_blocks,
                                 int32_t block_size, const int64_t* mask, int32_t mask_words,
                                 const void* k_codes, const void* k_scales, int64_t num_slots,
                                 float scale, const float* scores, float* scores_out,
                                 int64_t capacity, int32_t num_q_heads, int32_t num_heads,
                                 int32_t head_dim, int32_t dtype, void* stream);

/*
 * shortconv_cache_evict: keeps at most `budget` entries per sequence and head. Entry j of head h
 * of sequence s is that head's K and V at cache position j; heads keep different entries.
 *  lens        int32 [num_seqs]: entries now; n = lens[s], at least 0 and at most capacity and
 *              max_blocks * block_size.
 *  scores      fp32 [num_seqs][num_heads][capacity];  a NaN ranks below every number.
 *  positions   int32, same shape: the token position each entry came from (0, 1, 2, .. before the
 *              first eviction).   seen  int32 [num_seqs]: tokens the sequence has had so far.
 *  Order: entries whose position is below `sinks` or at or past seen[s] - recent, by ascending
 *  index, then the others by score from the largest, equal ones by the lower index. The first `budget` are kept. Entries
 *  j < budget that are not kept are holes; the i-th hole, ascending, takes K, V, score and
 *  position of the i-th kept entry at or past `budget`, ascending. Every other kept entry stays
 *  where it is. lens_out[s] = min(n, budget).
 *  scores_out, positions_out: written for j < lens_out[s]. Each output may be the memory of its
 *  input. The conv state is not touched. Pages of one sequence must not be shared with another; an
 *  entry in a page outside the pool keeps its place in the order, and nothing is copied from or to
 *  it.
 */
int shortconv_cache_evict(const float* scores, const int32_t* positions, const int32_t* lens,
                          const int32_t* seen, int32_t num_seqs, int64_t capacity, int32_t budget,
                          int32_t sinks, int32_t recent, const int32_t* block_table,
                          int32_t max_blocks, int32_t block_size, void* k_cache, void* v_cache,
                          int64_t num_slots, float* scores_out, int32_t* positions_out,
                          int32_t* lens_out, void* workspace, size_t workspace_bytes,
                          int32_t num_heads, int32_t head_dim, int32_t dtype, void* stream);

int shortconv_cache_evict_mxfp8(const float* scores, const int32_t* positions,
                                const int32_t* lens, const int32_t* seen, int32_t num_seqs,
                                int64_t capacity, int32_t budget, int32_t sinks, int32_t recent,
                                const int32_t* block_table, int32_t max_blocks,
                                int32_t block_size, void* k_codes, void* v_codes, void* k_scales,
                                void* v_scales, int64_t num_slots, float* scores_out,
                                int32_t* positions_out, int32_t* lens_out, void* workspace,
                                size_t workspace_bytes, int32_t num_heads, int32_t head_dim,
                                void* stream);

size_t shortconv_cache_evict_workspace_size(int32_t num_seqs, int64_t capacity, int32_t budget,
                                            int32_t num_heads);

/* Message for the last non-zero return on the calling thread ("" if none). */
const char* shortconv_cache_last_error(void);

/* SHORTCONV_CACHE_ABI_VERSION of the built library. */
int shortconv_cache_abi_version(void);

#ifdef __cplusplus
}
#endif

#endif /* SHORTCONV_CACHE_H */
