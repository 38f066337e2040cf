// Internal interface between the C-ABI layer of the cache operators (cache_abi.hip) and their
// kernels (tree_verify.hip, cache_attention.hip, cache_blocks.hip, cache_evict.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "cache_attention.h"
#include "shortconv_internal.h"

namespace sc {

// Page tables: position p of sequence s is cache row (table[s][p >> shift] << shift) + the low
// bits of p. A page id outside [0, num_pages) holds no keys.
struct Paging {
    const int32_t* table;  // [num_seqs][max_blocks]
    int32_t max_blocks;
    int32_t shift;         // log2(block_size)
    int32_t num_pages;     // num_slots >> shift
};

// A packed batch of new tokens behind cached contexts.
struct Batch {
    const int32_t* cu;   // int32 [num_seqs + 1]
    const int32_t* ctx;  // int32 [num_seqs]
    int64_t tokens;
    int32_t num_seqs;
};

// The step over a tree of drafted tokens: StepArgs and VerifyArgs of the chain, the parents, and
// the ancestor mask to write.
struct TreeArgs {
    const int32_t* parents;  // int32 [tokens], index within the sequence
    int64_t* mask;           // [tokens][words] or null
    int32_t words;
};

// Attention over the cache, and the sums of its weights.
struct AttnArgs {
    Batch b;
    Paging pg;
    const void* q;            // [tokens][heads * group][D], token stride q_stride elements
    int64_t q_stride;
    const void* cache[2];     // K, V rows (or codes)
    const void* scales[2];    // MXFP8 scales
    const int64_t* mask;      // [tokens][words] or null (causal)
    const int32_t* selected;  // block attention: [tokens][heads][topk]
    void* out;                // [tokens][heads * group][D]
    float* lse;               // [tokens][heads * group]: out, or null (in, for the scores)
    const float* scores_in;   // [num_seqs][heads][capacity] or null
    float* scores_out;
    int64_t capacity;
    void* ws;                 // prefix sums of the sequences' steps, then the parts of the units
    int64_t part_offset;      // bytes before the parts
    int32_t words;
    int32_t topk;
    int32_t heads;            // cache heads
    int32_t group;            // query heads per cache head
    float scale;
};

struct SummaryArgs {
    Batch b;
    Paging pg;
    const void* cache;
    const void* scales;
    int8_t* summary;     // [num_pages][heads][2][D]
    uint8_t* exponents;  // [num_pages][heads]
    int32_t heads;
    int32_t rebuild;
};

struct SelectArgs {
    Batch b;
    Paging pg;
    const void* q;
    int64_t q_stride;
    const int8_t* summary;
    const uint8_t* exponents;
    int32_t* selected;  // [tokens][heads][topk]
    uint32_t* keys;     // workspace [tokens][heads][key_stride]
    int64_t key_stride; // max_blocks, padded to whole groups of 4
    int32_t topk;
    int32_t sinks;
    int32_t recents;
    int32_t heads;
    int32_t group;
};

struct EvictArgs {
    Paging pg;
    const float* scores;       // [num_seqs][heads][capacity]
    const int32_t* positions;
    const int32_t* lens;       // [num_seqs]
    const int32_t* seen;
    float* scores_out;
    int32_t* positions_out;
    int32_t* lens_out;
    void* cache[2];
    void* scales[2];
    int32_t* count;   // workspace [num_seqs][heads]: rows to move
    int32_t* dst;     // workspace [num_seqs][heads][max_moves]
    int32_t* src;
    int64_t capacity;
    int32_t max_moves;
    int32_t num_seqs;
    int32_t heads;
    int32_t budget;
    int32_t sinks;
    int32_t recent;
};

hipError_t launch_verify_tree(const StepArgs& a, const VerifyArgs& va, const TreeArgs& ta,
                              bool mx, int dtype, int D, int W, hipStream_t stream);
hipError_t launch_attention(const AttnArgs& a, bool selected, bool mx, int dtype, int D,
                            int row_tiles, hipStream_t stream);
hipError_t launch_wide_attention(const AttnArgs& a, bool mx, int D, AttnShape shape,
                                 hipStream_t stream);
hipError_t launch_cache_scores(const AttnArgs& a, bool mx, int dtype, int D, hipStream_t stream);
hipError_t launch_block_summary(const SummaryArgs& a, bool mx, int dtype, int D,
                                hipStream_t stream);
hipError_t launch_block_select(const SelectArgs& a, int dtype, int D, hipStream_t stream);
hipError_t launch_cache_evict(const EvictArgs& a, bool mx, int dtype, int D, hipStream_t stream);

}  // namespace sc
