// Page summaries and the selection of pages by them (shortconv_block_summary,
// shortconv_block_select). Everything the selection compares is a whole number or a whole number
// scaled by a power of two, so the choice does not depend on the order of any sum.
#include "cache_device.h"

namespace sc {
namespace {

constexpr int kBlock = 256;

// One lane's VEC channels of a cache row as fp32: 16 bytes of fp32 or bf16, or 8 MXFP8 codes.
template <class E, bool MX>
struct KeyRow {
    static constexpr int VEC = MX ? 8 : E::VEC;
    __device__ static inline void load(const void* cache, const void* scales, int64_t row_elems,
                                       int32_t slot, int32_t off, float (&f)[VEC]) {
        if constexpr (!MX) {
            const uint4 r = ld16(cache, (int64_t)slot * row_elems + off, E::BYTES);
            E::widen(r, f);
        } else {
            const int64_t at = (int64_t)slot * row_elems + off;
            const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const char*>(cache) + at);
            const uint8_t e = static_cast<const uint8_t*>(scales)[at >> 5];
            const float sc = __uint_as_float(e ? (uint32_t)e << 23 : 0x00400000u);  // 2^(e - 127)
            typedef float f32x2 __attribute__((ext_vector_type(2)));
            const f32x2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w.x, sc, false);
            const f32x2 b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w.x, sc, true);
            const f32x2 c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w.y, sc, false);
            const f32x2 d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w.y, sc, true);
            f[0] = a[0]; f[1] = a[1]; f[2] = b[0]; f[3] = b[1];
            f[4] = c[0]; f[5] = c[1]; f[6] = d[0]; f[7] = d[1];
        }
    }
};

// Bound by the bytes of K: 65000 MXFP8 keys of 8 heads of 128 in 20 us (3.3 TB/s).
// Workgroup: one 64-lane column slice of a page (blockIdx.x strides over the pages of sequence
// blockIdx.y); its 4 waves take every fourth row and meet in LDS.
template <class E, int D, bool MX>
__global__ void __launch_bounds__(kBlock) summary_kernel(SummaryArgs a) {
    constexpr int VEC = KeyRow<E, MX>::VEC;
    constexpr int LPH = D / VEC;
    const int s = blockIdx.y;
    const SeqInfo q = seq_info(a.b, a.pg, s);
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int32_t col = (blockIdx.z * 64 + lane) * VEC;
    const int64_t row_elems = (int64_t)a.heads * D;
    const bool active = col < row_elems;
    const int bs = 1 << a.pg.shift;
    __shared__ float part[4][64][2 * VEC + 1];
    const int32_t first = a.rebuild ? 0 : q.ctx >> a.pg.shift;
    for (int32_t pb = first + blockIdx.x; ((int64_t)pb << a.pg.shift) < q.keys; pb += gridDim.x) {
        const int32_t slot = slot_of(a.pg, s, pb << a.pg.shift);
        if (slot < 0) continue;
        const int rows = min(bs, q.keys - (pb << a.pg.shift));
        float lo[VEC], hi[VEC];
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            lo[v] = __builtin_inff();
            hi[v] = -__builtin_inff();
        }
        if (active) {
            for (int r = wave; r < rows; r += 4) {
                float f[VEC];
                KeyRow<E, MX>::load(a.cache, a.scales, row_elems, slot + r, col, f);
#pragma unroll
                for (int v = 0; v < VEC; ++v) {  // comparisons pass over a NaN
                    lo[v] = f[v] < lo[v] ? f[v] : lo[v];
                    hi[v] = f[v] > hi[v] ? f[v] : hi[v];
                }
            }
        }
        __syncthreads();
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            part[wave][lane][v] = lo[v];
            part[wave][lane][VEC + v] = hi[v];
        }
        __syncthreads();
        if (wave == 0) {
            uint32_t top = 0;
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
#pragma unroll
                for (int w = 1; w < 4; ++w) {
                    const float l = part[w][lane][v], h = part[w][lane][VEC + v];
                    lo[v] = l < lo[v] ? l : lo[v];
                    hi[v] = h > hi[v] ? h : hi[v];
                }
                if (lo[v] > hi[v]) lo[v] = hi[v] = 0.0f;  // nothing but NaN
                top = max(top, __float_as_uint(__builtin_fabsf(lo[v])));
                top = max(top, __float_as_uint(__builtin_fabsf(hi[v])));
            }
            const int e = code_exponent(head_max<LPH>(top));
            if (active) {
                const int h = col / D, d0 = col % D;
                const int64_t at = ((int64_t)(slot >> a.pg.shift) * a.heads + h);
                uint32_t code[2][VEC / 4];
#pragma unroll
                for (int g = 0; g < VEC / 4; ++g) {
                    code[0][g] = code[1][g] = 0;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int l = (int)code_of(lo[4 * g + j], e);
                        const int m = (int)code_of(hi[4 * g + j], e);
                        code[0][g] |= ((uint32_t)l & 255u) << (8 * j);
                        code[1][g] |= ((uint32_t)m & 255u) << (8 * j);
                    }
                }
                uint32_t* out = reinterpret_cast<uint32_t*>(a.summary + at * 2 * D + d0);
#pragma unroll
                for (int g = 0; g < VEC / 4; ++g) {
                    out[g] = code[0][g];
                    out[D / 4 + g] = code[1][g];
                }
                if (d0 == 0) a.exponents[at] = (uint8_t)(e + 127);
            }
        }
    }
}

// ------------------------------------------------------------------------------------------------
// Scores. sum_d max(c min_d, c max_d) is the product of the page's row [minima, maxima] with the
// query's [codes below zero, codes above zero], so the score of a page is one dot product of 2 D
// bytes, and of 16 pages against 16 tokens one chain of 16x16x64 int8 matrix products. The query
// heads that read one cache head are summed before: codes up to 127 G in PLANES planes of 6 bits (the
// top one signed), whose products are put together as whole numbers.
// ------------------------------------------------------------------------------------------------
typedef int32_t i32x4 __attribute__((ext_vector_type(4)));
constexpr int kTokens = 16;  // tokens of one sequence per workgroup

// 16 bytes of a query as fp32; a NaN counts as 0.
template <class E>
__device__ inline void load_query(const char* p, float (&f)[E::VEC]) {
    E::widen(*reinterpret_cast<const uint4*>(p), f);
#pragma unroll
    for (int v = 0; v < E::VEC; ++v) f[v] = f[v] != f[v] ? 0.0f : f[v];
}

// 512 tokens against 1016 pages of 8 heads of 128 take 20 us, and picking 32 of them 18 us; one kernel
// with a thread per page, plain dot products and a histogram in LDS took 290.
// Workgroup: tile blockIdx.x of kTokens tokens (tiles do not cross sequences), head blockIdx.y,
// every gridDim.z-th group of 4 x 16 pages.
template <class E, int D, int PLANES>
__global__ void __launch_bounds__(kBlock) score_kernel(SelectArgs a) {
    constexpr int ROW = 2 * D;  // bytes of a page's row
    constexpr int NF = ROW / 64;
    __shared__ __attribute__((aligned(16))) int8_t code[PLANES][kTokens][ROW + 16];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = uniform(tid >> 6);
    const int c = lane & 15, g = lane >> 4;
    const int h = blockIdx.y;
    const int64_t tile = blockIdx.x;
    const int s = find_tile_seq<kTokens>(a.b.cu, a.b.num_seqs, a.b.tokens, tile);
    const SeqInfo q = seq_info(a.b, a.pg, s);
    const int64_t i0 = (tile - tile_base<kTokens>(a.b.cu, s, a.b.tokens)) * kTokens;
    if (i0 < 0 || i0 >= q.len) return;
    const int n = (int)min((int64_t)kTokens, q.len - i0);
    const int64_t t0 = q.start + i0;

    // ---- the tokens' codes: token 4 wave + g by the 16 lanes of group g (columns past the last
    // token are multiplied too, and not looked at)
    if (const int k = 4 * wave + g; k < n) {
        constexpr int VEC = E::VEC;
        const char* base = static_cast<const char*>(a.q) +
                           ((t0 + k) * a.q_stride + (int64_t)h * a.group * D) * E::BYTES;
        float f[VEC];
        uint32_t top = 0;
        for (int j = c * VEC; j < a.group * D; j += 16 * VEC) {
            load_query<E>(base + j * E::BYTES, f);
#pragma unroll
            for (int v = 0; v < VEC; ++v) top = max(top, __float_as_uint(__builtin_fabsf(f[v])));
        }
        const int e = code_exponent(head_max<16>(top));
        for (int d = c * VEC; d < D; d += 16 * VEC) {
            int below[VEC], above[VEC];
#pragma unroll
            for (int v = 0; v < VEC; ++v) below[v] = above[v] = 0;
            for (int x = 0; x < a.group; ++x) {
                load_query<E>(base + (x * D + d) * E::BYTES, f);
#pragma unroll
                for (int v = 0; v < VEC; ++v) {
                    const int y = (int)code_of(f[v], e);
                    below[v] += min(y, 0);
                    above[v] += max(y, 0);
                }
            }
#pragma unroll
            for (int p = 0; p < PLANES; ++p)
#pragma unroll
                for (int v = 0; v < VEC; ++v) {
                    const bool last = p == PLANES - 1;
                    code[p][k][d + v] = (int8_t)(last ? below[v] >> (6 * p) : (below[v] >> (6 * p)) & 63);
                    code[p][k][D + d + v] = (int8_t)(last ? above[v] >> (6 * p) : (above[v] >> (6 * p)) & 63);
                }
        }
    }
    __syncthreads();
    i32x4 qc[PLANES][NF];
#pragma unroll
    for (int p = 0; p < PLANES; ++p)
#pragma unroll
        for (int f = 0; f < NF; ++f)
            qc[p][f] = *reinterpret_cast<const i32x4*>(&code[p][c][f * 64 + g * 16]);

    // ---- 16 pages at a time: the lane gets token c's scores of pages 4 g + i
    const int32_t* table = a.pg.table + (int64_t)s * a.pg.max_blocks;
    const int64_t last_pos = (int64_t)q.ctx + i0 + n - 1;
    const int32_t pages = (int32_t)min((int64_t)a.pg.max_blocks, (last_pos >> a.pg.shift) + 1);
    const int32_t own = (int32_t)min((int64_t)a.pg.max_blocks,
                                     (((int64_t)q.ctx + i0 + c) >> a.pg.shift) + 1);
    uint32_t* keys = a.keys + ((t0 + c) * a.heads + h) * a.key_stride;
    auto page_at = [&](uint32_t pb) { return pb < (uint32_t)pages ? table[pb] : -1; };
    const uint32_t first = (blockIdx.z * 4 + wave) * 16, stride = gridDim.z * 64;
    int32_t next = page_at(first + c);
    for (uint32_t p0 = first; p0 < (uint32_t)pages; p0 += stride) {
        const int32_t page = next;
        next = page_at(p0 + stride + c);
        const bool ok = page >= 0 && page < a.pg.num_pages;
        const int64_t at = (int64_t)(ok ? page : 0) * a.heads + h;
        i32x4 row[NF];
        int e = 0;
        if (a.pg.num_pages > 0) {  // (a pool with pages has a page 0)
#pragma unroll
            for (int f = 0; f < NF; ++f)
                row[f] = *reinterpret_cast<const i32x4*>(a.summary + at * ROW + f * 64 + g * 16);
            e = (int)a.exponents[at] - 127;
        } else {
#pragma unroll
            for (int f = 0; f < NF; ++f) row[f] = i32x4{0, 0, 0, 0};
        }
        i32x4 sum = {0, 0, 0, 0};
#pragma unroll
        for (int p = PLANES - 1; p >= 0; --p) {
#pragma unroll
            for (int i = 0; i < 4; ++i) sum[i] = (int32_t)((uint32_t)sum[i] << 6);
#pragma unroll
            for (int f = 0; f < NF; ++f)
                sum = __builtin_amdgcn_mfma_i32_16x16x64_i8(row[f], qc[p][f], sum, 0, 0, 0);
        }
        uint32_t key[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int32_t b = (int32_t)p0 + g * 4 + i;
            const int eb = __shfl(e, g * 4 + i);
            const bool usable = __shfl((int)ok, g * 4 + i);
            const bool forced = b < a.sinks || b >= (int64_t)own - a.recents;
            key[i] = forced ? 0xffffffffu : order_key(__builtin_ldexpf((float)sum[i], eb));
            if (!usable || b >= own) key[i] = 0;  // below every score: never chosen
        }
        if (c < n) {  // (rows of keys are padded to whole groups of 4)
            if (p0 + g * 4 < (uint32_t)pages)
                *reinterpret_cast<uint4*>(keys + p0 + g * 4) =
                    make_uint4(key[0], key[1], key[2], key[3]);
        }
    }
}

// ------------------------------------------------------------------------------------------------
// The pages with the largest keys, one workgroup per (token, cache head). One wave where its registers
// hold the row: the meetings of several waves cost more than their help.
// ------------------------------------------------------------------------------------------------
__device__ inline int token_pages(const SelectArgs& a, int64_t t) {
    const int s = seq_of_token(a.b, t);
    const SeqInfo q = seq_info(a.b, a.pg, s);
    const int64_t i = t - q.start;
    if (i < 0 || i >= q.len) return -1;
    const int64_t all = (((int64_t)q.ctx + i) >> a.pg.shift) + 1;
    return (int)(all < a.pg.max_blocks ? all : a.pg.max_blocks);
}

// Up to KPT keys per thread in registers, key i * THREADS + tid in register i.
template <int THREADS, int KPT>
__global__ void __launch_bounds__(THREADS) pick_kernel(SelectArgs a) {
    constexpr int WAVES = THREADS / 64;
    static_assert(KPT * WAVES <= THREADS, "one count per thread");
    __shared__ KthScratch scratch;
    __shared__ int sums[WAVES + 1];
    __shared__ int first[2][KPT * WAVES];
    const int64_t t = blockIdx.x;
    const int h = blockIdx.y, tid = threadIdx.x;
    const int wave = uniform(tid >> 6);
    const int P = token_pages(a, t);
    if (P < 0) return;  // a token behind the last sequence
    const uint32_t* keys = a.keys + (t * a.heads + h) * a.key_stride;
    int32_t* out = a.selected + (t * a.heads + h) * a.topk;
    uint32_t key[KPT];
#pragma unroll
    for (int i = 0; i < KPT; ++i) {
        const int j = i * THREADS + tid;
        key[i] = P > 0 ? keys[min(j, P - 1)] : 0u;
        if (j >= P) key[i] = 0;
    }
    const int usable = count_at_least<THREADS, KPT>(key, 1u, 0, scratch);
    __syncthreads();
    const int k = min(a.topk, usable);
    int total = 0, done = 0;
    if (k > 0) {
        uint32_t threshold;
        int ties;
        kth_of_registers<THREADS, KPT>(key, usable, k, scratch, threshold, ties);
        auto scan = [&](int list) {  // counts of (i, wave) to places
            __syncthreads();
            const int n = tid < KPT * WAVES ? first[list][tid] : 0;
            const int x = block_prefix(n, sums, total);
            if (tid < KPT * WAVES) first[list][tid] = x;
            __syncthreads();
            return total;
        };
        if (ties > 0) {  // the lowest of the equal pages
            put_counts<WAVES, KPT>(first[0], [&](int i) { return key[i] == threshold; });
            scan(0);
        }
#pragma unroll
        for (int i = 0; i < KPT; ++i) {
            bool keep = key[i] > threshold;
            if (ties > 0) {
                const bool tie = key[i] == threshold;
                keep |= tie && first[0][i * WAVES + wave] + lanes_below(__ballot(tie)) < ties;
            }
            key[i] = keep;
        }
        put_counts<WAVES, KPT>(first[1], [&](int i) { return key[i] != 0; });
        done = scan(1);
#pragma unroll
        for (int i = 0; i < KPT; ++i) {
            const uint64_t m = __ballot(key[i] != 0);
            if (key[i]) out[first[1][i * WAVES + wave] + lanes_below(m)] = i * THREADS + tid;
        }
    }
    for (int j = done + tid; j < a.topk; j += THREADS) out[j] = -1;
}

// More pages than registers hold.
__global__ void __launch_bounds__(kBlock) pick_long_kernel(SelectArgs a) {
    __shared__ uint32_t hist[258];
    __shared__ int sums[kBlock / 64 + 1];
    const int64_t t = blockIdx.x;
    const int h = blockIdx.y, tid = threadIdx.x;
    const int P = token_pages(a, t);
    if (P < 0) return;
    const uint32_t* keys = a.keys + (t * a.heads + h) * a.key_stride;
    int usable = 0, total;
    for (int j = tid; j < P; j += kBlock) usable += keys[j] != 0;
    block_prefix(usable, sums, total);
    const int k = min(a.topk, total);
    uint32_t threshold = 1;
    int ties = 0;
    if (k > 0) kth_largest([&](int j) { return keys[j]; }, P, k, hist, threshold, ties);
    int32_t* out = a.selected + (t * a.heads + h) * a.topk;
    int done = 0, tied = 0;
    for (int p0 = 0; p0 < P && k > 0; p0 += kBlock) {
        const int pb = p0 + tid;
        const uint32_t key = pb < P ? keys[pb] : 0;
        int n_tie, n_keep;
        const bool tie = key == threshold;
        const int rank = tied + block_prefix(tie, sums, n_tie);
        const bool keep = key > threshold || (tie && rank < ties);
        const int at = done + block_prefix(keep, sums, n_keep);
        if (keep) out[at] = pb;
        done += n_keep;
        tied += n_tie;
    }
    for (int j = done + tid; j < a.topk; j += kBlock) out[j] = -1;
}

template <class E, int D, bool MX>
hipError_t run_summary(const SummaryArgs& a, hipStream_t st) {
    constexpr int VEC = KeyRow<E, MX>::VEC;
    // The pages to write are known on the device only: workgroups stride over them.
    const int slices = (a.heads * (D / VEC) + 63) / 64;
    const int64_t share = (a.rebuild ? 16384 : 2048) / ((int64_t)a.b.num_seqs * slices) + 1;
    const int64_t pages = share < a.pg.max_blocks ? share : a.pg.max_blocks;
    const dim3 grid((uint32_t)pages, (uint32_t)a.b.num_seqs, (uint32_t)slices);
    summary_kernel<E, D, MX><<<grid, kBlock, 0, st>>>(a);
    return hipGetLastError();
}

template <class E, bool MX>
hipError_t summary_by_dim(const SummaryArgs& a, int D, hipStream_t st) {
    if (D == 64) return run_summary<E, 64, MX>(a, st);
    if (D == 128) return run_summary<E, 128, MX>(a, st);
    return run_summary<E, 256, MX>(a, st);
}

template <class E, int D>
hipError_t run_select(const SelectArgs& a, hipStream_t st) {
    const int64_t tiles = a.b.tokens / kTokens + a.b.num_seqs;
    // Workgroups share the pages of a tile where there are few tiles.
    const int64_t groups = ((int64_t)a.pg.max_blocks + 63) / 64;
    int64_t share = 1024 / (tiles * a.heads) + 1;
    share = share < groups ? share : groups;
    if (share > 0) {
        const dim3 grid((uint32_t)tiles, (uint32_t)a.heads, (uint32_t)share);
        // 127 G of a code's sum in planes of 6 bits and a signed one of 7
        if (a.group <= 64) score_kernel<E, D, 2><<<grid, kBlock, 0, st>>>(a);
        else score_kernel<E, D, 3><<<grid, kBlock, 0, st>>>(a);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    const dim3 each((uint32_t)a.b.tokens, (uint32_t)a.heads);
    const int32_t n = a.pg.max_blocks;
    if (n <= 16 * 64) pick_kernel<64, 16><<<each, 64, 0, st>>>(a);
    else if (n <= 16 * 256) pick_kernel<256, 16><<<each, 256, 0, st>>>(a);
    else if (n <= 64 * 256) pick_kernel<256, 64><<<each, 256, 0, st>>>(a);
    else pick_long_kernel<<<each, kBlock, 0, st>>>(a);
    return hipGetLastError();
}

template <class E>
hipError_t select_by_dim(const SelectArgs& a, int D, hipStream_t st) {
    if (D == 64) return run_select<E, 64>(a, st);
    if (D == 128) return run_select<E, 128>(a, st);
    return run_select<E, 256>(a, st);
}

}  // namespace

hipError_t launch_block_summary(const SummaryArgs& a, bool mx, int dtype, int D, hipStream_t st) {
    if (mx) return summary_by_dim<BF16, true>(a, D, st);
    return dtype == 0 ? summary_by_dim<F32, false>(a, D, st) : summary_by_dim<BF16, false>(a, D, st);
}

hipError_t launch_block_select(const SelectArgs& a, int dtype, int D, hipStream_t st) {
    return dtype == 0 ? select_by_dim<F32>(a, D, st) : select_by_dim<BF16>(a, D, st);
}

}  // namespace sc
