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

// One workgroup per (token, cache head): the query's codes, a score for every page, the k-th
// largest score, and the chosen pages in order.
template <class E, int D>
__global__ void __launch_bounds__(kBlock) select_kernel(SelectArgs a) {
    __shared__ uint32_t hist[258];
    __shared__ int sums[8];
    __shared__ int box[2][D];  // sums over the heads of the codes below and above zero
    __shared__ uint32_t tops[4];
    const int64_t t = blockIdx.x;
    const int h = blockIdx.y;
    const int s = seq_of_token(a.b, t);
    const SeqInfo q = seq_info(a.b, a.pg, s);
    const int64_t i = t - q.start;
    if (i < 0 || i >= q.len) return;
    const int tid = threadIdx.x;
    const char* base = static_cast<const char*>(a.q) +
                       (t * a.q_stride + (int64_t)h * a.group * D) * E::BYTES;
    auto element = [&](int j) {
        const float f = E::BYTES == 4
                            ? reinterpret_cast<const float*>(base)[j]
                            : __uint_as_float((uint32_t) reinterpret_cast<const uint16_t*>(base)[j] << 16);
        return f != f ? 0.0f : f;
    };
    uint32_t top = 0;
    for (int j = tid; j < a.group * D; j += kBlock)
        top = max(top, __float_as_uint(__builtin_fabsf(element(j))));
    top = head_max<64>(top);
    if ((tid & 63) == 0) tops[tid >> 6] = top;
    __syncthreads();
    const int e = code_exponent(max(max(tops[0], tops[1]), max(tops[2], tops[3])));
    for (int d = tid; d < D; d += kBlock) {
        int below = 0, above = 0;
        for (int g = 0; g < a.group; ++g) {
            const int c = (int)code_of(element(g * D + d), e);
            below += min(c, 0);
            above += max(c, 0);
        }
        box[0][d] = below;
        box[1][d] = above;
    }
    __syncthreads();

    const int64_t pos = (int64_t)q.ctx + i;
    const int64_t all = (pos >> a.pg.shift) + 1;
    const int P = (int)(all < a.pg.max_blocks ? all : a.pg.max_blocks);
    uint32_t* keys = a.keys + (t * a.heads + h) * a.pg.max_blocks;
    const int32_t* table = a.pg.table + (int64_t)s * a.pg.max_blocks;
    int usable = 0;
    for (int pb = tid; pb < P; pb += kBlock) {
        const int32_t page = table[pb];
        uint32_t key = 0;  // below every score: never chosen
        if (page >= 0 && page < a.pg.num_pages) {
            ++usable;
            if (pb < a.sinks || pb >= (int64_t)P - a.recents) {
                key = 0xffffffffu;
            } else {
                const int64_t at = (int64_t)page * a.heads + h;
                const uint32_t* row = reinterpret_cast<const uint32_t*>(a.summary + at * 2 * D);
                const int* w = &box[0][0];
                int sum = 0;
                for (int j = 0; j < D / 2; ++j) {
                    const uint32_t x = row[j];
                    sum += (int)(int8_t)(x) * w[4 * j] + (int)(int8_t)(x >> 8) * w[4 * j + 1] +
                           (int)(int8_t)(x >> 16) * w[4 * j + 2] + (int)(int8_t)(x >> 24) * w[4 * j + 3];
                }
                key = order_key(__builtin_ldexpf((float)sum, (int)a.exponents[at] - 127));
            }
        }
        keys[pb] = key;
    }
    int total;
    block_prefix(usable, sums, total);
    __syncthreads();  // the keys of every thread are written
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
    select_kernel<E, D><<<dim3((uint32_t)a.b.tokens, (uint32_t)a.heads), kBlock, 0, st>>>(a);
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
