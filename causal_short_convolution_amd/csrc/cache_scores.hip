// The attention weight that each cached key received (shortconv_cache_scores).
#include "cache_device.h"

namespace sc {
namespace {

constexpr int kBlock = 256;

// The lane's D / 64 consecutive channels of one head of a cache row, in fp32.
template <class E, bool MX, int D>
__device__ inline void load_head(const void* cache, const void* scales, int32_t slot, int heads,
                                 int h, float (&f)[D / 64]) {
    constexpr int N = D / 64;
    const int64_t at = ((int64_t)slot * heads + h) * D + (threadIdx.x & 63) * N;
#pragma unroll
    for (int j = 0; j < N; ++j) {
        if constexpr (MX) {
            const uint8_t code = static_cast<const uint8_t*>(cache)[at + j];
            const uint8_t e = static_cast<const uint8_t*>(scales)[at >> 5];
            typedef float f32x2 __attribute__((ext_vector_type(2)));
            const f32x2 w = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(
                (uint32_t)code, __uint_as_float(e ? (uint32_t)e << 23 : 0x00400000u), false);
            f[j] = w[0];
        } else if constexpr (E::BYTES == 4) {
            f[j] = static_cast<const float*>(cache)[at + j];
        } else {
            f[j] = __uint_as_float((uint32_t)static_cast<const uint16_t*>(cache)[at + j] << 16);
        }
    }
}

__device__ inline bool looks_at(const AttnArgs& a, int64_t t, int32_t i, int32_t j) {
    if (a.mask == nullptr) return j <= i;
    if ((j >> 6) >= a.words) return false;
    return (a.mask[t * a.words + (j >> 6)] >> (j & 63)) & 1;
}

// One wave per (sequence, head, key), over the rows that look at it.
template <class E, bool MX, int D>
__global__ void __launch_bounds__(kBlock) scores_kernel(AttnArgs a) {
    constexpr int N = D / 64;
    const int h = blockIdx.y, s = blockIdx.z;
    const SeqInfo sq = seq_info(a.b, a.pg, s);
    const int64_t row = ((int64_t)s * a.heads + h) * a.capacity;
    for (int64_t p64 = blockIdx.x * 4 + (threadIdx.x >> 6); p64 < sq.keys && p64 < a.capacity;
         p64 += gridDim.x * 4) {
        const int32_t p = uniform((int32_t)p64);
        const int32_t slot = slot_of(a.pg, s, p);
        float sum = a.scores_in != nullptr && p < sq.ctx ? a.scores_in[row + p] : 0.0f;
        if (slot >= 0) {
            float k[N], q[N];
            load_head<E, MX, D>(a.cache[0], a.scales[0], slot, a.heads, h, k);
            for (int32_t i = 0; i < sq.len; ++i) {
                const int64_t t = sq.start + i;
                if (p >= sq.ctx && !looks_at(a, t, i, p - sq.ctx)) continue;
                for (int g = 0; g < a.group; ++g) {
                    const int hq = h * a.group + g;
                    load_head<E, false, D>(static_cast<const char*>(a.q) + t * a.q_stride * E::BYTES,
                                           nullptr, 0, a.heads * a.group, hq, q);
                    float x = 0.0f;
                    for (int j = 0; j < N; ++j) x = __builtin_fmaf(q[j], k[j], x);
                    x = head_sum<64>(x) * a.scale;
                    const float z = a.lse[t * a.heads * a.group + hq];
                    if (z != -__builtin_inff()) sum += __expf(x - z);
                }
            }
        }
        if ((threadIdx.x & 63) == 0) a.scores_out[row + p] = sum;
    }
}

template <class E, bool MX, int D>
hipError_t run(const AttnArgs& a, hipStream_t st) {
    const int64_t keys = (int64_t)a.pg.max_blocks << a.pg.shift;
    const uint32_t x = (uint32_t)(keys < 4096 ? (keys + 3) / 4 : 1024);
    scores_kernel<E, MX, D><<<dim3(x, a.heads, a.b.num_seqs), kBlock, 0, st>>>(a);
    return hipGetLastError();
}

template <class E, bool MX>
hipError_t by_dim(const AttnArgs& a, int D, hipStream_t st) {
    if (D == 64) return run<E, MX, 64>(a, st);
    if (D == 128) return run<E, MX, 128>(a, st);
    return run<E, MX, 256>(a, st);
}

}  // namespace

hipError_t launch_cache_scores(const AttnArgs& a, bool mx, int dtype, int D, hipStream_t st) {
    if (dtype == 0)
        return mx ? by_dim<F32, true>(a, D, st) : by_dim<F32, false>(a, D, st);
    return mx ? by_dim<BF16, true>(a, D, st) : by_dim<BF16, false>(a, D, st);
}

}  // namespace sc
