// Attention over the paged cache (shortconv_tree_attention, shortconv_block_attention) and the sums
// of its weights (shortconv_cache_scores).
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

// One wave per (token, query head): keys one after the other with a running maximum and sum.
template <class E, bool MX, int D, bool SPARSE>
__global__ void __launch_bounds__(kBlock) attention_kernel(AttnArgs a) {
    constexpr int N = D / 64;
    const int64_t t = blockIdx.x;
    const int hq = uniform((int)(blockIdx.y * 4 + (threadIdx.x >> 6)));
    const int s = seq_of_token(a.b, t);
    const SeqInfo sq = seq_info(a.b, a.pg, s);
    const int64_t i64 = t - sq.start;
    if (i64 < 0 || i64 >= sq.len || hq >= a.heads * a.group) return;
    const int32_t i = (int32_t)i64;
    const int h = hq / a.group;
    float q[N], o[N];
    load_head<E, false, D>(static_cast<const char*>(a.q) + t * a.q_stride * E::BYTES, nullptr, 0,
                           a.heads * a.group, hq, q);
    for (int j = 0; j < N; ++j) o[j] = 0.0f;
    float m = -__builtin_inff(), l = 0.0f;
    auto key = [&](int32_t p) {
        const int32_t slot = slot_of(a.pg, s, p);
        if (slot < 0) return;
        float k[N], v[N];
        load_head<E, MX, D>(a.cache[0], a.scales[0], slot, a.heads, h, k);
        load_head<E, MX, D>(a.cache[1], a.scales[1], slot, a.heads, h, v);
        float x = 0.0f;
        for (int j = 0; j < N; ++j) x = __builtin_fmaf(q[j], k[j], x);
        x = head_sum<64>(x) * a.scale;
        const float top = __builtin_fmaxf(m, x);
        if (top == -__builtin_inff()) return;
        const float old = __expf(m - top), w = __expf(x - top);
        l = l * old + w;
        for (int j = 0; j < N; ++j) o[j] = __builtin_fmaf(w, v[j], o[j] * old);
        m = top;
    };
    if constexpr (SPARSE) {
        const int32_t last = min((int64_t)sq.keys - 1, (int64_t)sq.ctx + i);
        for (int c = 0; c < a.topk; ++c) {
            const int32_t pb = a.selected[(t * a.heads + h) * a.topk + c];
            if (pb < 0 || pb >= a.pg.max_blocks) continue;
            for (int r = 0; r < (1 << a.pg.shift); ++r) {
                const int32_t p = (pb << a.pg.shift) + r;
                if (p <= last) key(p);
            }
        }
    } else {
        for (int32_t p = 0; p < sq.keys; ++p)
            if (p < sq.ctx || looks_at(a, t, i, p - sq.ctx)) key(p);
    }
    const float inv = l > 0.0f || l != l ? 1.0f / l : 0.0f;
    const int64_t at = (t * a.heads * a.group + hq) * D + (threadIdx.x & 63) * N;
    for (int j = 0; j < N; ++j) {
        const float y = o[j] * inv;
        if constexpr (E::BYTES == 4) static_cast<float*>(a.out)[at + j] = y;
        else static_cast<__bf16*>(a.out)[at + j] = (__bf16)y;
    }
    if (a.lse != nullptr && (threadIdx.x & 63) == 0)
        a.lse[t * a.heads * a.group + hq] = l > 0.0f || l != l ? m + __logf(l) : -__builtin_inff();
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
hipError_t run(const AttnArgs& a, int what, hipStream_t st) {
    if (what == 2) {
        const int64_t keys = (int64_t)a.pg.max_blocks << a.pg.shift;
        const uint32_t x = (uint32_t)(keys < 4096 ? (keys + 3) / 4 : 1024);
        scores_kernel<E, MX, D><<<dim3(x, a.heads, a.b.num_seqs), kBlock, 0, st>>>(a);
    } else {
        const dim3 grid((uint32_t)a.b.tokens, (uint32_t)(a.heads * a.group + 3) / 4);
        if (what == 1) attention_kernel<E, MX, D, true><<<grid, kBlock, 0, st>>>(a);
        else attention_kernel<E, MX, D, false><<<grid, kBlock, 0, st>>>(a);
    }
    return hipGetLastError();
}

template <class E, bool MX>
hipError_t by_dim(const AttnArgs& a, int what, int D, hipStream_t st) {
    if (D == 64) return run<E, MX, 64>(a, what, st);
    if (D == 128) return run<E, MX, 128>(a, what, st);
    return run<E, MX, 256>(a, what, st);
}

hipError_t dispatch(const AttnArgs& a, int what, bool mx, int dtype, int D, hipStream_t st) {
    if (dtype == 0)
        return mx ? by_dim<F32, true>(a, what, D, st) : by_dim<F32, false>(a, what, D, st);
    return mx ? by_dim<BF16, true>(a, what, D, st) : by_dim<BF16, false>(a, what, D, st);
}

}  // namespace

hipError_t launch_tree_attention(const AttnArgs& a, bool mx, int dtype, int D, hipStream_t st) {
    return dispatch(a, 0, mx, dtype, D, st);
}
hipError_t launch_block_attention(const AttnArgs& a, bool mx, int dtype, int D, hipStream_t st) {
    return dispatch(a, 1, mx, dtype, D, st);
}
hipError_t launch_cache_scores(const AttnArgs& a, bool mx, int dtype, int D, hipStream_t st) {
    return dispatch(a, 2, mx, dtype, D, st);
}

}  // namespace sc
