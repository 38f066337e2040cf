// Device helpers of the cache operators: the sequence of a token, page lookup, and the selection
// of the largest keys of a list.
#ifndef SHORTCONV_CACHE_DEVICE_H
#define SHORTCONV_CACHE_DEVICE_H

#include "cache_internal.h"
#include "device_common.h"

namespace sc {

// The largest s in [0, n) with clamp(cu[s]) <= t (0 if none), by whole waves: each round 64 lanes
// test 64 evenly spaced candidates, as in find_tile_seq.
__device__ inline int seq_of_token(const Batch& b, int64_t t) {
    const int wl = threadIdx.x & 63;
    int base = 0, count = b.num_seqs;
    while (count > 1) {
        const int step = (count + 63) / 64;
        const bool ok = wl * step < count && clamp_tok(b.cu[base + wl * step], b.tokens) <= t;
        const uint64_t mask = __ballot(ok);
        const int last = mask ? 63 - __builtin_clzll(mask) : 0;
        base += last * step;
        count = step < count - last * step ? step : count - last * step;
    }
    return uniform(base);
}

// One sequence of a batch: its new tokens [start, start + len), its cached keys, and the number
// of keys in all, which the page table bounds.
struct SeqInfo {
    int64_t start;
    int32_t len;
    int32_t ctx;
    int32_t keys;
};
__device__ inline SeqInfo seq_info(const Batch& b, const Paging& pg, int s) {
    SeqInfo r;
    const int32_t c0 = clamp_tok(b.cu[s], b.tokens);
    const int32_t c1 = clamp_tok(b.cu[s + 1], b.tokens);
    const int32_t cap = pg.max_blocks << pg.shift;
    const int32_t ctx = b.ctx[s];
    r.start = c0;
    r.len = c1 > c0 ? c1 - c0 : 0;
    r.ctx = ctx < 0 ? 0 : (ctx > cap ? cap : ctx);
    r.keys = r.len < cap - r.ctx ? r.ctx + r.len : cap;
    return r;
}

// The cache row of position p (0 <= p < max_blocks << shift), or -1 where the page is outside the
// pool.
__device__ inline int32_t slot_of(const Paging& pg, int s, int32_t p) {
    const int32_t page = pg.table[(int64_t)s * pg.max_blocks + (p >> pg.shift)];
    const bool ok = page >= 0 && page < pg.num_pages;
    return ok ? (page << pg.shift) + (p & ((1 << pg.shift) - 1)) : -1;
}

// Maximum over the LPH lanes of a head of values whose bit patterns order as unsigned integers
// (magnitudes of floats).
template <int LPH>
__device__ inline uint32_t head_max(uint32_t v) {
    v = max(v, dpp_u32<kQuadXor1>(v));
    v = max(v, dpp_u32<kQuadXor2>(v));
    v = max(v, dpp_u32<kRowHalfMirror>(v));
    if (LPH >= 16) v = max(v, dpp_u32<kRowMirror>(v));
    if (LPH >= 32) {
        const auto p = __builtin_amdgcn_permlane16_swap(v, v, false, false);
        v = max((uint32_t)p[0], (uint32_t)p[1]);
    }
    if (LPH >= 64) {
        const auto p = __builtin_amdgcn_permlane32_swap(v, v, false, false);
        v = max((uint32_t)p[0], (uint32_t)p[1]);
    }
    return v;
}

// N values to consecutive elements of type E, rounded once, in the widest stores that fit.
template <class E, int N>
__device__ inline void store_row(void* out, int64_t at, const float (&y)[N]) {
    if constexpr (E::BYTES == 4) {
        float* o = static_cast<float*>(out) + at;
        if constexpr (N % 4 == 0) {
#pragma unroll
            for (int j = 0; j < N; j += 4)
                *reinterpret_cast<float4*>(o + j) = make_float4(y[j], y[j + 1], y[j + 2], y[j + 3]);
        } else {
#pragma unroll
            for (int j = 0; j < N; ++j) o[j] = y[j];
        }
    } else {
        uint16_t* o = static_cast<uint16_t*>(out) + at;
        if constexpr (N == 1) {
            *reinterpret_cast<__bf16*>(o) = (__bf16)y[0];
        } else if constexpr (N == 2) {
            *reinterpret_cast<uint32_t*>(o) = BF16::pack2(y[0], y[1]);
        } else if constexpr (N == 4) {
            *reinterpret_cast<uint2*>(o) = make_uint2(BF16::pack2(y[0], y[1]), BF16::pack2(y[2], y[3]));
        } else {
            static_assert(N == 8, "elements per store");
            *reinterpret_cast<uint4*>(o) = BF16::narrow(y);
        }
    }
}

// Floats as unsigned integers in the same order (no NaN; -0 counts as +0).
__device__ inline uint32_t order_key(float f) {
    const uint32_t u = __float_as_uint(f + 0.0f);
    return (u >> 31) ? ~u : (u | 0x80000000u);
}

// The exponent E of a group of values whose largest magnitude has the bit pattern `top`:
// floor(log2) - 6, at least -127, so that the magnitude times 2^-E lies in [64, 128).
__device__ inline int code_exponent(uint32_t top) { return max((int)(top >> 23) - 133, -127); }

// One value as a whole number in +-127 under the exponent E.
__device__ inline float code_of(float x, int e) {
    return __builtin_amdgcn_fmed3f(__builtin_rintf(__builtin_ldexpf(x, -e)), -127.0f, 127.0f);
}

// The k-th largest of n keys, by one workgroup, 8 bits at a time: `threshold` is its value and
// `ties` how many keys equal to it belong to the k largest. 1 <= k <= n. `hist` is LDS of
// 256 + 2 words; key(i) gives key i. Every thread of the workgroup takes part, and all return the
// same. The counts are whole numbers, so the order of the atomics does not matter.
template <class Key>
__device__ inline void kth_largest(Key key, int n, int k, uint32_t* hist, uint32_t& threshold,
                                   int& ties) {
    uint32_t prefix = 0;
    int rest = k;
    for (int shift = 24; shift >= 0; shift -= 8) {
        for (int i = threadIdx.x; i < 256; i += blockDim.x) hist[i] = 0;
        __syncthreads();
        for (int i = threadIdx.x; i < n; i += blockDim.x) {
            const uint32_t x = key(i);
            if (shift == 24 || (x >> (shift + 8)) == (prefix >> (shift + 8)))
                atomicAdd(&hist[(x >> shift) & 255u], 1u);
        }
        __syncthreads();
        if (threadIdx.x < 64) {  // lane l owns bins 4l..4l+3; suffix sums from the top bin
            const int l = threadIdx.x;
            const uint32_t b0 = hist[4 * l], b1 = hist[4 * l + 1], b2 = hist[4 * l + 2],
                           b3 = hist[4 * l + 3];
            const uint32_t own = b0 + b1 + b2 + b3;
            uint32_t above = own;  // inclusive suffix sum over lanes
            for (int d = 1; d < 64; d <<= 1) {
                const uint32_t o = __shfl_down(above, d);
                if (l + d < 64) above += o;
            }
            above -= own;  // keys in higher lanes' bins
            uint32_t c = above;
            const uint32_t bins[4] = {b0, b1, b2, b3};
            for (int j = 3; j >= 0; --j) {
                if (c < (uint32_t)rest && c + bins[j] >= (uint32_t)rest) {
                    hist[256] = 4 * l + j;
                    hist[257] = c;
                }
                c += bins[j];
            }
        }
        __syncthreads();
        prefix |= hist[256] << shift;
        rest -= (int)hist[257];
        __syncthreads();
    }
    threshold = prefix;
    ties = rest;
}

// LDS of kth_of_registers.
struct KthScratch {
    static constexpr int kList = 1024;
    uint32_t list[kList];
    int counts[2][16];
    uint32_t used, differ;
};

// Keys of the workgroup at or above `cand`, in every thread: a compare per key and a population
// count of the wave's result, then one meeting of the waves. `turn` alternates the halves of
// the counts, since the other half may still be read.
template <int THREADS, int KPT>
__device__ inline int count_at_least(const uint32_t (&key)[KPT], uint32_t cand, int turn,
                                     KthScratch& sc) {
    constexpr int WAVES = THREADS / 64;
    int n = 0;
#pragma unroll
    for (int i = 0; i < KPT; ++i) n += __builtin_popcountll(__ballot(key[i] >= cand));
    int* slot = sc.counts[turn & 1];
    if ((threadIdx.x & 63) == 0) slot[threadIdx.x >> 6] = n;
    __syncthreads();
    n = 0;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) n += slot[w];
    return uniform(n);
}

// The k-th largest of n keys that a workgroup of THREADS threads holds in registers, key
// i * THREADS + threadIdx.x in register i (0 past the n-th), 1 <= k <= n: bit by bit from the top, each bit kept if at least k keys reach the
// value with it. Once few enough keys can still be it, those go to LDS and the remaining bits are
// found among them, from the highest bit they differ in. Returns `threshold` and `ties`: the k
// largest are the keys above the threshold and `ties` of those equal to it.
template <int THREADS, int KPT>
__device__ inline void kth_of_registers(const uint32_t (&key)[KPT], int n, int k, KthScratch& sc,
                                        uint32_t& threshold, int& ties) {
    constexpr int LPT = KthScratch::kList / THREADS;
    uint32_t t = 0;
    int above = 0;    // keys past those that can still be the k-th largest
    int reach = n;    // keys at or above t
    int bit = 31;
    __syncthreads();
    if (threadIdx.x == 0) sc.used = sc.differ = 0;
    for (; bit >= 0 && reach - above > KthScratch::kList; --bit) {
        const uint32_t cand = t | (1u << bit);
        const int c = count_at_least<THREADS, KPT>(key, cand, bit, sc);
        if (c >= k) {
            t = cand;
            reach = c;
        } else {
            above = c;
        }
        if (c == k) {  // exactly the keys from here on
            threshold = cand - 1;
            ties = 0;
            return;
        }
    }
    if (bit < 0) {
        threshold = t;
        ties = k - above;
        return;
    }
    __syncthreads();  // `used` is cleared, and no wave still reads the counts
    const uint32_t span = bit == 31 ? 0xffffffffu : (2u << bit) - 1u;  // keys t .. t + span are left
#pragma unroll
    for (int i = 0; i < KPT; ++i) {
        // key >= t and key <= t + span, unsigned
        const bool left = i * THREADS + (int)threadIdx.x < n && key[i] - t <= span;
        const uint64_t m = __ballot(left);
        if (m == 0) continue;
        uint32_t at = 0;
        if ((threadIdx.x & 63) == 0) at = atomicAdd(&sc.used, (uint32_t)__builtin_popcountll(m));
        at = (uint32_t)uniform((int32_t)at) +
             __builtin_amdgcn_mbcnt_hi((uint32_t)(m >> 32),
                                       __builtin_amdgcn_mbcnt_lo((uint32_t)m, 0));
        if (left && at < KthScratch::kList) sc.list[at] = key[i];
    }
    __syncthreads();
    const int used = min((int)sc.used, KthScratch::kList);
    const uint32_t probe = sc.list[0];
    uint32_t mine[LPT], differ = 0;
#pragma unroll
    for (int i = 0; i < LPT; ++i) {
        const int j = i * THREADS + threadIdx.x;
        mine[i] = j < used ? sc.list[j] : 0u;
        if (j < used) differ |= mine[i] ^ probe;
    }
    if (__ballot(differ != 0)) atomicOr(&sc.differ, differ);
    __syncthreads();
    differ = sc.differ;
    // the bits that all share are the k-th largest's too
    const int high = differ ? 31 - __builtin_clz(differ) : -1;
    t = high == 31 ? 0u : high < 0 ? probe : probe & ~((2u << high) - 1u);
    for (bit = high; bit >= 0; --bit) {
        const uint32_t cand = t | (1u << bit);
        const int c = above + count_at_least<THREADS, LPT>(mine, cand, bit, sc);
        if (c >= k) t = cand;
        if (c == k) {
            threshold = cand - 1;
            ties = 0;
            return;
        }
    }
    int more = 0;
    if (t != 0xffffffffu) more = count_at_least<THREADS, LPT>(mine, t + 1, bit, sc);
    threshold = t;
    ties = k - above - more;
}

// Exclusive prefix sum over the workgroup of one small count per thread, and the total. `sums` is
// LDS of one word per wave plus one.
__device__ inline int block_prefix(int v, int* sums, int& total) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
    int inc = v;
    for (int d = 1; d < 64; d <<= 1) {
        const int o = __shfl_up(inc, d);
        if (lane >= d) inc += o;
    }
    __syncthreads();  // the sums of an earlier call have been read
    if (lane == 63) sums[wave] = inc;
    __syncthreads();
    int before = 0, all = 0;
    for (int w = 0; w < waves; ++w) {
        const int c = sums[w];
        if (w < wave) before += c;
        all += c;
    }
    total = all;
    return before + inc - v;
}

}  // namespace sc

#endif  // SHORTCONV_CACHE_DEVICE_H
