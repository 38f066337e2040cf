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

// Bits of a wave's mask for lanes below this one.
__device__ inline int lanes_below(uint64_t mask) {
    return (int)__builtin_amdgcn_mbcnt_hi((uint32_t)(mask >> 32),
                                          __builtin_amdgcn_mbcnt_lo((uint32_t)mask, 0));
}

// Leaves the wave's counts of N flags per lane in `counts`[i * WAVES + wave]. (All lanes store the
// one value: no branch, and no lane mask held for each.)
template <int WAVES, int N, class F>
__device__ inline void put_counts(int* counts, F flag) {
#pragma unroll
    for (int i = 0; i < N; ++i)
        counts[i * WAVES + (threadIdx.x >> 6)] = __builtin_popcountll(__ballot(flag(i)));
}

// LDS of kth_of_registers.
struct KthScratch {
    static constexpr int kList = 1024;
    uint32_t list[kList];
    int counts[2][16];
    uint32_t ends[2][16];
    uint32_t used;
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

// The k-th largest key lies in [lo, hi]: `reach` >= k keys are at or above lo, `above` < k are past
// hi. Halves the range while more than `stop` keys are left in it; true once the k largest are
// exactly the keys from lo on.
struct KeyRange {
    uint32_t lo, hi;
    int reach, above;
};
template <int THREADS, int KPT>
__device__ inline bool halve_range(const uint32_t (&key)[KPT], int others, int k, int stop,
                                   KeyRange& r, int& turn, KthScratch& sc) {
    while (r.lo < r.hi && r.reach - r.above > stop) {
        const uint32_t mid = r.lo + ((r.hi - r.lo) >> 1) + 1;
        const int c = others + count_at_least<THREADS, KPT>(key, mid, ++turn, sc);
        if (c >= k) {
            r.lo = mid;
            r.reach = c;
        } else {
            r.hi = mid - 1;
            r.above = c;
        }
        if (c == k) return true;
    }
    return false;
}

// The k-th largest of the n keys that a workgroup of THREADS threads holds in registers, where 0 is
// no key, 1 <= k <= n: the range between the least
// and the largest key (but for keys of all ones, which are counted first) is halved by value until
// few enough are left; those go to LDS and the search ends among them. Returns `threshold` and
// `ties`: the k largest are the keys above the threshold and `ties` of those equal to it.
template <int THREADS, int KPT>
__device__ inline void kth_of_registers(const uint32_t (&key)[KPT], int n, int k, KthScratch& sc,
                                        uint32_t& threshold, int& ties) {
    constexpr int WAVES = THREADS / 64;
    constexpr int LPT = KthScratch::kList / THREADS;
    KeyRange r{0xffffffffu, 0u, n, 0};
#pragma unroll
    for (int i = 0; i < KPT; ++i) {
        const bool top = key[i] == 0xffffffffu;
        r.above += __builtin_popcountll(__ballot(top));
        r.lo = min(r.lo, key[i] - 1);  // (0 is the largest here)
        r.hi = max(r.hi, top ? 0u : key[i]);
    }
    r.lo = ~head_max<64>(~r.lo) + 1;
    r.hi = head_max<64>(r.hi);
    if (r.lo == 0) r.lo = 0xffffffffu;  // a wave without keys
    __syncthreads();  // the scratch is free
    if ((threadIdx.x & 63) == 0) {
        sc.counts[0][threadIdx.x >> 6] = r.above;
        sc.ends[0][threadIdx.x >> 6] = r.lo;
        sc.ends[1][threadIdx.x >> 6] = r.hi;
    }
    if (threadIdx.x == 0) sc.used = 0;
    __syncthreads();
    r = KeyRange{0xffffffffu, 0u, n, 0};
#pragma unroll
    for (int w = 0; w < WAVES; ++w) {
        r.above += sc.counts[0][w];
        r.lo = min(r.lo, sc.ends[0][w]);
        r.hi = max(r.hi, sc.ends[1][w]);
    }
    r = KeyRange{(uint32_t)uniform((int32_t)r.lo), (uint32_t)uniform((int32_t)r.hi), n,
                 uniform(r.above)};
    if (r.above >= k) {
        threshold = 0xffffffffu;
        ties = k;
        return;
    }
    int turn = 0;  // (the counts above were the even half)
    bool exact = halve_range<THREADS, KPT>(key, 0, k, KthScratch::kList, r, turn, sc);
    if (!exact && r.lo < r.hi) {
        const uint32_t lo = r.lo, span = r.hi - r.lo;
        const int others = r.above;  // keys past the range
        auto left = [&](int i) { return key[i] - lo <= span; };  // unsigned: lo <= key <= hi
        int n_left = 0;
#pragma unroll
        for (int i = 0; i < KPT; ++i) n_left += __builtin_popcountll(__ballot(left(i)));
        int at = 0;  // the wave's place in the list
        if ((threadIdx.x & 63) == 0) at = (int)atomicAdd(&sc.used, (uint32_t)n_left);
        at = uniform(at);
#pragma unroll
        for (int i = 0; i < KPT; ++i) {
            const uint64_t m = __ballot(left(i));
            const int place = at + lanes_below(m);
            if (left(i) && place < KthScratch::kList) sc.list[place] = key[i];
            at += __builtin_popcountll(m);
        }
        __syncthreads();
        const int used = min((int)sc.used, KthScratch::kList);
        uint32_t mine[LPT];
#pragma unroll
        for (int i = 0; i < LPT; ++i) {
            const int j = i * THREADS + threadIdx.x;
            mine[i] = j < used ? sc.list[j] : 0u;  // (0 is below every middle)
        }
        exact = halve_range<THREADS, LPT>(mine, others, k, 0, r, turn, sc);
    }
    threshold = exact ? r.lo - 1 : r.lo;
    ties = exact ? 0 : k - r.above;
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
