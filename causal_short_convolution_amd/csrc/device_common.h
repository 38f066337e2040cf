// Device helpers shared by the HIP kernels of the fused ShortConv K/V step (forward, speculative
// verification, MXFP8 encoding and backward): element types, 16-byte row access with streaming
// hints, cross-lane moves and reductions, the tile -> sequence search of the prefill grids, the row
// math and the cache row formats.
// Internal to the library; not part of the C ABI.
#ifndef SHORTCONV_DEVICE_COMMON_H
#define SHORTCONV_DEVICE_COMMON_H

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "shortconv_internal.h"

namespace sc {

// ------------------------------------------------------------------------------------------------
// Element types. A "packet" is the 16 bytes one lane moves: uint4.
// ------------------------------------------------------------------------------------------------
struct F32 {
    static constexpr int VEC = 4;
    static constexpr int BYTES = 4;
    __device__ static inline void widen(const uint4& r, float (&f)[VEC]) {
        f[0] = __uint_as_float(r.x);
        f[1] = __uint_as_float(r.y);
        f[2] = __uint_as_float(r.z);
        f[3] = __uint_as_float(r.w);
    }
    __device__ static inline uint4 narrow(const float (&f)[VEC]) {
        return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                          __float_as_uint(f[3]));
    }
};

typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));

struct BF16 {
    static constexpr int VEC = 8;
    static constexpr int BYTES = 2;
    __device__ static inline void widen(const uint4& r, float (&f)[VEC]) {
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(w[i] << 16);
            f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    // Round to nearest even (one v_cvt_pk_bf16_f32 per pair on gfx950).
    __device__ static inline uint32_t pack2(float a, float b) {
        bf16x2_t p = {(__bf16)a, (__bf16)b};
        return __builtin_bit_cast(uint32_t, p);
    }
    __device__ static inline uint4 narrow(const float (&f)[VEC]) {
        return make_uint4(pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]),
                          pack2(f[6], f[7]));
    }
};

__device__ inline uint4 ld16(const void* base, int64_t elem_off, int bytes) {
    return *reinterpret_cast<const uint4*>(static_cast<const char*>(base) + elem_off * bytes);
}
__device__ inline void st16(void* base, int64_t elem_off, int bytes, const uint4& v) {
    *reinterpret_cast<uint4*>(static_cast<char*>(base) + elem_off * bytes) = v;
}
// Row access as (wave-uniform byte base, per-lane 32-bit byte offset). K/V rows are read once and
// cache rows are written once, so both stream with the non-temporal hint: they do not displace
// reusable lines (taps, gamma, metadata) from L2 and the Infinity Cache, and dirty cache rows do
// not linger there (measured on MI355X: a cold 140 MB copy streams at ~5.7 TB/s with the hint
// against ~3.0 TB/s without).
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
__device__ inline uint4 ldrow(const char* base, uint32_t lane_off) {
    const u32x4 v = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(base + lane_off));
    return make_uint4(v.x, v.y, v.z, v.w);
}
// The same load without the streaming hint. The kernels use it for a few rows of each span (a
// mix that measured faster than streaming every row; see where it is used).
__device__ inline uint4 ldrow_keep(const char* base, uint32_t lane_off) {
    return *reinterpret_cast<const uint4*>(base + lane_off);
}
__device__ inline void strow(char* base, uint32_t lane_off, const uint4& v) {
    const u32x4 w = {v.x, v.y, v.z, v.w};
    __builtin_nontemporal_store(w, reinterpret_cast<u32x4*>(base + lane_off));
}

// Waits until every vector memory access this wave has issued is complete (s_waitcnt vmcnt(0),
// other counters unconstrained). On gfx9 stores count in vmcnt too: where a span's row loads are
// followed by conditional cache stores, the compiler cannot tell how many operations follow a
// row and waits for all of them, stores included, before each row. One explicit wait for the
// rows before the loop leaves nothing in flight that a row could be waiting on.
__device__ inline void wait_vmem() { __builtin_amdgcn_s_waitcnt(0x0F70); }

// Values that are the same in every lane, moved to scalar registers so that the compiler uses
// scalar loads for per-token metadata and scalar base addresses for the row accesses.
__device__ inline int32_t uniform(int32_t v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ inline int64_t uniform(int64_t v) {
    const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v);
    const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)((uint64_t)v >> 32));
    return (int64_t)(((uint64_t)hi << 32) | lo);
}

// Per-lane choice between the K and the V member of a pair of kernel arguments. Both members are
// read as scalars and the lane selects; indexing the pair with the lane's tensor would instead be
// a vector load from the argument segment, and every address derived from it would wait for it.
template <class P>
__device__ inline P pick(const P (&pair)[2], int tensor) {
    const P k = pair[0];
    const P v = pair[1];
    return tensor ? v : k;
}

// Lane i's value of v, as a wave-uniform (scalar) value.
__device__ inline int64_t lane_value(int64_t v, int i) {
    const uint32_t lo = __builtin_amdgcn_readlane((uint32_t)v, i);
    const uint32_t hi = __builtin_amdgcn_readlane((uint32_t)((uint64_t)v >> 32), i);
    return (int64_t)(((uint64_t)hi << 32) | lo);
}

// Data-parallel-primitive lane moves (row = 16 lanes).
template <int CTRL>
__device__ inline float dpp(float v) {
    return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), CTRL, 0xf, 0xf, true));
}
template <int CTRL>
__device__ inline uint32_t dpp_u32(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, CTRL, 0xf, 0xf, true);
}
constexpr int kQuadXor1 = 0xB1;       // quad_perm [1,0,3,2]
constexpr int kQuadXor2 = 0x4E;       // quad_perm [2,3,0,1]
constexpr int kRowHalfMirror = 0x141; // lane i <-> 7-i within each half row
constexpr int kRowMirror = 0x140;     // lane i <-> 15-i within each row

// Sum over the LPH lanes that own one head (aligned groups, LPH | 64). A butterfly: at every step
// each lane adds its value and its partner's, the partner adds the same two values in the other
// order, so all lanes of the group end with the same bits. Within a 16-lane row the partners come
// from DPP moves; the quad steps make the 4 lanes of a quad equal, so the mirror moves pair each
// lane with a lane of the neighbouring quad (half row) or half row (row). Across rows, gfx950's
// permlane swaps give every lane its own value and its partner's (lane ^ 16, lane ^ 32) in one
// VALU instruction, as two outputs whose sum is own + partner in every lane.
template <int LPH>
__device__ inline float head_sum(float v) {
    static_assert(LPH == 8 || LPH == 16 || LPH == 32 || LPH == 64, "lanes per head");
    v += dpp<kQuadXor1>(v);
    v += dpp<kQuadXor2>(v);
    v += dpp<kRowHalfMirror>(v);
    if (LPH >= 16) v += dpp<kRowMirror>(v);
    if (LPH >= 32) {
        const uint32_t u = __float_as_uint(v);
        const auto p = __builtin_amdgcn_permlane16_swap(u, u, false, false);
        v = __uint_as_float(p[0]) + __uint_as_float(p[1]);
    }
    if (LPH >= 64) {
        const uint32_t u = __float_as_uint(v);
        const auto p = __builtin_amdgcn_permlane32_swap(u, u, false, false);
        v = __uint_as_float(p[0]) + __uint_as_float(p[1]);
    }
    return v;
}

__device__ inline int32_t clamp_tok(int32_t v, int64_t T) {
    return v < 0 ? 0 : (v > T ? (int32_t)T : v);
}

template <int BB>
__device__ inline int64_t tile_base(const int32_t* cu, int s, int64_t T) {
    return (int64_t)(clamp_tok(cu[s], T) / BB) + s;
}

// The largest s in [0, n) with P(s) <= tile, P(s) = floor(cu[s] / BB) + s (strictly increasing).
// Wave-parallel: each round the 64 lanes test 64 evenly spaced candidates with one vector load and
// a ballot narrows the range 64-fold, so n <= 64 costs one memory round trip and n <= 4096 two,
// where a binary search would chain log2(n) dependent loads. Must be called by whole waves.
template <int BB>
__device__ inline int find_tile_seq(const int32_t* cu, int n, int64_t T, int64_t tile) {
    const int wl = threadIdx.x & 63;
    int base = 0, count = n;
    while (count > 1) {
        const int step = (count + 63) / 64;
        const int cand = base + wl * step;
        const bool ok = wl * step < count && tile_base<BB>(cu, cand, T) <= tile;
        const uint64_t mask = __ballot(ok);
        // P(base) <= tile always holds for a tile that belongs to some sequence; the prefix of
        // set bits ends at the last candidate that still starts at or before the tile.
        const int last = mask ? 63 - __builtin_clzll(mask) : 0;
        base += last * step;
        count = step < count - last * step ? step : count - last * step;
    }
    return uniform(base);
}

// find_tile_seq, also giving the sequence's bounds clamp_tok(cu[s]) and clamp_tok(cu[s + 1]) as
// wave-uniform values. For n <= 63 one round decides: lane l loads cu[min(l, n)], so the bounds
// are read from lanes s and s + 1 of that same load, with no further dependent load before the
// rows' addresses are known. Measured on MI355X (one process, medians of 5): varlen bf16 prefill
// of 8 sequences 28.03 -> 27.41 us, with MXFP8 rows 24.65 -> 23.76 us; in the backward neutral
// (57.8 us), and for one sequence (long prefill, W = 8) 1-3 % slower, where the plain search
// issues no vector load at all: there the kernels keep find_tile_seq. Must be called by whole
// waves.
template <int BB>
__device__ inline int tile_seq_bounds(const int32_t* cu, int n, int64_t T, int64_t tile,
                                      int64_t& start, int64_t& end) {
    if (n <= 63) {
        const int wl = threadIdx.x & 63;
        const int32_t c = clamp_tok(cu[wl <= n ? wl : n], T);
        const bool ok = wl < n && (int64_t)(c / BB) + wl <= tile;  // P(wl) <= tile
        const uint64_t mask = __ballot(ok);
        const int s = uniform(mask ? 63 - __builtin_clzll(mask) : 0);
        start = (int64_t)__builtin_amdgcn_readlane(c, s);
        end = (int64_t)__builtin_amdgcn_readlane(c, s + 1);
        return s;
    }
    const int s = find_tile_seq<BB>(cu, n, T, tile);
    start = uniform((int64_t)clamp_tok(cu[s], T));
    end = uniform((int64_t)clamp_tok(cu[s + 1], T));
    return s;
}

// ------------------------------------------------------------------------------------------------
// The row math and the cache row formats (prefill, decode, verification of chains and trees).
// ------------------------------------------------------------------------------------------------
// Per-lane constants of one (tensor, head, 16-byte column) position.
template <class E, int W>
struct LaneParams {
    float tap[W][E::VEC];
    float gam[E::VEC];
};

template <class E, int W>
__device__ inline void load_params(const float* taps, const float* gamma, int heads, int D, int h,
                                   int d0, LaneParams<E, W>& p) {
#pragma unroll
    for (int k = 0; k < W; ++k) {
        const float* t = taps + ((int64_t)k * heads + h) * D + d0;
#pragma unroll
        for (int v = 0; v < E::VEC; v += 4) {
            const float4 q = *reinterpret_cast<const float4*>(t + v);
            p.tap[k][v] = q.x;
            p.tap[k][v + 1] = q.y;
            p.tap[k][v + 2] = q.z;
            p.tap[k][v + 3] = q.w;
        }
    }
#pragma unroll
    for (int v = 0; v < E::VEC; v += 4) {
        const float4 q = *reinterpret_cast<const float4*>(gamma + d0 + v);
        p.gam[v] = q.x;
        p.gam[v + 1] = q.y;
        p.gam[v + 2] = q.z;
        p.gam[v + 3] = q.w;
    }
}

// The row math of one output row slice: window row k (k = W-1 is the current token) is
// win[(off + k) % W], off being a compile-time constant after unrolling; o gets the normalized
// values in fp32, before the one rounding to the cache format.
template <class E, int W, int LPH>
__device__ inline void fused_row(const float (&win)[W][E::VEC], int off,
                                 const LaneParams<E, W>& p, float eps, float inv_d,
                                 float (&o)[E::VEC]) {
    constexpr int VEC = E::VEC;
    float c[VEC];
#pragma unroll
    for (int v = 0; v < VEC; ++v) c[v] = p.tap[0][v] * win[off % W][v];
#pragma unroll
    for (int k = 1; k < W; ++k)
#pragma unroll
        for (int v = 0; v < VEC; ++v)
            c[v] = __builtin_fmaf(p.tap[k][v], win[(off + k) % W][v], c[v]);
    float ss = 0.0f;
#pragma unroll
    for (int v = 0; v < VEC; ++v) ss = __builtin_fmaf(c[v], c[v], ss);
    ss = head_sum<LPH>(ss);
    // v_rsq_f32: within ~1 ulp of 1/sqrt, one instruction instead of a correctly rounded square
    // root and divide; it scales exactly under power-of-4 scaling of its input.
    const float inv = __builtin_amdgcn_rsqf(__builtin_fmaf(ss, inv_d, eps));
#pragma unroll
    for (int v = 0; v < VEC; ++v) o[v] = (c[v] * inv) * p.gam[v];
}

// ------------------------------------------------------------------------------------------------
// Cache formats. A Sink takes one finished row slice (VEC fp32 values of one head) and writes it
// to cache row `slot`, unless the slot is outside [0, num_slots) or the lane is idle.
// ------------------------------------------------------------------------------------------------
// Plain rows in the I/O element type (one round-to-nearest-even conversion).
template <class E>
struct PlainSink {
    char* cache;
    int64_t row_bytes;
    uint32_t lane_off;
    int64_t num_slots;
    __device__ PlainSink(const StepArgs& a, int tensor, int h, int d0, int D)
        : cache(static_cast<char*>(pick(a.cache, tensor))),
          row_bytes((int64_t)a.heads * D * E::BYTES),
          lane_off((uint32_t)(((int64_t)h * D + d0) * E::BYTES)),
          num_slots(a.num_slots) {}
    // A row slice in its stored form, and its store (skipped for an idle lane or a slot outside
    // the pool).
    using Enc = uint4;
    __device__ Enc encode(const float (&o)[E::VEC]) const { return E::narrow(o); }
    // The slot is wave-uniform in every caller; its byte offset is kept scalar (read through
    // readfirstlane), so the address is one add to the lane's base instead of a 64-bit
    // multiply-add on the vector unit at quarter rate.
    __device__ void write(int64_t slot, bool active, const Enc& out) const {
        if (active && slot >= 0 && slot < num_slots)
            strow(cache + uniform(slot * row_bytes), lane_off, out);
    }
    __device__ void put(int64_t slot, bool active, const float (&o)[E::VEC]) const {
        write(slot, active, encode(o));
    }
};

// OCP FP8 E4M3 codes of v[b] * 2^-e for four finite values (byte b): nearest value, ties to even,
// saturating at +-448. gfx950's scaled conversion (v_cvt_scalef32_pk_fp8_f32) divides by its
// scale operand, here 2^e, exactly and rounds to nearest even into the OCP format, but does not
// saturate; clamping v to +-448 * 2^e first is the same as clamping v * 2^-e to +-448, scaling by
// a power of two being exact.
typedef short sc_i16x2 __attribute__((ext_vector_type(2)));
__device__ inline uint32_t e4m3x4_scaled(float v0, float v1, float v2, float v3, float scale,
                                         float lim) {
    v0 = __builtin_amdgcn_fmed3f(v0, -lim, lim);
    v1 = __builtin_amdgcn_fmed3f(v1, -lim, lim);
    v2 = __builtin_amdgcn_fmed3f(v2, -lim, lim);
    v3 = __builtin_amdgcn_fmed3f(v3, -lim, lim);
    // the two conversions write the low and the high half; the word they start from (any
    // register at hand) is overwritten entirely
    sc_i16x2 w = __builtin_bit_cast(sc_i16x2, __float_as_uint(v0));
    w = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(w, v0, v1, scale, false);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(w, v2, v3, scale, true);
    return __builtin_bit_cast(uint32_t, w);
}

// The MXFP8 encoding of one lane's VEC values: the maximum over the 32/VEC lanes of a 32-element
// block (DPP), the E8M0 exponent e = floor(log2(max)) - 8 clamped to [-127, 127] (-127 for an
// all-zero block), and the saturated E4M3 codes of v * 2^-e. Across lanes the maximum of the
// magnitudes is taken on their bit patterns, which order non-negative finite floats as unsigned
// integers do; the pattern's exponent field E gives floor(log2(max)) = E - 127 for a normal
// maximum, so e = E - 135, which is at most 119, and every zero or subnormal maximum (E = 0)
// falls to the clamp at -127.
template <class E>
struct MxEnc {
    uint32_t packed[E::VEC / 4];
    int e;
};
template <class E>
__device__ inline MxEnc<E> mx_encode(const float (&o)[E::VEC]) {
    constexpr int VEC = E::VEC;
    constexpr int LPB = 32 / VEC;
    float amax = 0.0f;
#pragma unroll
    for (int v = 0; v < VEC; ++v) amax = __builtin_fmaxf(amax, __builtin_fabsf(o[v]));
    uint32_t bits = __float_as_uint(amax);
    bits = max(bits, dpp_u32<kQuadXor1>(bits));
    bits = max(bits, dpp_u32<kQuadXor2>(bits));
    if (LPB == 8) bits = max(bits, dpp_u32<kRowHalfMirror>(bits));
    MxEnc<E> r;
    const int e = max((int)(bits >> 23) - 135, -127);
    r.e = e;
    const float scale = __builtin_ldexpf(1.0f, e);
    const float lim = __builtin_ldexpf(448.0f, e);  // +inf at e = 127: nothing saturates there
#pragma unroll
    for (int q = 0; q < VEC / 4; ++q)
        r.packed[q] = e4m3x4_scaled(o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3], scale, lim);
    return r;
}

// MXFP8 rows: 32-element blocks along head_dim share one E8M0 scale 2^e with
// e = floor(log2(max |v|)) - 8 (clamped to [-127, 127]; -127 for an all-zero block), and each
// element is stored as the E4M3 code of v * 2^-e. Codes [num_slots][H][D] bytes, scales
// [num_slots][H][D/32] bytes (e + 127). The 32/VEC lanes of a block exchange their maxima by DPP.
template <class E>
struct MxSink {
    static constexpr int VEC = E::VEC;
    static constexpr int LPB = 32 / VEC;  // lanes per block: 4 (bf16) or 8 (fp32)
    char* codes;
    char* scales;
    int64_t row_elems;
    uint32_t code_off;
    uint32_t scale_off;
    bool scale_lane;
    int64_t num_slots;
    __device__ MxSink(const StepArgs& a, int tensor, int h, int d0, int D)
        : codes(static_cast<char*>(pick(a.cache, tensor))),
          scales(static_cast<char*>(pick(a.scales, tensor))),
          row_elems((int64_t)a.heads * D),
          code_off((uint32_t)((int64_t)h * D + d0)),
          scale_off((uint32_t)(((int64_t)h * D + d0) / 32)),
          scale_lane(d0 % 32 == 0),
          num_slots(a.num_slots) {}
    using Enc = MxEnc<E>;  // the VEC codes, 4 per word, and the block's scale exponent
    __device__ Enc encode(const float (&o)[VEC]) const { return mx_encode<E>(o); }
    __device__ void write(int64_t slot, bool active, const Enc& enc) const {
        if (!(active && slot >= 0 && slot < num_slots)) return;
        char* row = codes + uniform(slot * row_elems) + code_off;  // (offset kept scalar)
        if (VEC == 8) {
            typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
            const u32x2 w = {enc.packed[0], enc.packed[VEC / 4 - 1]};
            __builtin_nontemporal_store(w, reinterpret_cast<u32x2*>(row));
        } else {
            __builtin_nontemporal_store(enc.packed[0], reinterpret_cast<uint32_t*>(row));
        }
        if (scale_lane)
            *reinterpret_cast<uint8_t*>(scales + uniform(slot * (row_elems / 32)) + scale_off) =
                (uint8_t)(enc.e + 127);
    }
    __device__ void put(int64_t slot, bool active, const float (&o)[VEC]) const {
        write(slot, active, encode(o));
    }
};

template <class E, bool MX>
struct SinkFor { using type = PlainSink<E>; };
template <class E>
struct SinkFor<E, true> { using type = MxSink<E>; };

}  // namespace sc

#endif  // SHORTCONV_DEVICE_COMMON_H
