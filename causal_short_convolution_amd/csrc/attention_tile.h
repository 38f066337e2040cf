// One wave's share of attention over the paged cache: 16 query rows (times R) against KW cached
// keys at a time on the matrix cores, with a running maximum and sum per row.
//
// The products are taken transposed, S^T = K Q^T and O^T = V^T P^T, on 16x16 tiles. The hardware
// leaves a 16x16 result with column n = lane % 16 and rows 4 (lane / 16) + i in register i, and
// takes its operands with the 16 side on lane % 16 and the contracted side on lane / 16. So with
// c = lane % 16, g = lane / 16:
//   S^T: the lane holds the logits of query row c for keys 4g + i (each 16-key subtile);
//   P^T: exactly these, as they lie, are the second operand of O^T, if the contraction runs over
//        the keys in the order (subtile, i) within lane group g: no exchange between lanes;
//   O^T: the lane holds channels of query row c again, so the running maximum, the sum and the
//        rescaling of a row are per-lane values.
// A contraction may run in any order, so K is loaded 16 bytes per lane straight into its operand
// (key c, channels by g), and V 16 bytes per lane by rows (keys 4g + i, channels by c), transposed
// in registers by byte permutes. Neither goes through LDS; of an MXFP8 tile only the scales do.
#ifndef SHORTCONV_ATTENTION_TILE_H
#define SHORTCONV_ATTENTION_TILE_H

#include "cache_device.h"

namespace sc {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

__device__ inline float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ inline float log2_fast(float x) { return __builtin_amdgcn_logf(x); }

// Logits are q . k times a factor c > 0 in base 2 (a negative scale turns the queries' signs instead,
// a scale of 0 clears them), so a row's running maximum is kept of the products alone and a
// weight is one fused multiply-add and one exp2, 0 for a masked -inf. The reference value of a row, c
// times its maximum; 0 while it has none.
__device__ inline float logit_factor(float scale) {
    return scale == 0.0f ? 1.0f : __builtin_fabsf(scale) * kLog2e;
}
__device__ inline float row_base(float top, float c) {
    return top == -__builtin_inff() ? 0.0f : top * c;
}
// The maximum in base-2 logits, for joining parts.
__device__ inline float row_top(float top, float c) {
    return top == -__builtin_inff() ? top : top * c;
}
// A 16-byte piece of queries under the sign of the scale.
template <class E>
__device__ inline uint4 signed_by(uint4 x, float scale) {
    const uint32_t turn = scale >= 0.0f ? 0u : E::BYTES == 2 ? 0x80008000u : 0x80000000u;
    const uint32_t keep = scale == 0.0f ? 0u : 0xffffffffu;
    return make_uint4((x.x ^ turn) & keep, (x.y ^ turn) & keep, (x.z ^ turn) & keep,
                      (x.w ^ turn) & keep);
}

// Maximum and sum over the four lanes that hold one query row (lanes c, c + 16, c + 32, c + 48).
__device__ inline float row_max(float v) {
    uint32_t u = __float_as_uint(v);
    auto p = __builtin_amdgcn_permlane16_swap(u, u, false, false);
    v = __builtin_fmaxf(__uint_as_float(p[0]), __uint_as_float(p[1]));
    u = __float_as_uint(v);
    p = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    return __builtin_fmaxf(__uint_as_float(p[0]), __uint_as_float(p[1]));
}
__device__ inline float row_sum(float v) {
    uint32_t u = __float_as_uint(v);
    auto p = __builtin_amdgcn_permlane16_swap(u, u, false, false);
    v = __uint_as_float(p[0]) + __uint_as_float(p[1]);
    u = __float_as_uint(v);
    p = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    return __uint_as_float(p[0]) + __uint_as_float(p[1]);
}

// An E8M0 byte as the float 2^(e - 127).
__device__ inline float e8m0(uint32_t e) { return __uint_as_float(e ? e << 23 : 0x00400000u); }

// One element of a cache row in fp32 (at: elements from the start of the cache).
template <class E, bool MX>
__device__ inline float cache_element(const void* cache, const void* scales, int64_t at) {
    if constexpr (MX) {
        const uint32_t code = static_cast<const uint8_t*>(cache)[at];
        const float e = e8m0(static_cast<const uint8_t*>(scales)[at >> 5]);
        const f32x2 w = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(code, e, false);
        return w[0];
    } else if constexpr (E::BYTES == 4) {
        return static_cast<const float*>(cache)[at];
    } else {
        return __uint_as_float((uint32_t)static_cast<const uint16_t*>(cache)[at] << 16);
    }
}

// Where one wave's keys lie: with PAGE16 (pages of at least 16 rows) each 16-key subtile is a run
// of rows starting at the wave-uniform `base`; otherwise lane l knows the row of key l % KW. Bit k
// of `valid` says that key k exists; a key that does not has row 0, which exists if any key does.
template <int SUB, bool PAGE16>
struct KeyTile {
    uint32_t valid;
    int32_t base[PAGE16 ? SUB : 1];
};

// The address of key `key` (0 <= key < 16 SUB; key / 16 == sub) of a tile, in bytes.
template <int SUB, bool PAGE16>
__device__ inline const char* key_row(const char* cache, const KeyTile<SUB, PAGE16>& t, int sub,
                                      int key, uint32_t row_bytes) {
    if constexpr (PAGE16) {
        return cache + uniform((int64_t)t.base[sub] * row_bytes) + (uint32_t)(key & 15) * row_bytes;
    } else {
        return cache + (int64_t)__shfl(t.base[0], key) * row_bytes;
    }
}

// The scale bytes of one tile's keys, D / 32 for each row of K and of V: lane l loads those of key
// l % KW, of K (l < 32) or V, and leaves them in the wave's LDS as words [K, V][D / 128][KW], where
// an operand finds the ones of its keys. (Loaded by each lane for its own operands they were 10 of a
// step's 22 load instructions, and the address units' time bounded the step.)
template <int SUB, int D>
struct Scales {
    static constexpr int KW = 16 * SUB, NW = (D + 127) / 128;
    static constexpr int kWords = 2 * NW * KW;
    uint32_t w[NW];

    template <bool PG>
    __device__ inline void load(const char* k, const char* v, const KeyTile<SUB, PG>& t,
                                uint32_t row, int lane) {
        int32_t r = t.base[0];
        if constexpr (PG) r = (SUB == 2 && (lane & 16) ? t.base[SUB - 1] : r) + (lane & 15);
        const char* p = (lane < 32 ? k : v) + (int64_t)r * row;
        if constexpr (D == 64) {
            w[0] = *reinterpret_cast<const uint16_t*>(p);
        } else {
#pragma unroll
            for (int j = 0; j < NW; ++j) w[j] = *reinterpret_cast<const uint32_t*>(p + 4 * j);
        }
    }
    __device__ inline void put(uint32_t* lds, int lane) const {
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
        for (int j = 0; j < NW; ++j) lds[((lane >> 5) * NW + j) * KW + (lane & (KW - 1))] = w[j];
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    }
    // Word j of K's key, and of V's keys 4 n ..
    __device__ static inline uint32_t of_key(const uint32_t* lds, int j, int key) {
        return lds[j * KW + key];
    }
    __device__ static inline uint4 of_values(const uint32_t* lds, int j, int n) {
        return *reinterpret_cast<const uint4*>(lds + (NW + j) * KW + n * 4);
    }
};

template <class E, bool MX, int D>
struct Tile;

// ------------------------------------------------------------------------------------------------
// bf16 queries: 16x16x32 products of bf16 operands, 32 keys at a time. MXFP8 rows are widened to
// bf16 in registers, which is exact (a code has 4 significant bits, its scale is a power of two).
// ------------------------------------------------------------------------------------------------
template <bool MX, int D>
struct Tile<BF16, MX, D> {
    static constexpr int SUB = 2;
    static constexpr int NF = D / 32;               // K operands per subtile
    static constexpr int CH = D / 16 < 8 ? D / 16 : 8;  // V channels per lane and piece
    static constexpr int NU = D / 16 / CH;          // pieces of V
    static constexpr int NT = D / 16;               // output tiles
    static constexpr int QB = 2;                    // bytes of a query element
    static constexpr int KN = MX ? NF / 2 : NF;

    struct K {
        uint4 x[SUB][KN];
    };
    struct V {
        uint32_t x[SUB * 4][NU][MX ? CH / 4 : CH / 2];
    };
    using Q = bf16x8[NF];

    // First channel of query operand f in lane group g.
    __device__ static inline int q_channel(int f, int g) {
        return MX ? (f >> 1) * 64 + g * 16 + (f & 1) * 8 : f * 32 + g * 8;
    }
    __device__ static inline void load_q(const char* row, int g, Q& q) {
#pragma unroll
        for (int f = 0; f < NF; ++f)
            q[f] = *reinterpret_cast<const bf16x8*>(row + q_channel(f, g) * QB);
    }

    template <bool PG>
    __device__ static inline void load_k(const char* cache, const KeyTile<SUB, PG>& t,
                                         uint32_t row, int c, int g, K& k) {
#pragma unroll
        for (int s = 0; s < SUB; ++s) {
            const char* r = key_row(cache, t, s, s * 16 + c, row) + g * 16;
#pragma unroll
            for (int f = 0; f < KN; ++f) k.x[s][f] = *reinterpret_cast<const uint4*>(r + f * 64);
        }
    }
    template <bool PG>
    __device__ static inline void load_v(const char* cache, const KeyTile<SUB, PG>& t,
                                         uint32_t row, int c, int g, V& v) {
#pragma unroll
        for (int j = 0; j < SUB * 4; ++j) {
            const int key = (j >> 2) * 16 + g * 4 + (j & 3);
            const char* r = key_row(cache, t, j >> 2, key, row);
#pragma unroll
            for (int u = 0; u < NU; ++u) {
                if constexpr (MX) {
                    const char* p = r + u * 16 * CH + c * CH;
                    if constexpr (CH == 8) {
                        const uint2 w = *reinterpret_cast<const uint2*>(p);
                        v.x[j][u][0] = w.x;
                        v.x[j][u][1] = w.y;
                    } else {
                        v.x[j][u][0] = *reinterpret_cast<const uint32_t*>(p);
                    }
                } else {
                    const char* p = r + (u * 16 * CH + c * CH) * 2;
                    if constexpr (CH == 8) {
                        const uint4 w = *reinterpret_cast<const uint4*>(p);
                        v.x[j][u][0] = w.x;
                        v.x[j][u][1] = w.y;
                        v.x[j][u][2] = w.z;
                        v.x[j][u][3] = w.w;
                    } else {
                        const uint2 w = *reinterpret_cast<const uint2*>(p);
                        v.x[j][u][0] = w.x;
                        v.x[j][u][1] = w.y;
                    }
                }
            }
        }
    }

    __device__ static inline uint32_t widen2(uint32_t w, float scale, bool hi) {
        return hi ? __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(
                                                     w, scale, true))
                  : __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(
                                                     w, scale, false));
    }
    // The K operands of subtile s; `sc`: the tile's scales in LDS.
    __device__ static inline void k_operands(const K& k, const uint32_t* sc, int s, int c, int g,
                                             bf16x8 (&a)[NF]) {
        uint32_t words[MX ? Scales<SUB, D>::NW : 1];
        if constexpr (MX) {
#pragma unroll
            for (int j = 0; j < Scales<SUB, D>::NW; ++j)
                words[j] = Scales<SUB, D>::of_key(sc, j, s * 16 + c);
        }
#pragma unroll
        for (int f = 0; f < KN; ++f) {
            if constexpr (MX) {
                // 16 channels f * 64 + 16 g ..: scale byte 2 f + g / 2 of the row
                const float e = e8m0((words[f / 2] >> ((f & 1) * 16 + (g >> 1) * 8)) & 255u);
                const uint32_t w[4] = {k.x[s][f].x, k.x[s][f].y, k.x[s][f].z, k.x[s][f].w};
#pragma unroll
                for (int p = 0; p < 2; ++p) {
                    const uint4 o = make_uint4(widen2(w[2 * p], e, false), widen2(w[2 * p], e, true),
                                               widen2(w[2 * p + 1], e, false),
                                               widen2(w[2 * p + 1], e, true));
                    a[2 * f + p] = __builtin_bit_cast(bf16x8, o);
                }
            } else {
                a[f] = __builtin_bit_cast(bf16x8, k.x[s][f]);
            }
        }
    }
    __device__ static inline f32x4 logits(const bf16x8 (&a)[NF], const Q& q) {
        f32x4 x = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int f = 0; f < NF; ++f)
            x = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[f], q[f], x, 0, 0, 0);
        return x;
    }
    using KOp = bf16x8[NF];

    // V as bf16 pairs [key][piece][channel pair].
    struct VOp {
        uint32_t w[SUB * 4][NU][CH / 2];
    };
    __device__ static inline void v_operands(const V& v, const uint32_t* sc, int c, int g, VOp& o) {
        uint32_t words[SUB * 4][MX ? Scales<SUB, D>::NW : 1];
        if constexpr (MX) {
#pragma unroll
            for (int s = 0; s < SUB; ++s)
#pragma unroll
                for (int k = 0; k < Scales<SUB, D>::NW; ++k) {
                    const uint4 w = Scales<SUB, D>::of_values(sc, k, s * 4 + g);
                    words[s * 4][k] = w.x;
                    words[s * 4 + 1][k] = w.y;
                    words[s * 4 + 2][k] = w.z;
                    words[s * 4 + 3][k] = w.w;
                }
        }
#pragma unroll
        for (int j = 0; j < SUB * 4; ++j)
#pragma unroll
            for (int u = 0; u < NU; ++u) {
                if constexpr (MX) {
                    // channels u * 16 CH + c * CH ..: at CH 8 a word of scales per piece
                    const float e = e8m0((words[j][u] >> ((CH == 8 ? c >> 2 : c >> 3) * 8)) & 255u);
#pragma unroll
                    for (int q = 0; q < CH / 4; ++q) {
                        o.w[j][u][2 * q] = widen2(v.x[j][u][q], e, false);
                        o.w[j][u][2 * q + 1] = widen2(v.x[j][u][q], e, true);
                    }
                } else {
#pragma unroll
                    for (int q = 0; q < CH / 2; ++q) o.w[j][u][q] = v.x[j][u][q];
                }
            }
    }
    // Clears the rows of keys that do not exist (their memory holds anything).
    __device__ static inline void clear(VOp& o, uint32_t valid, int g) {
#pragma unroll
        for (int j = 0; j < SUB * 4; ++j) {
            const bool ok = (valid >> ((j >> 2) * 16 + g * 4 + (j & 3))) & 1;
#pragma unroll
            for (int u = 0; u < NU; ++u)
#pragma unroll
                for (int q = 0; q < CH / 2; ++q) o.w[j][u][q] = ok ? o.w[j][u][q] : 0u;
        }
    }
    // Replaces infinities and NaN by zeros; true if this lane held any.
    __device__ static inline bool cleanse(VOp& o) {
        bool any = false;
#pragma unroll
        for (int j = 0; j < SUB * 4; ++j)
#pragma unroll
            for (int u = 0; u < NU; ++u)
#pragma unroll
                for (int q = 0; q < CH / 2; ++q) {
                    uint32_t& w = o.w[j][u][q];
                    const bool lo = (w & 0x7f80u) == 0x7f80u;
                    const bool hi = (w & 0x7f800000u) == 0x7f800000u;
                    any |= lo || hi;
                    w &= (lo ? 0xffff0000u : 0xffffffffu) & (hi ? 0x0000ffffu : 0xffffffffu);
                }
        return any;
    }
    // acc += V^T P^T for one row tile; p in the order (subtile, i).
    __device__ static inline void values(const VOp& o, const float (&p)[SUB * 4],
                                         f32x4 (&acc)[NT]) {
        const uint4 pw = make_uint4(BF16::pack2(p[0], p[1]), BF16::pack2(p[2], p[3]),
                                    BF16::pack2(p[4], p[5]), BF16::pack2(p[6], p[7]));
        const bf16x8 b = __builtin_bit_cast(bf16x8, pw);
#pragma unroll
        for (int u = 0; u < NU; ++u)
#pragma unroll
            for (int e = 0; e < CH; ++e) {
                const uint32_t sel = (e & 1) ? 0x07060302u : 0x05040100u;
                uint32_t a[4];
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    a[j] = __builtin_amdgcn_perm(o.w[2 * j + 1][u][e / 2], o.w[2 * j][u][e / 2], sel);
                const bf16x8 av = __builtin_bit_cast(bf16x8, make_uint4(a[0], a[1], a[2], a[3]));
                acc[u * CH + e] =
                    __builtin_amdgcn_mfma_f32_16x16x32_bf16(av, b, acc[u * CH + e], 0, 0, 0);
            }
    }
};

// ------------------------------------------------------------------------------------------------
// fp32 queries: 16x16x4 products of fp32 operands, 16 keys at a time; nothing is rounded.
// ------------------------------------------------------------------------------------------------
template <bool MX, int D>
struct Tile<F32, MX, D> {
    static constexpr int SUB = 1;
    static constexpr int NF = D / 16;
    static constexpr int CH = 4;
    static constexpr int NU = D / 64;
    static constexpr int NT = D / 16;
    static constexpr int QB = 4;
    static constexpr int KN = MX ? D / 64 : NF;

    struct K {
        uint4 x[KN];
    };
    struct V {
        uint32_t x[4][NU][MX ? 1 : 4];
    };
    using Q = f32x4[NF];

    __device__ static inline int q_channel(int f, int g) {
        return MX ? (f >> 2) * 64 + g * 16 + (f & 3) * 4 : f * 16 + g * 4;
    }
    __device__ static inline void load_q(const char* row, int g, Q& q) {
#pragma unroll
        for (int f = 0; f < NF; ++f)
            q[f] = *reinterpret_cast<const f32x4*>(row + q_channel(f, g) * QB);
    }
    template <bool PG>
    __device__ static inline void load_k(const char* cache, const KeyTile<SUB, PG>& t,
                                         uint32_t row, int c, int g, K& k) {
        const char* r = key_row(cache, t, 0, c, row) + g * 16;
#pragma unroll
        for (int f = 0; f < KN; ++f) k.x[f] = *reinterpret_cast<const uint4*>(r + f * 64);
    }
    template <bool PG>
    __device__ static inline void load_v(const char* cache, const KeyTile<SUB, PG>& t,
                                         uint32_t row, int c, int g, V& v) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const char* r = key_row(cache, t, 0, g * 4 + j, row);
#pragma unroll
            for (int u = 0; u < NU; ++u) {
                if constexpr (MX) {
                    v.x[j][u][0] = *reinterpret_cast<const uint32_t*>(r + u * 64 + c * 4);
                } else {
                    const uint4 w = *reinterpret_cast<const uint4*>(r + (u * 64 + c * 4) * 4);
                    v.x[j][u][0] = w.x;
                    v.x[j][u][1] = w.y;
                    v.x[j][u][2] = w.z;
                    v.x[j][u][3] = w.w;
                }
            }
        }
    }
    using KOp = f32x4[NF];
    __device__ static inline void k_operands(const K& k, const uint32_t* sc, int, int c, int g,
                                             KOp& a) {
        uint32_t words[MX ? Scales<SUB, D>::NW : 1];
        if constexpr (MX) {
#pragma unroll
            for (int j = 0; j < Scales<SUB, D>::NW; ++j) words[j] = Scales<SUB, D>::of_key(sc, j, c);
        }
#pragma unroll
        for (int f = 0; f < KN; ++f) {
            if constexpr (MX) {
                const float e = e8m0((words[f / 2] >> ((f & 1) * 16 + (g >> 1) * 8)) & 255u);
                const uint32_t w[4] = {k.x[f].x, k.x[f].y, k.x[f].z, k.x[f].w};
#pragma unroll
                for (int p = 0; p < 4; ++p) {
                    const f32x2 lo = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w[p], e, false);
                    const f32x2 hi = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w[p], e, true);
                    a[4 * f + p] = f32x4{lo[0], lo[1], hi[0], hi[1]};
                }
            } else {
                a[f] = __builtin_bit_cast(f32x4, k.x[f]);
            }
        }
    }
    __device__ static inline f32x4 logits(const KOp& a, const Q& q) {
        f32x4 x = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int f = 0; f < NF; ++f)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                x = __builtin_amdgcn_mfma_f32_16x16x4f32(a[f][e], q[f][e], x, 0, 0, 0);
        return x;
    }
    struct VOp {
        float w[4][NU][4];
    };
    __device__ static inline void v_operands(const V& v, const uint32_t* sc, int c, int g, VOp& o) {
        uint32_t words[4][MX ? Scales<SUB, D>::NW : 1];
        if constexpr (MX) {
#pragma unroll
            for (int k = 0; k < Scales<SUB, D>::NW; ++k) {
                const uint4 w = Scales<SUB, D>::of_values(sc, k, g);
                words[0][k] = w.x;
                words[1][k] = w.y;
                words[2][k] = w.z;
                words[3][k] = w.w;
            }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int u = 0; u < NU; ++u) {
                if constexpr (MX) {
                    // channels u * 64 + c * 4 ..: scale byte 2 u + c / 8 of the row
                    const float e = e8m0((words[j][u / 2] >> ((u & 1) * 16 + (c >> 3) * 8)) & 255u);
                    const f32x2 lo = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(v.x[j][u][0], e, false);
                    const f32x2 hi = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(v.x[j][u][0], e, true);
                    o.w[j][u][0] = lo[0];
                    o.w[j][u][1] = lo[1];
                    o.w[j][u][2] = hi[0];
                    o.w[j][u][3] = hi[1];
                } else {
#pragma unroll
                    for (int q = 0; q < 4; ++q) o.w[j][u][q] = __uint_as_float(v.x[j][u][q]);
                }
            }
    }
    __device__ static inline void clear(VOp& o, uint32_t valid, int g) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const bool ok = (valid >> (g * 4 + j)) & 1;
#pragma unroll
            for (int u = 0; u < NU; ++u)
#pragma unroll
                for (int q = 0; q < 4; ++q) o.w[j][u][q] = ok ? o.w[j][u][q] : 0.0f;
        }
    }
    __device__ static inline bool cleanse(VOp& o) {
        bool any = false;
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int u = 0; u < NU; ++u)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const bool big = (__float_as_uint(o.w[j][u][q]) & 0x7f800000u) == 0x7f800000u;
                    any |= big;
                    o.w[j][u][q] = big ? 0.0f : o.w[j][u][q];
                }
        return any;
    }
    __device__ static inline void values(const VOp& o, const float (&p)[4], f32x4 (&acc)[NT]) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int u = 0; u < NU; ++u)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    acc[u * 4 + e] = __builtin_amdgcn_mfma_f32_16x16x4f32(o.w[j][u][e], p[j],
                                                                         acc[u * 4 + e], 0, 0, 0);
    }
};

// 32 mask bits of a row from bit `at` on; bits before 0 are the cached keys (ones).
__device__ inline uint32_t mask_bits(const AttnArgs& a, int64_t t, int32_t i, int32_t at) {
    if (at <= -32) return 0xffffffffu;
    if (a.mask == nullptr) {
        const int32_t n = i - at + 1;  // new tokens 0..i, and the cached keys before them
        return n >= 32 ? 0xffffffffu : n <= 0 ? 0u : (1u << n) - 1u;
    }
    const uint64_t* m = reinterpret_cast<const uint64_t*>(a.mask) + t * a.words;
    if (at < 0) {
        const uint64_t w = a.words > 0 ? m[0] : 0;
        return (uint32_t)(w << -at) | ((1u << -at) - 1u);
    }
    const int32_t j = at >> 6, sh = at & 63;
    const uint64_t lo = j < a.words ? m[j] : 0;
    const uint64_t hi = j + 1 < a.words ? m[j + 1] : 0;
    return (uint32_t)(sh ? (lo >> sh) | (hi << (64 - sh)) : lo);
}

}  // namespace sc

#endif  // SHORTCONV_ATTENTION_TILE_H
