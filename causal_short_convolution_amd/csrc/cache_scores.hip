// The attention weight that each cached key received (shortconv_cache_scores): with the rows' log-sum-exp
// known, the weight of a key is exp(logit - lse), and a key's sum needs nothing of the other keys.
// So every wave takes 16 SUB keys at a time, their K operands in registers, against all query rows
// of the cache head, 16 at a time from LDS; logits as in the attention (S^T = K Q^T, the lane holds
// query row lane % 16), weights summed per lane over the row tiles and over the 16 rows at the end.
// K is read once, nothing is shared between waves but the queries, and there is nothing to join.
#include "attention_tile.h"

namespace sc {
namespace {

constexpr int kBlock = 256;
constexpr int kWaves = 4;
constexpr int kRows = 128;  // query rows in LDS at a time

// Sum over the 16 lanes of a row, in all of them.
__device__ inline float sum16(float v) {
    v += dpp<kQuadXor1>(v);
    v += dpp<kQuadXor2>(v);
    v += dpp<kRowHalfMirror>(v);
    v += dpp<kRowMirror>(v);
    return v;
}

// Workgroup: steps blockIdx.x, + gridDim.x, .. of 4 wave tiles of cache head blockIdx.y of sequence
// blockIdx.z.
template <class E, bool MX, int D, bool PAGE16>
__global__ void __launch_bounds__(kBlock) scores_kernel(AttnArgs a) {
    using T = Tile<E, MX, D>;
    constexpr int SUB = T::SUB;
    constexpr int KW = 16 * SUB;
    constexpr uint32_t kFull = SUB == 2 ? 0xffffffffu : 0xffffu;
    constexpr int ROWS = D * T::QB * kRows > 65536 ? kRows / 2 : kRows;
    constexpr int QSTRIDE = D * T::QB + 16;
    __shared__ __attribute__((aligned(16))) char lds[ROWS * QSTRIDE];
    using SC = Scales<SUB, D>;
    __shared__ __attribute__((aligned(16))) uint32_t scale_lds[kWaves][MX ? SC::kWords : 1];
    __shared__ float norm[ROWS];  // lse in base 2; a row of -inf adds nothing
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = uniform(tid >> 6);
    const int c = lane & 15, g = lane >> 4;
    const int h = blockIdx.y, s = blockIdx.z;
    const SeqInfo q = seq_info(a.b, a.pg, s);
    const int32_t keys = (int32_t)min((int64_t)q.keys, a.capacity);
    if ((int64_t)blockIdx.x * KW * kWaves >= keys) return;
    const int64_t rows = (int64_t)q.len * a.group;
    const int eb = MX ? 1 : E::BYTES;
    const uint32_t row_bytes = (uint32_t)(a.heads * D * eb);
    const char* kc = static_cast<const char*>(a.cache[0]) + (int64_t)h * D * eb;
    const char* ks = static_cast<const char*>(a.scales[0]) + h * (D / 32);
    const int64_t out_row = ((int64_t)s * a.heads + h) * a.capacity;
    const float to_log2 = a.scale * kLog2e;

    auto stage = [&](int64_t r0) {  // query rows r0.. to LDS; past the last row its repeat
        constexpr int PIECES = D * T::QB / 16;
        const int n = (int)min((int64_t)ROWS, (rows - r0 + 15) / 16 * 16);
        for (int x = tid; x < n * PIECES; x += kBlock) {
            const int64_t r = min(r0 + x / PIECES, rows - 1);
            const int64_t off = (q.start + r / a.group) * a.q_stride +
                                (int64_t)(h * a.group + r % a.group) * D;
            *reinterpret_cast<uint4*>(lds + (x / PIECES) * QSTRIDE + x % PIECES * 16) =
                *reinterpret_cast<const uint4*>(static_cast<const char*>(a.q) + off * T::QB +
                                                x % PIECES * 16);
        }
        for (int x = tid; x < n; x += kBlock) {
            const int64_t r = r0 + x;
            float z = -__builtin_inff();
            if (r < rows)
                z = a.lse[(q.start + r / a.group) * a.heads * a.group + h * a.group + r % a.group];
            norm[x] = z * kLog2e;
        }
    };
    const bool once = rows <= ROWS;  // the queries stay in LDS
    if (once) {
        stage(0);
        __syncthreads();
    }
    for (int32_t k0 = (int32_t)blockIdx.x * KW * kWaves + wave * KW;
         k0 - wave * KW < keys; k0 += gridDim.x * KW * kWaves) {
        KeyTile<SUB, PAGE16> tile;
        tile.valid = 0;
        if constexpr (PAGE16) {
#pragma unroll
            for (int x = 0; x < SUB; ++x) {
                const int32_t p = k0 + x * 16;
                const int32_t slot = uniform(p < keys ? slot_of(a.pg, s, p) : -1);
                tile.base[x] = slot < 0 ? 0 : slot;
                const int32_t n = slot < 0 ? 0 : keys - p;
                tile.valid |= (n >= 16 ? 0xffffu : (1u << n) - 1u) << (16 * x);
            }
            if (SUB == 2) {
                if (!(tile.valid & 0xffffu)) tile.base[0] = tile.base[SUB - 1];
                if (!(tile.valid >> 16)) tile.base[SUB - 1] = tile.base[0];
            }
        } else {
            const int32_t p = k0 + (lane & (KW - 1));
            const int32_t slot = p < keys ? slot_of(a.pg, s, p) : -1;
            tile.base[0] = slot < 0 ? 0 : slot;
            tile.valid = (uint32_t)__ballot(slot >= 0) & kFull;
        }
        float sum[SUB * 4];
#pragma unroll
        for (int j = 0; j < SUB * 4; ++j) sum[j] = 0.0f;
        typename T::KOp ko[SUB];
        if (tile.valid) {
            typename T::K kreg;
            if constexpr (MX) {
                SC sreg;
                sreg.load(ks, ks, tile, row_bytes / 32, lane);
                T::load_k(kc, tile, row_bytes, c, g, kreg);
                sreg.put(scale_lds[wave], lane);
            } else {
                T::load_k(kc, tile, row_bytes, c, g, kreg);
            }
#pragma unroll
            for (int x = 0; x < SUB; ++x) T::k_operands(kreg, scale_lds[wave], x, c, g, ko[x]);
        }
        for (int64_t r0 = 0; r0 < rows; r0 += ROWS) {
            if (!once) {
                __syncthreads();
                stage(r0);
                __syncthreads();
            }
            const int tiles = tile.valid ? (int)min((int64_t)ROWS / 16, (rows - r0 + 15) / 16) : 0;
            for (int r = 0; r < tiles; ++r) {
                typename T::Q qr;
                T::load_q(lds + (r * 16 + c) * QSTRIDE, g, qr);
                const float z = norm[r * 16 + c];
                uint32_t bits = z == -__builtin_inff() ? 0 : tile.valid;
                if (k0 + KW > q.ctx && bits) {
                    const int64_t t = q.start + (r0 + r * 16 + c) / a.group;
                    bits &= mask_bits(a, t, (int32_t)(t - q.start), k0 - q.ctx);
                }
                bits >>= g * 4;
#pragma unroll
                for (int x = 0; x < SUB; ++x) {
                    const f32x4 y = T::logits(ko[x], qr);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float w = exp2_fast(__builtin_fmaf(y[i], to_log2, -z));
                        sum[x * 4 + i] += (bits >> (x * 16 + i)) & 1 ? w : 0.0f;
                    }
                }
            }
        }
        // every lane of a group of 16 gets the sums; lane c < 4 SUB writes key (c / 4, 4 g + c % 4)
        float mine = 0.0f;
#pragma unroll
        for (int j = 0; j < SUB * 4; ++j) {
            const float v = sum16(sum[j]);
            mine = c == j ? v : mine;
        }
        const int32_t p = k0 + (c >> 2) * 16 + g * 4 + (c & 3);
        if (c < SUB * 4 && p < keys) {
            if (a.scores_in != nullptr && p < q.ctx) mine += a.scores_in[out_row + p];
            a.scores_out[out_row + p] = mine;
        }
    }
}

template <class E, bool MX, int D>
hipError_t run(const AttnArgs& a, hipStream_t st) {
    constexpr int KS = 16 * Tile<E, MX, D>::SUB * kWaves;
    const int64_t keys = (int64_t)a.pg.max_blocks << a.pg.shift;
    const int64_t most = ((keys < a.capacity ? keys : a.capacity) + KS - 1) / KS;
    // About 8 workgroups per CU, each with several steps for one staging of its queries.
    const int64_t share = 2048 / ((int64_t)a.heads * a.b.num_seqs) + 1;
    const dim3 grid((uint32_t)(share < most ? share : most), a.heads, a.b.num_seqs);
    if (a.pg.shift >= 4) scores_kernel<E, MX, D, true><<<grid, kBlock, 0, st>>>(a);
    else scores_kernel<E, MX, D, false><<<grid, kBlock, 0, st>>>(a);
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
    if (dtype == 0) return mx ? by_dim<F32, true>(a, D, st) : by_dim<F32, false>(a, D, st);
    return mx ? by_dim<BF16, true>(a, D, st) : by_dim<BF16, false>(a, D, st);
}

}  // namespace sc
