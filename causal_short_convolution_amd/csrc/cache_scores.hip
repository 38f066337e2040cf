// The attention weight that each cached key received (shortconv_cache_scores): with the rows' log-sum-exp
// known, the weight of a key is exp(logit - lse), and a key's sum needs nothing of the other keys.
// So every wave takes 16 SUB keys at a time, their K operands in registers, against all query rows
// of the cache head, 16 at a time from LDS; logits as in the attention (S^T = K Q^T, the lane holds
// query row lane % 16), weights summed per lane over the row tiles and over the 16 rows at the end.
// K is read once, nothing is shared between waves but the queries, and there is nothing to join.
// Measured: 64 sequences of 1-8192 MXFP8 keys, 8 heads of 128 with 4 rows each, 80 us (3.9 TB/s of
// keys); 16 sequences of 2000-8192 bf16 keys with 128 rows, 54 us (3.3 TB/s).
#include "attention_line.h"

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

// The steps of 4 wave tiles of all (sequence, cache head) lie in one line that the workgroups share
// out evenly, as in the attention, so ragged lengths fill the chip to the end: 4 workgroups on each
// CU (a fourth took spilled registers, 67 us for 58), 2 where their queries fill LDS.
// (A sequence without new tokens has its keys' scores carried over, so its keys count too.)
template <int KS>
struct KeySteps : Steps<KS, 1 << 30, 0> {
    __device__ static inline int64_t of_rows(int64_t) { return 1; }
    __device__ static inline int64_t of_sequence(const AttnArgs& a, const SeqInfo& q) {
        return a.heads * Steps<KS, 1 << 30, 0>::of_keys(q.keys);
    }
};

template <class E, bool MX, int D>
struct Shape {
    using T = Tile<E, MX, D>;
    static constexpr int ROWS = D * T::QB * kRows > 65536 ? kRows / 2 : kRows;
    static constexpr int QSTRIDE = D * T::QB + 16;
    static constexpr int WORKERS = ROWS * QSTRIDE <= 36 * 1024 ? 768 : 512;
    using S = KeySteps<16 * T::SUB * kWaves>;
};

template <class E, bool MX, int D, bool PAGE16>
__global__ void __launch_bounds__(kBlock, (Shape<E, MX, D>::WORKERS / 256)) scores_kernel(AttnArgs a) {
    using T = Tile<E, MX, D>;
    using SH = Shape<E, MX, D>;
    using S = typename SH::S;
    constexpr int SUB = T::SUB;
    constexpr int KW = 16 * SUB;
    constexpr int KS = KW * kWaves;
    constexpr uint32_t kFull = SUB == 2 ? 0xffffffffu : 0xffffu;
    constexpr int ROWS = SH::ROWS;
    constexpr int QSTRIDE = SH::QSTRIDE;
    constexpr bool AHEAD = D <= 128;  // K is loaded a step ahead
    __shared__ __attribute__((aligned(16))) char lds[ROWS * QSTRIDE];
    using SC = Scales<SUB, D>;
    __shared__ __attribute__((aligned(16))) uint32_t scale_lds[kWaves][MX ? SC::kWords : 1];
    __shared__ float norm[ROWS];  // lse in base 2; a row of -inf adds nothing
    __shared__ RunScratch run;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = uniform(tid >> 6);
    const int c = lane & 15, g = lane >> 4;
    const int eb = MX ? 1 : E::BYTES;
    const uint32_t row_bytes = (uint32_t)(a.heads * D * eb);
    const float to_log2 = a.scale * kLog2e;

    const int64_t total = find_run<S, SH::WORKERS, kBlock>(a, nullptr, run);
    const Shares<SH::WORKERS> sh(total, S::kMost);
    const int32_t me = sh.me();
    if (me >= sh.workers) return;
    int64_t at = sh.begin(me);
    const int64_t end = sh.begin(me + 1);
    Unit u;
    u.s = uniform(run.s);
    int64_t seq_first = uniform(run.first);
    SeqInfo q = seq_info(a.b, a.pg, u.s);

    while (at < end) {
        unit_at<S>(a, at, u, q, seq_first);
        const int32_t step0 = u.step_at(at), step1 = u.step_at(end);
        at = u.end();
        const int32_t keys = (int32_t)min((int64_t)q.keys, a.capacity);
        const int64_t rows = (int64_t)q.len * a.group;
        const char* kc = static_cast<const char*>(a.cache[0]) + (int64_t)u.h * D * eb;
        const char* ks = static_cast<const char*>(a.scales[0]) + u.h * (D / 32);
        const int64_t out_row = ((int64_t)u.s * a.heads + u.h) * a.capacity;

        // ---- the wave's keys of a step; with PAGE16 the lanes look up the subtiles of the next
        // kAhead steps at once
        using KT = KeyTile<SUB, PAGE16>;
        constexpr int kAhead = 64 / SUB;
        int32_t found0 = step0 - kAhead, found_row = 0, found_keys = 0;
        auto locate = [&](int32_t step) {
            KT t;
            const int32_t k0 = step * KS + wave * KW;
            t.valid = 0;
            auto find = [&](int32_t p, int32_t& exist) {
                const int32_t slot = p < keys ? slot_of(a.pg, u.s, p) : -1;
                exist = slot < 0 ? 0 : keys - p;
                return slot < 0 ? 0 : slot;
            };
            if constexpr (PAGE16) {
                if (step >= found0 + kAhead) {
                    found0 = step;
                    found_row = found_keys = 0;
                    if (step + lane / SUB < step1)
                        found_row = find(k0 + lane / SUB * KS + lane % SUB * 16, found_keys);
                }
#pragma unroll
                for (int x = 0; x < SUB; ++x) {
                    const int from = (step - found0) * SUB + x;
                    t.base[x] = __builtin_amdgcn_readlane(found_row, from);
                    const int32_t n = __builtin_amdgcn_readlane(found_keys, from);
                    t.valid |= (n >= 16 ? 0xffffu : (1u << n) - 1u) << (16 * x);
                }
                if (SUB == 2) {  // a subtile without keys reads the other one's rows
                    if (!(t.valid & 0xffffu)) t.base[0] = t.base[SUB - 1];
                    if (!(t.valid >> 16)) t.base[SUB - 1] = t.base[0];
                }
            } else {
                int32_t exist;
                t.base[0] = find(k0 + (lane & (KW - 1)), exist);
                t.valid = (uint32_t)__ballot(exist > 0) & kFull;
            }
            return t;
        };
        typename T::K kreg;
        SC sreg;
        auto load_keys = [&](const KT& t) {
            if constexpr (MX) sreg.load(ks, ks, t, row_bytes / 32, lane);
            T::load_k(kc, t, row_bytes, c, g, kreg);
        };
        auto stage = [&](int64_t r0) {  // query rows r0.. to LDS; past the last row its repeat
            constexpr int PIECES = D * T::QB / 16;
            const int n = (int)min((int64_t)ROWS, (rows - r0 + 15) / 16 * 16);
            constexpr int U = 4;  // loads in flight
            for (int x0 = tid; x0 < n * PIECES; x0 += U * kBlock) {
                uint4 y[U];
#pragma unroll
                for (int k = 0; k < U; ++k) {
                    const int x = min(x0 + k * kBlock, n * PIECES - 1);
                    const int64_t r = min(r0 + x / PIECES, rows - 1);
                    const int64_t off = (q.start + r / a.group) * a.q_stride +
                                        (int64_t)(u.h * a.group + r % a.group) * D;
                    y[k] = *reinterpret_cast<const uint4*>(static_cast<const char*>(a.q) +
                                                           off * T::QB + x % PIECES * 16);
                }
#pragma unroll
                for (int k = 0; k < U; ++k) {
                    const int x = x0 + k * kBlock;
                    if (x < n * PIECES)
                        *reinterpret_cast<uint4*>(lds + (x / PIECES) * QSTRIDE + x % PIECES * 16) =
                            y[k];
                }
            }
            for (int x = tid; x < n; x += kBlock) {
                const int64_t r = r0 + x;
                float z = -__builtin_inff();
                if (r < rows)
                    z = a.lse[(q.start + r / a.group) * a.heads * a.group + u.h * a.group +
                              r % a.group];
                norm[x] = z * kLog2e;
            }
        };
        KT tile = locate(step0);
        if (AHEAD && tile.valid) load_keys(tile);
        const bool once = rows <= ROWS;  // the queries stay in LDS
        __syncthreads();                 // the last unit is done with them
        if (once) {
            stage(0);
            __syncthreads();
        }
        for (int32_t step = step0; step < step1; ++step) {
            const int32_t k0 = step * KS + wave * KW;
            const uint32_t valid = tile.valid;
            typename T::KOp ko[SUB];
            if (valid) {
                if constexpr (!AHEAD) load_keys(tile);
                if constexpr (MX) sreg.put(scale_lds[wave], lane);
#pragma unroll
                for (int x = 0; x < SUB; ++x) T::k_operands(kreg, scale_lds[wave], x, c, g, ko[x]);
            }
            if (step + 1 < step1) {
                tile = locate(step + 1);
                if (AHEAD && tile.valid) load_keys(tile);
            }
            float sum[SUB * 4];
#pragma unroll
            for (int j = 0; j < SUB * 4; ++j) sum[j] = 0.0f;
            for (int64_t r0 = 0; r0 < rows; r0 += ROWS) {
                if (!once) {
                    __syncthreads();
                    stage(r0);
                    __syncthreads();
                }
                const int tiles = valid ? (int)min((int64_t)ROWS / 16, (rows - r0 + 15) / 16) : 0;
                for (int r = 0; r < tiles; ++r) {
                    typename T::Q qr;
                    T::load_q(lds + (r * 16 + c) * QSTRIDE, g, qr);
                    const float z = norm[r * 16 + c];
                    uint32_t bits = z == -__builtin_inff() ? 0 : valid;
                    if (k0 + KW > q.ctx && bits) {
                        const int64_t t = q.start + (r0 + r * 16 + c) / a.group;
                        bits &= mask_bits(a, t, (int32_t)(t - q.start), k0 - q.ctx);
                    }
                    float w[SUB * 4];
#pragma unroll
                    for (int x = 0; x < SUB; ++x) {
                        const f32x4 y = T::logits(ko[x], qr);
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            w[x * 4 + i] = exp2_fast(__builtin_fmaf(y[i], to_log2, -z));
                    }
                    if (__ballot(bits != kFull)) {
                        bits >>= g * 4;
#pragma unroll
                        for (int j = 0; j < SUB * 4; ++j)
                            w[j] = (bits >> ((j >> 2) * 16 + (j & 3))) & 1 ? w[j] : 0.0f;
                    }
#pragma unroll
                    for (int j = 0; j < SUB * 4; ++j) sum[j] += w[j];
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
}

template <class E, bool MX, int D>
hipError_t run(const AttnArgs& a, hipStream_t st) {
    constexpr int WORKERS = Shape<E, MX, D>::WORKERS;
    if (a.pg.shift >= 4) scores_kernel<E, MX, D, true><<<WORKERS, kBlock, 0, st>>>(a);
    else scores_kernel<E, MX, D, false><<<WORKERS, kBlock, 0, st>>>(a);
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
