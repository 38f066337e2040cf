// Attention over the paged cache: shortconv_tree_attention (the new tokens of each sequence, a tree
// or one token, over all its keys) and shortconv_block_attention (each new token over the pages
// selected for it).
//
// The work is cut into units: a cache head of a sequence (of a token, for selected pages) with the
// query rows that read it, up to 16 R of them, R = 1 or 2. A unit's keys are cut into steps of
// 4 wave tiles. All steps of all units lie in one line that the workgroups share out evenly, each
// taking a run of consecutive steps, so one long sequence among short ones, or few units with many
// keys, still fill the chip; the lengths are read on the device, so a captured launch follows them.
// In a step the 4 waves take different keys, each with its own running maximum and sum; at the end
// of the unit they meet in LDS. A unit that ends inside one workgroup's run is written at once;
// one that crosses workgroups leaves its unnormalized sums in the workspace, and a second launch
// joins them (a fixed order: the same inputs give the same bits).
//
// Few rows leave it bound by the cache's bytes, so K and V go straight to registers, a step ahead: 64
// pages of 64 keys for 32 tokens and 8 heads of 128, bf16, 104 us, 5.2 TB/s. MXFP8 rows take about
// twice the instructions to widen: 32 pages for each of 512 tokens (2.2 GB of rows, mostly from
// L2), 254 us.
#include "attention_line.h"

namespace sc {
namespace {

constexpr int kBlock = 256;
constexpr int kWaves = 4;

template <class E, bool MX, int D, int R, bool SPARSE, bool PAGE16>
__global__ void __launch_bounds__(kBlock, 2) attention_kernel(AttnArgs a) {
    using T = Tile<E, MX, D>;
    constexpr int WORKERS = kWorkers;
    constexpr int M = 16 * R;
    constexpr int SUB = T::SUB;
    constexpr int KW = 16 * SUB;      // keys per wave and step
    constexpr int KS = KW * kWaves;   // keys per step
    using S = Steps<KS, M, 0>;
    constexpr uint32_t kFull = SUB == 2 ? 0xffffffffu : 0xffffu;
    constexpr int QSTRIDE = D * T::QB + 16;  // query rows in LDS, staggered over the banks
    constexpr bool QREG = R == 1 && D <= 128;  // query operands stay in registers
    constexpr bool AHEAD = R == 1 && D <= 128; // keys are loaded a step ahead
    constexpr int OSTRIDE = D + 4;           // output rows in LDS (floats)
    constexpr int kLds = 2 * M * OSTRIDE * 4 > M * QSTRIDE ? 2 * M * OSTRIDE * 4 : M * QSTRIDE;
    __shared__ __attribute__((aligned(16))) char lds[kLds];
    __shared__ float stat[kWaves][2][M];
    using SC = Scales<SUB, D>;
    __shared__ __attribute__((aligned(16))) uint32_t scale_lds[kWaves][MX ? SC::kWords : 1];
    __shared__ RunScratch run;
    __shared__ int32_t left_out_any;

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = uniform(tid >> 6);
    const int c = lane & 15, g = lane >> 4;
    const int eb = MX ? 1 : E::BYTES;
    const uint32_t row_bytes = (uint32_t)(a.heads * D * eb);
    char* ws = static_cast<char*>(a.ws);

    // ---- this worker's run of steps, and the unit it begins in
    int64_t total, at, end;
    Unit u;
    if constexpr (SPARSE) {
        u.steps = S::of_pages(a);
        total = a.b.tokens * a.heads * S::group_tiles(a) * u.steps;
    } else {
        total = find_run<S, WORKERS, kBlock>(a, reinterpret_cast<int64_t*>(ws), run);
    }
    const Shares<WORKERS> sh(total, S::kMost);
    const int32_t me = sh.me();
    if (me >= sh.workers) return;
    at = sh.begin(me);
    end = sh.begin(me + 1);
    SeqInfo q;
    int64_t seq_first = 0, known = -1;  // selected pages: the token that q is of
    if constexpr (!SPARSE) {
        u.s = uniform(run.s);
        seq_first = uniform(run.first);
        q = seq_info(a.b, a.pg, u.s);
    }

    while (at < end) {
        // ---- the unit that step `at` belongs to
        int32_t last = 0;  // selected pages: the token's own position
        bool real = true;
        if constexpr (SPARSE) {
            const int32_t tiles = S::group_tiles(a);
            const int64_t n = at / u.steps;
            const int64_t th = n / tiles;
            u.h = (int32_t)(th % a.heads);
            u.tok = th / a.heads;
            S::place(u, a.group, n % tiles * M, th * tiles * u.steps);
            if (u.tok != known) {
                u.s = seq_of_token(a.b, u.tok);
                q = seq_info(a.b, a.pg, u.s);
                known = u.tok;
            }
            const int64_t i = u.tok - q.start;
            real = i >= 0 && i < q.len;  // a token behind the last sequence has no output
            last = (int32_t)min((int64_t)(a.pg.max_blocks << a.pg.shift) - 1, (int64_t)q.ctx + i);
        } else {
            unit_at<S>(a, at, u, q, seq_first);
        }
        const int64_t tok = u.tok;  // the first token of its rows
        const int32_t step0 = u.step_at(at), step1 = u.step_at(end);
        at = u.end();
        if (!real) continue;

        // Query row r of the unit: token and query head (rows past the last repeat it).
        auto row_token = [&](int r) {
            const int32_t x = u.row0 + (r < u.rows ? r : u.rows - 1);
            return SPARSE ? tok : tok + x / a.group;
        };
        auto row_head = [&](int r) {
            const int32_t x = u.row0 + (r < u.rows ? r : u.rows - 1);
            return u.h * a.group + (SPARSE ? x : x % a.group);
        };
        // ---- the wave's keys of one step
        const char* kc = static_cast<const char*>(a.cache[0]) + (int64_t)u.h * D * eb;
        const char* vc = static_cast<const char*>(a.cache[1]) + (int64_t)u.h * D * eb;
        const char* ks = static_cast<const char*>(a.scales[0]) + u.h * (D / 32);
        const char* vs = static_cast<const char*>(a.scales[1]) + u.h * (D / 32);
        const int32_t* table = a.pg.table + (int64_t)u.s * a.pg.max_blocks;
        const int32_t* sel = SPARSE ? a.selected + (tok * a.heads + u.h) * a.topk : nullptr;
        // The row of flattened key kk (16 of them with PAGE16) and how many keys exist from there.
        auto find = [&](int32_t kk, int32_t& exist) -> int32_t {
            int32_t pos = kk;
            int32_t limit = q.keys - 1;
            exist = 0;
            if constexpr (SPARSE) {
                const int32_t n = kk >> a.pg.shift;
                if (n >= a.topk) return 0;
                const int32_t pb = sel[n];
                if (pb < 0 || pb >= a.pg.max_blocks) return 0;
                pos = (pb << a.pg.shift) + (kk & ((1 << a.pg.shift) - 1));
                limit = last;
            }
            if (pos > limit) return 0;
            const int32_t page = table[pos >> a.pg.shift];
            if (page < 0 || page >= a.pg.num_pages) return 0;
            exist = limit - pos + 1;
            return (page << a.pg.shift) + (pos & ((1 << a.pg.shift) - 1));
        };
        using KT = KeyTile<SUB, PAGE16>;
        // With PAGE16 the lanes look up the subtiles of the next kAhead steps at once, so the chain
        // of loads (selected page, page table, keys) is waited for once in kAhead steps.
        constexpr int kAhead = 64 / SUB;
        int32_t found0 = step0 - kAhead, found_row = 0, found_keys = 0;
        auto locate = [&](int32_t step) {
            KT t;
            const int32_t k0 = step * KS + wave * KW;
            t.valid = 0;
            if constexpr (PAGE16) {
                if (step >= found0 + kAhead) {
                    found0 = step;
                    found_row = found_keys = 0;
                    if (step + lane / SUB < u.steps)
                        found_row = find(k0 + lane / SUB * KS + lane % SUB * 16, found_keys);
                }
#pragma unroll
                for (int s = 0; s < SUB; ++s) {
                    const int from = (step - found0) * SUB + s;
                    t.base[s] = __builtin_amdgcn_readlane(found_row, from);
                    const int32_t exist = __builtin_amdgcn_readlane(found_keys, from);
                    const uint32_t bits = exist >= 16 ? 0xffffu : (1u << exist) - 1u;
                    t.valid |= bits << (16 * s);
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

        float m[R], l[R];
        f32x4 acc[R][T::NT];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            m[r] = -__builtin_inff();
            l[r] = 0.0f;
#pragma unroll
            for (int i = 0; i < T::NT; ++i) acc[r][i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        }
        const float to_log2 = logit_factor(a.scale);
        typename T::K kreg;
        typename T::V vreg;
        auto next_tile = [&](int32_t& step, KT& t) {  // the next step from `step` on with a key
            for (; step < step1; ++step) {
                t = locate(step);
                if (t.valid) return true;
            }
            return false;
        };
        int32_t left_out = 0;
        int32_t step = step0;
        KT tile;
        bool more = next_tile(step, tile);
        SC sreg;
        uint32_t* sc = scale_lds[wave];
        auto load_keys = [&](const KT& t) {
            if constexpr (MX) sreg.load(ks, vs, t, row_bytes / 32, lane);
            T::load_k(kc, t, row_bytes, c, g, kreg);
        };
        auto load_values = [&](const KT& t) { T::load_v(vc, t, row_bytes, c, g, vreg); };
        if (AHEAD && more) {
            load_keys(tile);
            load_values(tile);
        }
        // ---- queries: to LDS, whole rows
        __syncthreads();  // the last unit's use of LDS is over
        if (tid == 0) left_out_any = 0;
        {
            constexpr int PIECES = D * T::QB / 16;
            const char* qb = static_cast<const char*>(a.q);
            for (int x = tid; x < M * PIECES; x += kBlock) {
                const int r = x / PIECES, p = x % PIECES;
                const int64_t off = row_token(r) * a.q_stride + (int64_t)row_head(r) * D;
                *reinterpret_cast<uint4*>(lds + r * QSTRIDE + p * 16) = signed_by<E>(
                    *reinterpret_cast<const uint4*>(qb + off * T::QB + p * 16), a.scale);
            }
        }
        __syncthreads();
        typename T::Q qreg;
        if constexpr (QREG) T::load_q(lds + c * QSTRIDE, g, qreg);

        // Per step: logits from K, then the loads of the next K into the same registers, softmax
        // and the product with V, then the loads of the next V (of MXFP8 as soon as this V has been
        // widened). Where that takes more than half of
        // a SIMD's registers a step loads its own keys, and the other waves cover the wait.
        while (more) {
            if constexpr (!QREG) asm volatile("" ::: "memory");  // queries are read anew from LDS
            if constexpr (!AHEAD) {
                load_keys(tile);
                load_values(tile);
            }
            if constexpr (MX) sreg.put(sc, lane);
            const int32_t k0 = step * KS + wave * KW;
            const uint32_t valid = tile.valid;
            f32x4 x[R][SUB];
#pragma unroll
            for (int s = 0; s < SUB; ++s) {
                typename T::KOp ko;
                T::k_operands(kreg, sc, s, c, g, ko);
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    if constexpr (QREG) {
                        x[r][s] = T::logits(ko, qreg);
                    } else {
                        typename T::Q qr;
                        T::load_q(lds + (r * 16 + c) * QSTRIDE, g, qr);
                        x[r][s] = T::logits(ko, qr);
                    }
                }
            }
            KT next;
            int32_t next_step = step + 1;
            const bool another = next_tile(next_step, next);
            if (AHEAD && another) load_keys(next);

            // Which keys a row looks at. Every key of a full step below the context is seen by all
            // rows; selected pages are one token's, seen alike by all its heads.
            const bool all_seen = valid == kFull && (SPARSE || k0 + KW <= q.ctx);
            typename T::VOp vo;
            T::v_operands(vreg, sc, c, g, vo);
            if (AHEAD && MX && another) load_values(next);  // (widened: other registers)
            if (!all_seen) {
                // Keys that do not exist have rows that hold anything. Among the new tokens a row
                // of V may be one that only some query rows look at, and an infinity or a NaN
                // times a weight of zero would reach the others: those elements are left out
                // here and added at the end of the unit to the rows that do look at them.
                if (valid != kFull) T::clear(vo, valid, g);
                if (!SPARSE && T::cleanse(vo)) left_out = 1;
            }
            if (!all_seen) {
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    uint32_t bits = valid;
                    if constexpr (!SPARSE) {
                        const int64_t t = row_token(r * 16 + c);
                        bits &= mask_bits(a, t, (int32_t)(t - q.start), k0 - q.ctx);
                    }
                    bits >>= g * 4;
#pragma unroll
                    for (int j = 0; j < SUB * 4; ++j)
                        if (!((bits >> ((j >> 2) * 16 + (j & 3))) & 1))
                            x[r][j >> 2][j & 3] = -__builtin_inff();
                }
            }
#pragma unroll
            for (int r = 0; r < R; ++r) {
                float p[SUB * 4];
                float top = m[r];
#pragma unroll
                for (int j = 0; j < SUB * 4; ++j)
                    top = __builtin_fmaxf(top, x[r][j >> 2][j & 3]);
                top = row_max(top);
                if (__ballot(top > m[r])) {  // rescale only when a maximum has moved
                    const float f = exp2_fast(row_top(m[r], to_log2) - row_base(top, to_log2));
                    l[r] *= f;
#pragma unroll
                    for (int i = 0; i < T::NT; ++i)
#pragma unroll
                        for (int e = 0; e < 4; ++e) acc[r][i][e] *= f;
                    m[r] = top;
                }
                const float base = row_base(m[r], to_log2);
#pragma unroll
                for (int j = 0; j < SUB * 4; ++j) {
                    p[j] = exp2_fast(__builtin_fmaf(x[r][j >> 2][j & 3], to_log2, -base));
                    l[r] += p[j];
                }
                T::values(vo, p, acc[r]);
            }
            if (AHEAD && !MX && another) load_values(next);
            more = another;
            step = next_step;
            tile = next;
        }

        // ---- the four waves meet: common maximum, then the sums in a fixed order
        __syncthreads();  // every wave is done with the queries in LDS
        float big[R], sum[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            l[r] = row_sum(l[r]);
            m[r] = row_top(m[r], to_log2);  // from here on in base-2 logits
            if (g == 0) {
                stat[wave][0][r * 16 + c] = m[r];
                stat[wave][1][r * 16 + c] = l[r];
            }
        }
        if (left_out) left_out_any = 1;
        __syncthreads();
#pragma unroll
        for (int r = 0; r < R; ++r) {
            big[r] = -__builtin_inff();
            for (int w = 0; w < kWaves; ++w)
                big[r] = __builtin_fmaxf(big[r], stat[w][0][r * 16 + c]);
            const float base = big[r] == -__builtin_inff() ? 0.0f : big[r];
            sum[r] = 0.0f;
            for (int w = 0; w < kWaves; ++w)
                sum[r] += stat[w][1][r * 16 + c] * exp2_fast(stat[w][0][r * 16 + c] - base);
            const float f = exp2_fast(m[r] - base);
#pragma unroll
            for (int i = 0; i < T::NT; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[r][i][e] *= f;
        }
        float* buf = reinterpret_cast<float*>(lds);
        auto exchange = [&](int half, bool put) {
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int v = 0; v < T::NU; ++v)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int e = 0; e < T::CH; e += 4) {
                            f32x4* at_ = reinterpret_cast<f32x4*>(
                                buf + (half * M + r * 16 + c) * OSTRIDE + v * 16 * T::CH +
                                (g * 4 + i) * T::CH + e);
                            const int n = v * T::CH + e;
                            if (put) {
                                *at_ = f32x4{acc[r][n][i], acc[r][n + 1][i], acc[r][n + 2][i],
                                             acc[r][n + 3][i]};
                            } else {
                                const f32x4 y = *at_;
#pragma unroll
                                for (int k = 0; k < 4; ++k) acc[r][n + k][i] += y[k];
                            }
                        }
        };
        if (wave >= 2) exchange(wave - 2, true);
        __syncthreads();
        if (wave < 2) exchange(wave, false);
        __syncthreads();
        if (wave == 1) exchange(0, true);
        __syncthreads();
        const bool whole = step0 == 0 && step1 == u.steps;
        float* part = part_of<M, D>(ws, a.part_offset, me, step0 == 0);
        if (wave == 0) {
            exchange(0, false);
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const int row = r * 16 + c;
                const bool some = sum[r] > 0.0f || sum[r] != sum[r];
                const float inv = whole ? (some ? 1.0f / sum[r] : 0.0f) : 1.0f;
                if (!whole) {
                    if (g == 0) {
                        part[M * D + row] = big[r];
                        part[M * D + M + row] = sum[r];
                    }
                } else if (row < u.rows && g == 0 && a.lse != nullptr) {
                    a.lse[row_token(row) * a.heads * a.group + row_head(row)] =
                        some ? (big[r] + log2_fast(sum[r])) * kLn2 : -__builtin_inff();
                }
                if (row >= u.rows) continue;
                const int64_t o = (row_token(row) * a.heads * a.group + row_head(row)) * D;
#pragma unroll
                for (int v = 0; v < T::NU; ++v)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int d = v * 16 * T::CH + (g * 4 + i) * T::CH;
                        float y[T::CH];
#pragma unroll
                        for (int e = 0; e < T::CH; ++e) y[e] = acc[r][v * T::CH + e][i] * inv;
                        if (whole) {
                            store_row<E, T::CH>(a.out, o + d, y);
                        } else {
#pragma unroll
                            for (int e = 0; e < T::CH; e += 4)
                                *reinterpret_cast<f32x4*>(part + row * D + d + e) =
                                    f32x4{y[e], y[e + 1], y[e + 2], y[e + 3]};
                        }
                    }
            }
        }
        if (!SPARSE && left_out_any) {  // (set before the waves met, the same for all)
            __syncthreads();            // the rows are written
            add_left_out<E, MX, D>(a, q, u, (int64_t)step0 * KS, (int64_t)step1 * KS,
                                   whole ? nullptr : part);
        }
    }
}

template <class E, bool MX, int D, int R, bool SPARSE>
hipError_t run(const AttnArgs& a, hipStream_t st) {
    if (a.pg.shift >= 4) attention_kernel<E, MX, D, R, SPARSE, true><<<kWorkers, kBlock, 0, st>>>(a);
    else attention_kernel<E, MX, D, R, SPARSE, false><<<kWorkers, kBlock, 0, st>>>(a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    using S = Steps<16 * Tile<E, MX, D>::SUB * kWaves, 16 * R, 0>;
    return launch_join<E, D, S, kWorkers, SPARSE>(a, st);
}

template <class E, bool MX, int D, bool SPARSE>
hipError_t by_rows(const AttnArgs& a, int R, hipStream_t st) {
    if constexpr (D <= 128) {
        if (R == 2) return run<E, MX, D, 2, SPARSE>(a, st);
    }
    return run<E, MX, D, 1, SPARSE>(a, st);
}

template <class E, bool MX, bool SPARSE>
hipError_t by_dim(const AttnArgs& a, int D, int R, hipStream_t st) {
    if (D == 64) return by_rows<E, MX, 64, SPARSE>(a, R, st);
    if (D == 128) return by_rows<E, MX, 128, SPARSE>(a, R, st);
    return by_rows<E, MX, 256, SPARSE>(a, R, st);
}

template <bool SPARSE>
hipError_t dispatch(const AttnArgs& a, bool mx, int dtype, int D, int R, hipStream_t st) {
    if (dtype == 0)
        return mx ? by_dim<F32, true, SPARSE>(a, D, R, st) : by_dim<F32, false, SPARSE>(a, D, R, st);
    return mx ? by_dim<BF16, true, SPARSE>(a, D, R, st) : by_dim<BF16, false, SPARSE>(a, D, R, st);
}

}  // namespace

hipError_t launch_attention(const AttnArgs& a, bool selected, bool mx, int dtype, int D, int R,
                            hipStream_t st) {
    return selected ? dispatch<true>(a, mx, dtype, D, R, st)
                    : dispatch<false>(a, mx, dtype, D, R, st);
}

}  // namespace sc
