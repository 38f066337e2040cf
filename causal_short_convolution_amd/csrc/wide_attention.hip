// Tree attention for units of many query rows (shortconv_tree_attention, bf16 queries): the waves
// share the keys and split the rows, 16 R rows each.
//
// With more than 32 rows the products outweigh the reads of the cache, and the waves of
// cache_attention.hip, which each stream their own keys, would each hold all rows. Here a step of
// 64 keys is brought in once per workgroup, into LDS in the form in which the products take it:
// K by rows, V transposed (rows of channels, keys in the order in which the lane of a query row
// holds their weights), both in bf16 whatever the cache holds. With 8 waves two such buffers
// alternate: while step t is computed from one, step t + 1, loaded to registers a step earlier, is
// written to the other, and the loads of step t + 2 are under way; one barrier per step. With 4 waves
// (D <= 128) there is one buffer, written between two barriers while the next step's loads are under way:
// LDS and registers then hold three workgroups on a CU, whose phases overlap better than those of
// two with two buffers (64 sequences x 64 rows over 512-8192 MXFP8 keys of 8 heads: 189 against 207 us;
// loads two steps ahead changed nothing).
//
// Measured: 2 x 256 rows over 131072 keys of 8 heads of 128, bf16: 500-545 us, 0.5 PFLOP/s, 65 % of
// the issue slots taken, 44 % of the matrix cores' time.
//
// Rows in LDS are not padded; their 16-byte pieces are permuted by exclusive or with bits of the row,
// so that the lanes that an access serves at a time fall on different banks: 16 rows of one piece
// (or of two neighbouring pieces, rows 4 by 4) where operands are read, whole rows and 16 rows of V
// where they are written. Padding rows by 16 bytes instead cost 850 conflict cycles of 5000 per step.
#include "attention_line.h"

namespace sc {
namespace {

constexpr int kKeys = 64;  // keys per step
// What a step costs beside its tiles of 16 query rows, in the cost of one tile. Measured on 131072 keys
// of 8 heads: steps of 2.9 us with 16 tiles, of 2.0 us with one.
constexpr int kLoadCost = 32;

template <int D>
struct Places {
    static constexpr int KROW = D * 2;
    static constexpr int VROW = kKeys * 2;
    static constexpr int K_BYTES = kKeys * KROW;
    static constexpr int V_BYTES = D * VROW;
    // What the piece numbers of a row of BYTES are permuted by: 256 bytes hold all banks, so rows of
    // 128 change it every second row.
    template <int BYTES>
    __device__ static inline int turn(int row) {
        return BYTES == 128 ? (row >> 1) & 7 : row & 15;
    }
    // Place of 16-byte piece `piece` of the K row of key `key`.
    __device__ static inline int k(int key, int piece) {
        return key * KROW + ((piece ^ turn<KROW>(key)) << 4);
    }
    // V's rows: channel CW c + e is row e D / CW + c, which holds the keys i, i + 16 for
    // i = 32 kb + 4 g .. (in the order of the weights) as its piece 4 kb + g.
    static constexpr int CW = D / 16 < 8 ? D / 16 : 8;  // channels that a thread turns at a time
    __device__ static inline int v_row(int c, int e) { return e * (D / CW) + c; }
    __device__ static inline int v(int row, int piece) {
        return row * VROW + ((piece ^ turn<VROW>(row)) << 4);
    }
};

// What one thread loads of a step: pieces of 16 bytes of K rows, and the same CW channels of 4 rows
// of V. Of 8 waves four load V and four load K, into the same registers; 4 waves load both.
template <bool MX, int D, int NW>
struct Pieces {
    static constexpr bool SPLIT = NW == 8;
    static constexpr int CW = Places<D>::CW;
    static constexpr int KP = MX ? D / 16 : D / 8;  // pieces per K row
    static constexpr int KN = kKeys * KP / 256;     // pieces per thread
    static constexpr int VP = D / CW;               // pieces per V row
    static constexpr int VN = kKeys / 4 * VP / 256;
    static constexpr int VW = MX ? CW / 4 : CW / 2; // words per piece of a V row
    static constexpr int K_WORDS = KN * 4, V_WORDS = VN * 4 * VW;
    static constexpr int V0 = SPLIT ? 0 : K_WORDS;
    static constexpr int WORDS = !SPLIT ? K_WORDS + V_WORDS
                                        : K_WORDS > V_WORDS ? K_WORDS : V_WORDS;
    static constexpr int KK = 64 / KP, VK = 256 / VP;  // keys of a wave's n-th piece
    static_assert(KN * 256 == kKeys * KP && VN * 256 == kKeys / 4 * VP, "whole shares");
    uint32_t w[WORDS];
    // MXFP8: a wave's pieces are of 16 keys of K and 16 of V, whose scales its lanes load as words,
    // one each (lane % 16 the key, lane / 32 the word; bit 4 says V where a wave loads both) and
    // hand each other when the pieces are widened. Each lane loading its own bytes took half of all
    // load instructions.
    uint32_t scale;
};

template <bool MX, int D, int NW, int R>
__global__ void __launch_bounds__(64 * NW, D == 256 && NW == 4 ? 1 : NW == 4 ? 3 : 2) wide_kernel(AttnArgs a) {
    using T = Tile<BF16, false, D>;  // after staging the operands are bf16
    using X = Tile<BF16, MX, D>;
    using PL = Places<D>;
    constexpr int NT = 64 * NW;
    constexpr int M = 16 * R * NW;
    constexpr int WORKERS = wide_workers(NW, D);
    using S = Steps<kKeys, M, kLoadCost>;
    using PC = Pieces<MX, D, NW>;
    constexpr int BUFS = NW == 4 && D <= 128 ? 1 : 2;
    __shared__ __attribute__((aligned(16))) char kbuf[BUFS][PL::K_BYTES];
    __shared__ __attribute__((aligned(16))) char vbuf[BUFS][PL::V_BYTES];
    __shared__ RunScratch run;
    __shared__ int32_t left_out_any;

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = uniform(tid >> 6);
    const int c = lane & 15, g = lane >> 4;
    constexpr int EB = MX ? 1 : 2;
    const uint32_t row_bytes = (uint32_t)(a.heads * D * EB);
    char* ws = static_cast<char*>(a.ws);

    const int64_t total = find_run<S, WORKERS, NT>(a, reinterpret_cast<int64_t*>(ws), run);
    const Shares<WORKERS> sh(total, S::kMost);
    const int32_t me = sh.me();
    if (me >= sh.workers) return;
    int64_t at = sh.begin(me);
    const int64_t end = sh.begin(me + 1);
    Unit u;
    u.s = uniform(run.s);
    int64_t seq_first = uniform(run.first);
    SeqInfo q = seq_info(a.b, a.pg, u.s);
    const float to_log2 = logit_factor(a.scale);

    while (at < end) {
        unit_at<S>(a, at, u, q, seq_first);
        const int32_t step0 = u.step_at(at), step1 = u.step_at(end);
        at = u.end();
        if (step0 == step1) continue;  // the unit's last step started in the run before

        // Row tiles go round the waves: tile wave + NW r is the wave's r-th.
        const int tiles = (u.rows + 15) / 16;
        const int mine = tiles > wave ? (tiles - wave - 1) / NW + 1 : 0;
        auto row_of = [&](int r) { return (wave + NW * r) * 16 + c; };
        auto row_index = [&](int row) { return u.row0 + (row < u.rows ? row : u.rows - 1); };
        typename T::Q qreg[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int32_t x = row_index(row_of(r));
            const int64_t off = (u.tok + x / a.group) * a.q_stride +
                                (int64_t)(u.h * a.group + x % a.group) * D;
            T::load_q(static_cast<const char*>(a.q) + off * 2, g, qreg[r]);
#pragma unroll
            for (int f = 0; f < T::NF; ++f)
                qreg[r][f] = __builtin_bit_cast(
                    bf16x8, signed_by<BF16>(__builtin_bit_cast(uint4, qreg[r][f]), a.scale));
        }
        const char* kc = static_cast<const char*>(a.cache[0]) + (int64_t)u.h * D * EB;
        const char* vc = static_cast<const char*>(a.cache[1]) + (int64_t)u.h * D * EB;
        const uint8_t* ks = static_cast<const uint8_t*>(a.scales[0]) + u.h * (D / 32);
        const uint8_t* vs = static_cast<const uint8_t*>(a.scales[1]) + u.h * (D / 32);

        // ---- a step's keys: lane l finds the row of key l (-1: there is none). The page id is
        // fetched a step before it is looked at, so that nothing waits for it.
        const int32_t* table = a.pg.table + (int64_t)u.s * a.pg.max_blocks;
        auto fetch = [&](int32_t step) -> int32_t {
            const uint32_t p = (uint32_t)step * kKeys + lane;
            return table[min(p, (uint32_t)q.keys - 1) >> a.pg.shift];
        };
        auto row_slot = [&](int32_t page, int32_t step) -> int32_t {
            const uint32_t p = (uint32_t)step * kKeys + lane;
            const bool ok = step < step1 && p < (uint32_t)q.keys && page >= 0 &&
                            page < a.pg.num_pages;
            return ok ? (page << a.pg.shift) + (int32_t)(p & ((1u << a.pg.shift) - 1u)) : -1;
        };
        PC pc;
        const int t8 = tid & 255;
        // The n-th piece of V of this thread: keys 32 kb + 16 s + 4 gg .. + 3, channels CW ch ..
        auto v_item = [&](int n, int& kb, int& gg, int& s, int& ch) {
            const int x = n * 256 + t8;
            ch = x % PC::VP;
            const int y = x / PC::VP;
            s = y & 1;
            gg = (y >> 1) & 3;
            kb = y >> 3;
        };
        // With pages of at least a step's keys the step's rows lie one after the other behind a row
        // that is the same for all lanes, and only scalars change from step to step.
        const bool one_page = (1 << a.pg.shift) >= kKeys;
        auto row_of_key = [&](int32_t row, int key) -> int64_t {  // in bytes
            return one_page ? uniform((int64_t)((uint64_t)(uint32_t)uniform(row) * row_bytes)) +
                                  (uint32_t)key * row_bytes
                            : (int64_t)((uint64_t)(uint32_t)__shfl(row, key) * row_bytes);
        };
        auto load_k = [&](PC& pc, int32_t row) {
#pragma unroll
            for (int n = 0; n < PC::KN; ++n) {
                const int x = n * 256 + t8;
                const int64_t r = row_of_key(row, x / PC::KP);
                const u32x4 y = *reinterpret_cast<const u32x4*>(kc + r + x % PC::KP * 16);
#pragma unroll
                for (int i = 0; i < 4; ++i) pc.w[n * 4 + i] = y[i];
            }
        };
        auto load_v = [&](PC& pc, int32_t row) {
#pragma unroll
            for (int n = 0; n < PC::VN; ++n) {
                int kb, gg, s, ch;
                v_item(n, kb, gg, s, ch);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int64_t r = row_of_key(row, kb * 32 + s * 16 + gg * 4 + j);
                    const char* p = vc + r + ch * PL::CW * EB;
                    uint32_t* w = pc.w + PC::V0 + (n * 4 + j) * PC::VW;
                    if constexpr (PC::VW == 4) {
                        const u32x4 y = *reinterpret_cast<const u32x4*>(p);
#pragma unroll
                        for (int i = 0; i < 4; ++i) w[i] = y[i];
                    } else if constexpr (PC::VW == 2) {
                        const u32x2_t y = *reinterpret_cast<const u32x2_t*>(p);
                        w[0] = y[0];
                        w[1] = y[1];
                    } else {
                        w[0] = *reinterpret_cast<const uint32_t*>(p);
                    }
                }
            }
        };
        const bool loads_v = PC::SPLIT ? wave < 4 : (lane >> 4) & 1;
        auto load_scales = [&](PC& pc, int32_t row) {
            const int i = lane & 15, w4 = t8 >> 6;
            const int y = (i / PC::VK * 256 + w4 * 64) / PC::VP + i % PC::VK / 4;
            const int key = loads_v ? (y >> 3) * 32 + (y & 1) * 16 + ((y >> 1) & 3) * 4 + (i & 3)
                                    : (i / PC::KK * 256 + w4 * 64) / PC::KP + i % PC::KK;
            const uint8_t* p = (loads_v ? vs : ks) + row_of_key(row, key) / 32;
            if constexpr (D == 64) pc.scale = *reinterpret_cast<const uint16_t*>(p);
            else pc.scale = *reinterpret_cast<const uint32_t*>(p + (D > 128 ? lane >> 5 : 0) * 4);
        };
        // Byte `byte` of the scales of the wave's key i, of V or K.
        auto scale_of = [&](const PC& pc, bool v, int i, int byte) {
            const uint32_t w = __shfl(pc.scale, (byte >> 2) * 32 + (v && !PC::SPLIT ? 16 : 0) + i);
            return e8m0((w >> ((byte & 3) * 8)) & 255u);
        };
        // (a slot of -1 is loaded as row 0, which a pool with pages has)
        auto load = [&](PC& pc, int32_t slots) {
            const int32_t row = slots < 0 ? 0 : slots;
            if constexpr (MX) load_scales(pc, row);
            if constexpr (PC::SPLIT) {
                if (wave < 4) load_v(pc, row);
                else load_k(pc, row);
            } else {
                load_k(pc, row);
                load_v(pc, row);
            }
        };
        auto store_k = [&](const PC& pc, int buf) {
#pragma unroll
            for (int n = 0; n < PC::KN; ++n) {
                const int x = n * 256 + t8;
                const int key = x / PC::KP, piece = x % PC::KP;
                const uint32_t* w = pc.w + n * 4;
                if constexpr (MX) {
                    const float e = scale_of(pc, false, n * PC::KK + lane / PC::KP, lane % PC::KP / 2);
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        *reinterpret_cast<u32x4*>(kbuf[buf] + PL::k(key, piece * 2 + i)) = u32x4{
                            X::widen2(w[2 * i], e, false), X::widen2(w[2 * i], e, true),
                            X::widen2(w[2 * i + 1], e, false), X::widen2(w[2 * i + 1], e, true)};
                } else {
                    *reinterpret_cast<u32x4*>(kbuf[buf] + PL::k(key, piece)) =
                        u32x4{w[0], w[1], w[2], w[3]};
                }
            }
        };
        auto store_v = [&](const PC& pc, int buf, int32_t step, uint64_t valid) {
            const bool plain = valid == ~0ull && (int64_t)(step + 1) * kKeys <= q.ctx;
#pragma unroll
            for (int n = 0; n < PC::VN; ++n) {
                int kb, gg, s, ch;
                v_item(n, kb, gg, s, ch);
                constexpr int CP = PL::CW / 2;
                uint32_t w[4][CP];  // [key][channel pair]
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    float scale = 1.0f;
                    if constexpr (MX)
                        scale = scale_of(pc, true, n * PC::VK + lane / PC::VP * 4 + j, ch * PL::CW / 32);
#pragma unroll
                    for (int i = 0; i < CP; ++i) {
                        const uint32_t* from = pc.w + PC::V0 + (n * 4 + j) * PC::VW;
                        if constexpr (MX) w[j][i] = X::widen2(from[i / 2], scale, i & 1);
                        else w[j][i] = from[i];
                    }
                }
                if (!plain) {
                    // Keys that do not exist count as zeros. Among the new tokens a row of V may
                    // be one that only some query rows look at, and an infinity or a NaN times
                    // a weight of zero would reach the others: those elements are left out here
                    // and added at the end of the unit to the rows that do look at them.
                    bool any = false;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const bool ok = (valid >> (kb * 32 + s * 16 + gg * 4 + j)) & 1;
#pragma unroll
                        for (int i = 0; i < CP; ++i) {
                            const bool lo = (w[j][i] & 0x7f80u) == 0x7f80u;
                            const bool hi = (w[j][i] & 0x7f800000u) == 0x7f800000u;
                            any |= ok && (lo || hi);
                            w[j][i] &= (lo ? 0xffff0000u : ~0u) & (hi ? 0x0000ffffu : ~0u);
                            w[j][i] = ok ? w[j][i] : 0u;
                        }
                    }
                    if (any) left_out_any = 1;
                }
#pragma unroll
                for (int e = 0; e < PL::CW; ++e) {
                    const uint32_t sel = (e & 1) ? 0x07060302u : 0x05040100u;
                    const u32x2_t pair = {
                        __builtin_amdgcn_perm(w[1][e / 2], w[0][e / 2], sel),
                        __builtin_amdgcn_perm(w[3][e / 2], w[2][e / 2], sel)};
                    *reinterpret_cast<u32x2_t*>(
                        vbuf[buf] + PL::v(PL::v_row(ch, e), kb * 4 + gg) + s * 8) = pair;
                }
            }
        };
        auto store = [&](const PC& pc, int buf, int32_t step, uint64_t valid) {
            if constexpr (PC::SPLIT) {
                if (wave < 4) store_v(pc, buf, step, valid);
                else store_k(pc, buf);
            } else {
                store_k(pc, buf);
                store_v(pc, buf, step, valid);
            }
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
        // One step for the wave's row tiles. LDS is read AHEAD operands ahead of
        // the products that take them (the scheduling barriers keep them so).
        auto compute = [&](int buf, int32_t step, uint64_t valid) {
            const int32_t k0 = step * kKeys;
            // operand i of K: subtile i / NF, channels f = i % NF; of V: channel tile i / 2, keys 32 (i % 2)
            constexpr int AHEAD = 4;
            constexpr int NK = 4 * T::NF, NV = 2 * T::NT;
            bf16x8 op[AHEAD];
            auto read_k = [&](int i) {
                op[i % AHEAD] = *reinterpret_cast<const bf16x8*>(
                    kbuf[buf] + i / T::NF * 16 * PL::KROW + PL::k(c, i % T::NF * 4 + g));
            };
            auto read_v = [&](int i) {
                op[i % AHEAD] = *reinterpret_cast<const bf16x8*>(
                    vbuf[buf] + i / 2 * 16 * PL::VROW + PL::v(c, i % 2 * 4 + g));
            };
            f32x4 x[R][4];
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int s = 0; s < 4; ++s) x[r][s] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int i = 0; i < AHEAD; ++i) read_k(i);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int i = 0; i < NK; ++i) {
#pragma unroll
                for (int r = 0; r < R; ++r)
                    x[r][i / T::NF] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                        op[i % AHEAD], qreg[r][i % T::NF], x[r][i / T::NF], 0, 0, 0);
                if (i + AHEAD < NK) read_k(i + AHEAD);
                __builtin_amdgcn_sched_barrier(0);
            }
            if (valid != ~0ull || k0 + kKeys > q.ctx) {  // some rows do not look at some keys
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    const int32_t i = row_index(row_of(r)) / a.group;
                    const uint32_t bits[2] = {
                        ((uint32_t)valid & mask_bits(a, u.tok + i, i, k0 - q.ctx)) >> (g * 4),
                        ((uint32_t)(valid >> 32) & mask_bits(a, u.tok + i, i, k0 + 32 - q.ctx)) >>
                            (g * 4)};
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        if (!((bits[j >> 3] >> ((j >> 2 & 1) * 16 + (j & 3))) & 1))
                            x[r][j >> 2][j & 3] = -__builtin_inff();
                }
            }
#pragma unroll
            for (int i = 0; i < AHEAD; ++i) read_v(i);
            __builtin_amdgcn_sched_barrier(0);
            bf16x8 p[R][2];
#pragma unroll
            for (int r = 0; r < R; ++r) {
                float y[16];
                float top = m[r];
#pragma unroll
                for (int j = 0; j < 16; ++j) top = __builtin_fmaxf(top, x[r][j >> 2][j & 3]);
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
                for (int j = 0; j < 16; ++j) {
                    y[j] = exp2_fast(__builtin_fmaf(x[r][j >> 2][j & 3], to_log2, -base));
                    l[r] += y[j];
                }
#pragma unroll
                for (int b = 0; b < 2; ++b)
                    p[r][b] = __builtin_bit_cast(
                        bf16x8, make_uint4(BF16::pack2(y[8 * b], y[8 * b + 1]),
                                           BF16::pack2(y[8 * b + 2], y[8 * b + 3]),
                                           BF16::pack2(y[8 * b + 4], y[8 * b + 5]),
                                           BF16::pack2(y[8 * b + 6], y[8 * b + 7])));
            }
#pragma unroll
            for (int i = 0; i < NV; ++i) {
#pragma unroll
                for (int r = 0; r < R; ++r)
                    acc[r][i / 2] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                        op[i % AHEAD], p[r][i % 2], acc[r][i / 2], 0, 0, 0);
                if (i + AHEAD < NV) read_v(i + AHEAD);
                __builtin_amdgcn_sched_barrier(0);
            }
        };
        __syncthreads();  // the last unit is done with LDS
        if (tid == 0) left_out_any = 0;
        if (q.keys > 0 && a.pg.num_pages > 0) {
            // (steps past the last are loaded as row 0 and count as no keys)
            int32_t page = fetch(step0);
            auto load_next = [&](int32_t step) {  // the step after those under way
                const int32_t slots = row_slot(page, step);
                page = fetch(step + 1);
                load(pc, slots);
                return (uint64_t)__ballot(slots >= 0);
            };
            uint64_t now = load_next(step0), next = 0;
            __syncthreads();  // left_out_any is cleared
            if constexpr (BUFS == 2) {
                store(pc, 0, step0, now);
                next = load_next(step0 + 1);
                __syncthreads();
            }
            for (int32_t step = step0; step < step1; ++step) {
                if constexpr (BUFS == 2) {
                    const int buf = (step - step0) & 1;
                    store(pc, buf ^ 1, step + 1, next);
                    const uint64_t after = load_next(step + 2);
                    if (now && mine > 0) compute(buf, step, now);
                    now = next;
                    next = after;
                } else {
                    store(pc, 0, step, now);
                    next = load_next(step + 1);
                    __syncthreads();
                    if (now && mine > 0) compute(0, step, now);
                    now = next;
                }
                __syncthreads();
            }
        } else {
            __syncthreads();  // left_out_any is cleared
        }

        // ---- every wave writes its own rows
        const bool whole = step0 == 0 && step1 == u.steps;
        float* part = part_of<M, D>(ws, a.part_offset, me, step0 == 0);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int row = row_of(r);
            const float sum = row_sum(l[r]);
            const bool some = sum > 0.0f || sum != sum;
            const float inv = whole ? (some ? 1.0f / sum : 0.0f) : 1.0f;
            if (row >= u.rows) continue;
            const int32_t x = u.row0 + row;
            const int64_t t = u.tok + x / a.group;
            const int64_t o = t * a.heads * a.group + u.h * a.group + x % a.group;
            if (g == 0) {
                const float top = row_top(m[r], to_log2);
                if (!whole) {
                    part[M * D + row] = top;
                    part[M * D + M + row] = sum;
                } else if (a.lse != nullptr) {
                    a.lse[o] = some ? (top + log2_fast(sum)) * kLn2 : -__builtin_inff();
                }
            }
            // Register i of tile n holds row 16 n + 4 g + i of V, so the tiles k, k + KT, .. hold CW
            // consecutive channels.
            constexpr int CW = PL::CW, KT = T::NT / CW;
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int k = 0; k < KT; ++k) {
                    const int d = (k * 16 + g * 4 + i) * CW;
                    float y[CW];
#pragma unroll
                    for (int e = 0; e < CW; ++e) y[e] = acc[r][e * KT + k][i] * inv;
                    if (whole) {
                        store_row<BF16, CW>(a.out, o * D + d, y);
                    } else {
#pragma unroll
                        for (int e = 0; e < CW; e += 4)
                            *reinterpret_cast<f32x4*>(part + row * D + d + e) =
                                f32x4{y[e], y[e + 1], y[e + 2], y[e + 3]};
                    }
                }
        }
        if (left_out_any) {   // (set before the last step's barrier, the same for all)
            __syncthreads();  // the rows are written
            add_left_out<BF16, MX, D>(a, q, u, (int64_t)step0 * kKeys, (int64_t)step1 * kKeys,
                                      whole ? nullptr : part);
        }
    }
}

template <bool MX, int D, int NW, int R>
hipError_t run(const AttnArgs& a, hipStream_t st) {
    wide_kernel<MX, D, NW, R><<<wide_workers(NW, D), 64 * NW, 0, st>>>(a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    using S = Steps<kKeys, 16 * R * NW, kLoadCost>;
    return launch_join<BF16, D, S, wide_workers(NW, D), false>(a, st);
}

template <bool MX, int D>
hipError_t by_shape(const AttnArgs& a, AttnShape s, hipStream_t st) {
    if (s.waves == 4) return run<MX, D, 4, 1>(a, st);
    if constexpr (D <= 128) {
        if (s.tiles == 3) return run<MX, D, 8, 3>(a, st);
        if (s.tiles == 2) return run<MX, D, 8, 2>(a, st);
    }
    return run<MX, D, 8, 1>(a, st);
}

template <bool MX>
hipError_t by_dim(const AttnArgs& a, int D, AttnShape s, hipStream_t st) {
    if (D == 64) return by_shape<MX, 64>(a, s, st);
    if (D == 128) return by_shape<MX, 128>(a, s, st);
    return by_shape<MX, 256>(a, s, st);
}

}  // namespace

hipError_t launch_wide_attention(const AttnArgs& a, bool mx, int D, AttnShape s, hipStream_t st) {
    return mx ? by_dim<true>(a, D, s, st) : by_dim<false>(a, D, s, st);
}

}  // namespace sc
