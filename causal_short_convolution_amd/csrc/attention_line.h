// The line of steps that the attention kernels share out: units of work, their place in the line,
// each worker's run, and the launch that joins the parts of units which crossed workers.
#ifndef SHORTCONV_ATTENTION_LINE_H
#define SHORTCONV_ATTENTION_LINE_H

#include "attention_tile.h"
#include "cache_attention.h"

namespace sc {

// A line of `total` units of cost over at most WORKERS workers, each with no less than `most`, the
// cost of one step: worker w owns the steps that start in [begin(w), begin(w + 1)).
template <int WORKERS>
struct Shares {
    int64_t total, each, more;
    int32_t workers;
    __device__ Shares(int64_t t, int32_t most) : total(t) {
        const int64_t n = t / most;
        workers = (int32_t)(n < WORKERS ? n : WORKERS);
        each = workers ? t / workers : 0;
        more = workers ? t - each * workers : 0;
    }
    __device__ int64_t begin(int32_t w) const { return w * each + (w < more ? w : more); }
    __device__ int32_t owner(int64_t at) const {
        const int64_t cut = more * (each + 1);
        return (int32_t)(at < cut ? at / (each + 1) : more + (at - cut) / each);
    }
    // The worker that this workgroup is. Workgroups go round the 8 XCDs by blockIdx. Where every
    // workgroup has work, consecutive runs go to one XCD, so that units that read the same rows
    // meet in its L2; fewer are spread over the XCDs.
    __device__ int32_t me() const {
        return workers < WORKERS ? (int32_t)blockIdx.x
                                 : (int32_t)(blockIdx.x & 7) * (WORKERS / 8) +
                                       (int32_t)(blockIdx.x >> 3);
    }
};

// One unit of work: a cache head of a sequence (of a token, for selected pages) and up to M of the
// query rows that read it.
struct Unit {
    int32_t s;          // sequence
    int32_t h;          // cache head
    int32_t row0;       // first query row (of the sequence's len * group, or the token's group)
    int32_t rows;       // rows in this unit, 1 .. M
    int32_t steps;      // steps of all its keys, at least 1
    int32_t cost;       // of one step
    int64_t tok;        // selected pages: the token; else the sequence's first
    int64_t first;      // its place in the line
    // The first step at or behind place `at` of the line, at most `steps`.
    __device__ int32_t step_at(int64_t at) const {
        const int64_t n = at <= first ? 0 : (at - first + cost - 1) / cost;
        return (int32_t)(n < steps ? n : steps);
    }
    __device__ int64_t end() const { return first + (int64_t)steps * cost; }
};

// Sizes in steps of KS keys and units of M rows. A step costs what loading its keys does, LOAD, and
// one for each tile of 16 rows; where LOAD is 0, every wave does all rows of a step, filled or not,
// and each step counts 1.
template <int KS_, int M_, int LOAD_>
struct Steps {
    static constexpr int KS = KS_, M = M_, LOAD = LOAD_;
    __device__ static inline int32_t cost(int32_t rows) {
        return LOAD == 0 ? 1 : LOAD + (rows + 15) / 16;
    }
    static constexpr int32_t kMost = LOAD == 0 ? 1 : LOAD + M / 16;
    __device__ static inline int64_t of_keys(int64_t keys) {
        return keys > KS ? (keys + KS - 1) / KS : 1;
    }
    // Cost of a step of all units of one head, the whole ones and the last.
    __device__ static inline int64_t of_rows(int64_t rows) {
        const int64_t whole = rows / M;
        const int32_t rest = (int32_t)(rows - whole * M);
        return whole * kMost + (rest ? cost(rest) : 0);
    }
    // Cost of a sequence: its cache heads, times the units of its rows, times its key steps.
    __device__ static inline int64_t of_sequence(const AttnArgs& a, const SeqInfo& q) {
        if (q.len == 0) return 0;
        return a.heads * of_rows((int64_t)q.len * a.group) * of_keys(q.keys);
    }
    __device__ static inline int32_t of_pages(const AttnArgs& a) {
        return (int32_t)of_keys((int64_t)a.topk << a.pg.shift);
    }
    __device__ static inline int32_t group_tiles(const AttnArgs& a) {
        return (a.group + M - 1) / M;
    }
    // The unit of row `row` (of the sequence's, or the token's) of head h, behind `head0`, where
    // the line's units of its head begin.
    __device__ static inline void place(Unit& u, int64_t rows, int64_t row, int64_t head0) {
        const int64_t index = row / M;
        u.row0 = (int32_t)(index * M);
        u.rows = (int32_t)(rows - u.row0 < M ? rows - u.row0 : M);
        u.cost = cost(u.rows);
        u.first = head0 + index * u.steps * kMost;
    }
};

// LDS of find_run.
struct RunScratch {
    int64_t sums[16];
    int64_t first;
    int32_t s;
};

// By the whole workgroup: the cost of all sequences; in `scratch` the sequence that this worker's run
// begins in and that sequence's place in the line. The first worker leaves the prefix sums for the
// joining launch, if there is one, in `prefix`.
template <class S, int WORKERS, int THREADS>
__device__ inline int64_t find_run(const AttnArgs& a, int64_t* prefix, RunScratch& scratch) {
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int per = (a.b.num_seqs + THREADS - 1) / THREADS;
    int64_t mine = 0;
    for (int j = 0; j < per; ++j) {
        const int s = tid * per + j;
        if (s < a.b.num_seqs) mine += S::of_sequence(a, seq_info(a.b, a.pg, s));
    }
    int64_t inc = mine;
    for (int d = 1; d < 64; d <<= 1) {
        const int64_t o = __shfl_up(inc, d);
        if (lane >= d) inc += o;
    }
    if (lane == 63) scratch.sums[wave] = inc;
    __syncthreads();
    int64_t before = 0, total = 0;
    for (int w = 0; w < THREADS / 64; ++w) {
        if (w < wave) before += scratch.sums[w];
        total += scratch.sums[w];
    }
    const Shares<WORKERS> sh(total, S::kMost);
    const int32_t me = sh.me();
    const int64_t want = me < sh.workers ? sh.begin(me) : -1;
    int64_t x = before + inc - mine;
    for (int j = 0; j < per; ++j) {
        const int s = tid * per + j;
        if (s >= a.b.num_seqs) break;
        const int64_t n = S::of_sequence(a, seq_info(a.b, a.pg, s));
        if (want >= x && want < x + n) {
            scratch.s = s;
            scratch.first = x;
        }
        if (me == 0 && prefix != nullptr) prefix[s] = x;
        x += n;
    }
    if (me == 0 && tid == THREADS - 1 && prefix != nullptr) prefix[a.b.num_seqs] = total;
    __syncthreads();
    return total;
}

// The unit of place `at` in a line of whole sequences; u.s, q and seq_first (where sequence u.s
// begins) move on as needed.
template <class S>
__device__ inline void unit_at(const AttnArgs& a, int64_t at, Unit& u, SeqInfo& q,
                               int64_t& seq_first) {
    int64_t n = S::of_sequence(a, q);
    while (at >= seq_first + n) {
        seq_first += n;
        q = seq_info(a.b, a.pg, ++u.s);
        n = S::of_sequence(a, q);
    }
    u.steps = (int32_t)S::of_keys(q.keys);
    u.tok = q.start;
    const int64_t rows = (int64_t)q.len * a.group;
    const int64_t head = S::of_rows(rows) * u.steps;  // cost of one head
    u.h = (int32_t)((at - seq_first) / head);
    const int64_t head0 = seq_first + u.h * head;
    const int64_t whole = (int64_t)u.steps * S::kMost;
    S::place(u, rows, (at - head0) / whole * S::M, head0);
}

// A part of a unit that worker `me` computed, in the workspace: M rows of D sums, then the rows'
// maxima and sums of weights. Slot 1 if it holds the unit's first step (the worker's last part),
// else slot 0 (its first).
template <int M, int D>
__device__ inline float* part_of(void* ws, int64_t offset, int32_t worker, bool holds_first) {
    return reinterpret_cast<float*>(static_cast<char*>(ws) + offset) +
           ((int64_t)worker * 2 + holds_first) * (M * (D + 2));
}

// The infinities and NaN that V has in the new tokens of key positions [k0, k1), which the products
// left out: adds them to the written rows (or part) of the unit that look at them. By the whole
// workgroup, after the rows are written; rare.
template <class E, bool MX, int D>
__device__ inline void add_left_out(const AttnArgs& a, const SeqInfo& q, const Unit& u, int64_t k0,
                                    int64_t k1, float* part) {
    const int32_t first = (int32_t)max((int64_t)q.ctx, k0);
    const int32_t last = (int32_t)min((int64_t)q.keys, k1);
    for (int x = threadIdx.x; x < u.rows * D; x += blockDim.x) {
        const int row = x / D, d = x % D;
        const int32_t y = u.row0 + row, i = y / a.group;
        const int64_t t = u.tok + i;
        float extra = 0.0f;
        for (int32_t k = first; k < last; ++k) {
            if (!(mask_bits(a, t, i, k - q.ctx) & 1)) continue;
            const int32_t slot = slot_of(a.pg, u.s, k);
            if (slot < 0) continue;
            const float f = cache_element<E, MX>(a.cache[1], a.scales[1],
                                                 ((int64_t)slot * a.heads + u.h) * D + d);
            if ((__float_as_uint(f) & 0x7f800000u) == 0x7f800000u) extra += f;
        }
        if (extra == 0.0f) continue;
        if (part != nullptr) {
            part[x] += extra;
        } else {
            const int64_t o = (t * a.heads * a.group + u.h * a.group + y % a.group) * D + d;
            if constexpr (E::BYTES == 4) static_cast<float*>(a.out)[o] += extra;
            else static_cast<__bf16*>(a.out)[o] = (__bf16)((float)static_cast<__bf16*>(a.out)[o] + extra);
        }
    }
}

// Joins the parts of the units that crossed workers: 16 lanes per (token, query head), which all do
// the same chain of dependent loads at the same time; a whole wave for each took four times as many
// rounds of that chain (27 against 13 us for 32768 rows of 128).
template <class E, int D, class S, int WORKERS, bool SPARSE>
__global__ void __launch_bounds__(256) join_kernel(AttnArgs a) {
    constexpr int M = S::M;
    constexpr int N = D / 16;  // channels per lane
    const int lane = threadIdx.x & 15, lane0 = threadIdx.x & 48;
    const int64_t t = blockIdx.x;
    const int hq = (int)(blockIdx.y * 16 + (threadIdx.x >> 4));
    const int s = seq_of_token(a.b, t);
    const SeqInfo q = seq_info(a.b, a.pg, s);
    const int64_t i = t - q.start;
    if (i < 0 || i >= q.len || hq >= a.heads * a.group) return;
    const char* ws = static_cast<const char*>(a.ws);
    const int h = hq / a.group;
    int64_t total;
    int32_t row;
    Unit u;
    if constexpr (SPARSE) {
        u.steps = S::of_pages(a);
        const int32_t tiles = S::group_tiles(a);
        row = hq - h * a.group;
        S::place(u, a.group, row, (t * a.heads + h) * tiles * u.steps);
        total = a.b.tokens * a.heads * tiles * u.steps;
    } else {
        const int64_t* prefix = reinterpret_cast<const int64_t*>(ws);
        u.steps = (int32_t)S::of_keys(q.keys);
        const int64_t rows = (int64_t)q.len * a.group;
        row = (int32_t)(i * a.group + hq - h * a.group);
        S::place(u, rows, row, prefix[s] + h * S::of_rows(rows) * u.steps);
        total = prefix[a.b.num_seqs];
    }
    row -= u.row0;
    const Shares<WORKERS> sh(total, S::kMost);
    const int32_t w0 = sh.owner(u.first), w1 = sh.owner(u.end() - u.cost);
    if (w0 == w1) return;  // written by its worker
    auto part = [&](int32_t w) { return part_of<M, D>(a.ws, a.part_offset, w, w == w0); };
    // lane i takes the maximum and the sum of part w0 + i, 16 parts at a time
    float big = -__builtin_inff();
    for (int32_t w = w0 + lane; w <= w1; w += 16) big = __builtin_fmaxf(big, part(w)[M * D + row]);
    for (int d = 1; d < 16; d <<= 1) big = __builtin_fmaxf(big, __shfl_xor(big, d));
    const float base = big == -__builtin_inff() ? 0.0f : big;
    float sum = 0.0f, o[N];
#pragma unroll
    for (int j = 0; j < N; ++j) o[j] = 0.0f;
    for (int32_t v0 = w0; v0 <= w1; v0 += 16) {
        const int n = min(16, w1 - v0 + 1);
        float f = 0.0f;
        if (lane < n) {
            const float* p = part(v0 + lane);
            f = exp2_fast(p[M * D + row] - base);
            sum += p[M * D + M + row] * f;
        }
        constexpr int U = 4;  // rows in flight
        for (int k = 0; k < n; k += U) {
            f32x4 y[U][N / 4];
#pragma unroll
            for (int v = 0; v < U; ++v) {
                const float* p = part(v0 + min(k + v, n - 1)) + row * D + lane * 4;
#pragma unroll
                for (int j = 0; j < N / 4; ++j)
                    y[v][j] = *reinterpret_cast<const f32x4*>(p + j * 64);
            }
#pragma unroll
            for (int v = 0; v < U; ++v) {
                const float fw = __shfl(f, lane0 + min(k + v, n - 1));
                if (k + v < n)
#pragma unroll
                    for (int j = 0; j < N; ++j) o[j] = __builtin_fmaf(y[v][j / 4][j & 3], fw, o[j]);
            }
        }
    }
    for (int d = 1; d < 16; d <<= 1) sum += __shfl_xor(sum, d);
    const bool some = sum > 0.0f || sum != sum;
    const float inv = some ? 1.0f / sum : 0.0f;
    const int64_t at = t * a.heads * a.group + hq;
#pragma unroll
    for (int j = 0; j < N; j += 4) {
        const float y[4] = {o[j] * inv, o[j + 1] * inv, o[j + 2] * inv, o[j + 3] * inv};
        store_row<E, 4>(a.out, at * D + lane * 4 + j * 16, y);
    }
    if (a.lse != nullptr && lane == 0)
        a.lse[at] = some ? (big + log2_fast(sum)) * kLn2 : -__builtin_inff();
}

template <class E, int D, class S, int WORKERS, bool SPARSE>
hipError_t launch_join(const AttnArgs& a, hipStream_t st) {
    const dim3 grid((uint32_t)a.b.tokens, (uint32_t)(a.heads * a.group + 15) / 16);
    join_kernel<E, D, S, WORKERS, SPARSE><<<grid, 256, 0, st>>>(a);
    return hipGetLastError();
}

}  // namespace sc

#endif  // SHORTCONV_ATTENTION_LINE_H
