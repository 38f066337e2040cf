// Eviction from the cache by accumulated attention weight (shortconv_cache_evict): one workgroup
// per (sequence, head) finds the entries to keep and pairs the holes with the entries that fill
// them; a second launch moves the K and V rows. Ranking is a chain of meetings of the workgroup, not
// bytes: 512 heads of 4100 entries, 16 dropped, take 24 us (the bytes 7), 64 heads of up to 32768 to 4096
// entries 40-47 us; the move of the latter's rows runs at 5 TB/s.
#include "cache_device.h"

namespace sc {
namespace {

constexpr int kPlan = 1024;  // threads that rank one head's entries
constexpr int kMove = 256;

__device__ inline int32_t entries_of(const EvictArgs& a, int s) {
    int64_t n = a.lens[s];
    const int64_t cap = (int64_t)a.pg.max_blocks << a.pg.shift;
    if (n > a.capacity) n = a.capacity;
    if (n > cap) n = cap;
    return n < 0 ? 0 : (int32_t)n;
}

// One head of one sequence.
struct Head {
    const float* scores;
    const int32_t* positions;
    float* scores_out;
    int32_t* positions_out;
    int32_t* dst;
    int32_t* src;
    int64_t index;
    int64_t late;  // positions from here on are among the recent ones
    int32_t sinks;
    __device__ Head(const EvictArgs& a, int s, int h) {
        index = (int64_t)s * a.heads + h;
        scores = a.scores + index * a.capacity;
        positions = a.positions + index * a.capacity;
        scores_out = a.scores_out + index * a.capacity;
        positions_out = a.positions_out + index * a.capacity;
        dst = a.dst + index * a.max_moves;
        src = a.src + index * a.max_moves;
        late = (int64_t)a.seen[s] - a.recent;
        sinks = a.sinks;
    }
    // Protected entries above all numbers, NaN below them; 0 is no entry.
    __device__ uint32_t key(float f, int32_t pos) const {
        const uint32_t k = f != f ? 1u : order_key(f);
        const bool safe = (pos < sinks) | (pos >= late);  // (no branch for each entry)
        return safe ? 0xffffffffu : k;
    }
    // Scores and positions of the kept entries: those that stay (unless the output is the input),
    // then those that move, whose sources lie at or past the budget.
    __device__ void write(int32_t kept, int32_t holes) const {
        if (scores_out != scores || positions_out != positions) {
            constexpr int U = 4;  // loads in flight
            for (int j0 = threadIdx.x; j0 < kept; j0 += U * blockDim.x) {
                float f[U];
                int32_t p[U];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int j = min(j0 + u * (int)blockDim.x, kept - 1);
                    f[u] = scores[j];
                    p[u] = positions[j];
                }
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int j = j0 + u * (int)blockDim.x;
                    if (j < kept) {
                        scores_out[j] = f[u];
                        positions_out[j] = p[u];
                    }
                }
            }
        }
        __syncthreads();
        for (int j = threadIdx.x; j < holes; j += blockDim.x) {
            const int32_t from = src[j], to = dst[j];
            scores_out[to] = scores[from];
            positions_out[to] = positions[from];
        }
    }
};

// Up to KPT entries per thread, entry i * THREADS + tid in register i, ranked there. The order of the
// entries is (i, wave, lane): places within a list come from a wave's ballots and a scan over the
// counts of all (i, wave).
template <int THREADS, int KPT>
__global__ void __launch_bounds__(THREADS) evict_plan_kernel(EvictArgs a) {
    constexpr int WAVES = THREADS / 64;
    __shared__ KthScratch scratch;
    __shared__ int sums[WAVES + 1];
    __shared__ int first[2][KPT * WAVES];
    const int h = blockIdx.x, s = blockIdx.y, tid = threadIdx.x;
    const int wave = uniform(tid >> 6);
    const int32_t n = entries_of(a, s);
    const Head head(a, s, h);
    const int32_t kept = min(n, a.budget);
    int holes = 0;
    if (n > a.budget && kept > 0) {
        uint32_t key[KPT];
        {
            float f[KPT];
            int32_t p[KPT];
#pragma unroll
            for (int i = 0; i < KPT; ++i) {
                const int j = min(i * THREADS + tid, n - 1);
                f[i] = head.scores[j];
                p[i] = head.positions[j];
            }
#pragma unroll
            for (int i = 0; i < KPT; ++i) key[i] = i * THREADS + tid < n ? head.key(f[i], p[i]) : 0u;
        }
        uint32_t threshold;
        int ties, total;
        kth_of_registers<THREADS, KPT>(key, n, kept, scratch, threshold, ties);
        auto scan = [&](int list) {
            __syncthreads();
            static_assert(KPT * WAVES <= THREADS, "one count per thread");
            const int c = tid < KPT * WAVES ? first[list][tid] : 0;
            const int x = block_prefix(c, sums, total);
            if (tid < KPT * WAVES) first[list][tid] = x;
            __syncthreads();
            return total;
        };
        if (ties > 0) {  // the lowest of the equal entries
            put_counts<WAVES, KPT>(first[0], [&](int i) {
                return key[i] == threshold;
            });
            scan(0);
        }
#pragma unroll
        for (int i = 0; i < KPT; ++i) {  // from here on key[i] is 1 for an entry to keep
            bool keep = key[i] > threshold;
            if (ties > 0) {
                const bool tie = key[i] == threshold;
                keep |= tie && first[0][i * WAVES + wave] + lanes_below(__ballot(tie)) < ties;
            }
            key[i] = keep;
        }
        // Holes and movers of register i in the wave, as masks; scalar work but for one comparison.
        auto split = [&](int i, uint64_t& hole, uint64_t& move) {
            const uint64_t m = __ballot(key[i] != 0);
            const int n_low = kept - (i * THREADS + wave * 64);  // lanes below the budget
            const uint64_t low = n_low >= 64 ? ~0ull : n_low <= 0 ? 0ull : (1ull << n_low) - 1;
            hole = ~m & low;
            move = m & ~low;
        };
        // Both counts in one word: there are as many of each, at most half of 65536 entries.
        static_assert(THREADS * KPT <= 65536, "16 bits each");
#pragma unroll
        for (int i = 0; i < KPT; ++i) {
            uint64_t hole, move;
            split(i, hole, move);
            first[1][i * WAVES + wave] =
                __builtin_popcountll(hole) | __builtin_popcountll(move) << 16;
        }
        holes = scan(1) & 0xffff;
#pragma unroll
        for (int i = 0; i < KPT; ++i) {
            uint64_t hole, move;
            split(i, hole, move);
            if ((hole | move) == 0) continue;
            const uint32_t at = (uint32_t)first[1][i * WAVES + wave];
            const int j = i * THREADS + tid;
            if (hole >> (tid & 63) & 1) head.dst[(at & 0xffff) + lanes_below(hole)] = j;
            if (move >> (tid & 63) & 1) head.src[(at >> 16) + lanes_below(move)] = j;
        }
        __syncthreads();
    }
    if (tid == 0) a.count[head.index] = holes;
    head.write(kept, holes);
}

// More entries than registers hold: the keys are read again for every 8 bits of the threshold and
// once more, in order, to split them.
__global__ void __launch_bounds__(kPlan) evict_plan_long_kernel(EvictArgs a) {
    __shared__ uint32_t hist[258];
    __shared__ int sums[kPlan / 64 + 1];
    const int h = blockIdx.x, s = blockIdx.y, tid = threadIdx.x;
    const int32_t n = entries_of(a, s);
    const Head head(a, s, h);
    const int32_t kept = min(n, a.budget);
    auto key = [&](int j) { return head.key(head.scores[j], head.positions[j]); };
    int holes = 0, movers = 0;
    if (n > a.budget && kept > 0) {
        uint32_t threshold;
        int ties;
        kth_largest(key, n, kept, hist, threshold, ties);
        int tied = 0;
        for (int j0 = 0; j0 < n; j0 += kPlan) {
            const int j = j0 + tid;
            const uint32_t x = j < n ? key(j) : 0;
            const bool tie = j < n && x == threshold;
            int n_tie, n_hole, n_move;
            const int rank = tied + block_prefix(tie, sums, n_tie);
            const bool keep = j < n && (x > threshold || (tie && rank < ties));
            const bool hole = j < kept && !keep;
            const bool move = j >= kept && keep;
            const int hi = holes + block_prefix(hole, sums, n_hole);
            const int mi = movers + block_prefix(move, sums, n_move);
            if (hole) head.dst[hi] = j;
            if (move) head.src[mi] = j;
            tied += n_tie;
            holes += n_hole;
            movers += n_move;
        }
        __syncthreads();
    }
    if (tid == 0) a.count[head.index] = holes;
    head.write(kept, holes);
}

// Copies the moved rows: BYTES = one head's row in one tensor, in 16-byte pieces, plus its scale
// bytes for MXFP8 rows.
template <int BYTES, int SCALES>
__global__ void __launch_bounds__(kMove) evict_move_kernel(EvictArgs a) {
    constexpr int LANES = BYTES / 16;
    const int h = blockIdx.y, s = blockIdx.z;
    const int64_t head = (int64_t)s * a.heads + h;
    if (h == 0 && blockIdx.x == 0 && threadIdx.x == 0)
        a.lens_out[s] = min(entries_of(a, s), a.budget);
    const int32_t count = a.count[head];
    const int piece = threadIdx.x % LANES;
    const int per = kMove / LANES;
    for (int32_t j = blockIdx.x * per + threadIdx.x / LANES; j < count; j += gridDim.x * per) {
        const int32_t from = slot_of(a.pg, s, a.src[head * a.max_moves + j]);
        const int32_t to = slot_of(a.pg, s, a.dst[head * a.max_moves + j]);
        if (from < 0 || to < 0) continue;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            char* rows = static_cast<char*>(a.cache[i]);
            const uint4 r = *reinterpret_cast<const uint4*>(
                rows + ((int64_t)from * a.heads + h) * BYTES + piece * 16);
            *reinterpret_cast<uint4*>(rows + ((int64_t)to * a.heads + h) * BYTES + piece * 16) = r;
            if (SCALES > 0 && piece < SCALES) {
                char* sc = static_cast<char*>(a.scales[i]);
                sc[((int64_t)to * a.heads + h) * SCALES + piece] =
                    sc[((int64_t)from * a.heads + h) * SCALES + piece];
            }
        }
    }
}

template <int BYTES, int SCALES>
void move(const EvictArgs& a, hipStream_t st) {
    constexpr int per = kMove / (BYTES / 16);
    int64_t blocks = ((int64_t)a.max_moves + per - 1) / per;
    blocks = blocks < 1 ? 1 : (blocks > 64 ? 64 : blocks);
    const dim3 grid((uint32_t)blocks, (uint32_t)a.heads, (uint32_t)a.num_seqs);
    evict_move_kernel<BYTES, SCALES><<<grid, kMove, 0, st>>>(a);
}

}  // namespace

hipError_t launch_cache_evict(const EvictArgs& a, bool mx, int dtype, int D, hipStream_t st) {
    const dim3 grid((uint32_t)a.heads, (uint32_t)a.num_seqs);
    const int64_t cap = (int64_t)a.pg.max_blocks << a.pg.shift;
    const int64_t most = a.capacity < cap ? a.capacity : cap;  // entries of a head
    // Few threads per head while their registers hold it: a bit costs every wave the meeting.
    if (most <= 8 * 256) evict_plan_kernel<256, 8><<<grid, 256, 0, st>>>(a);
    else if (most <= 20 * 256) evict_plan_kernel<256, 20><<<grid, 256, 0, st>>>(a);
    else if (most <= 16 * 1024) evict_plan_kernel<1024, 16><<<grid, 1024, 0, st>>>(a);
    else if (most <= 32 * 1024) evict_plan_kernel<1024, 32><<<grid, 1024, 0, st>>>(a);
    else if (most <= 64 * 1024) evict_plan_kernel<1024, 64><<<grid, 1024, 0, st>>>(a);
    else evict_plan_long_kernel<<<grid, kPlan, 0, st>>>(a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    if (mx) {
        if (D == 64) move<64, 2>(a, st);
        else if (D == 128) move<128, 4>(a, st);
        else move<256, 8>(a, st);
    } else {
        const int bytes = D * (dtype == 0 ? 4 : 2);
        if (bytes == 128) move<128, 0>(a, st);
        else if (bytes == 256) move<256, 0>(a, st);
        else if (bytes == 512) move<512, 0>(a, st);
        else move<1024, 0>(a, st);
    }
    return hipGetLastError();
}

}  // namespace sc
