// Eviction from the cache by accumulated attention weight (shortconv_cache_evict): one workgroup
// per (sequence, head) finds the entries to keep and pairs the holes with the entries that fill
// them; a second launch moves the K and V rows.
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

__global__ void __launch_bounds__(kPlan) evict_plan_kernel(EvictArgs a) {
    __shared__ uint32_t hist[258];
    __shared__ int sums[kPlan / 64 + 1];
    const int h = blockIdx.x, s = blockIdx.y, tid = threadIdx.x;
    const int32_t n = entries_of(a, s);
    const int64_t head = (int64_t)s * a.heads + h;
    const float* scores = a.scores + head * a.capacity;
    const int32_t* positions = a.positions + head * a.capacity;
    float* scores_out = a.scores_out + head * a.capacity;
    int32_t* positions_out = a.positions_out + head * a.capacity;
    const int32_t kept = min(n, a.budget);
    int32_t* dst = a.dst + head * a.max_moves;
    int32_t* src = a.src + head * a.max_moves;
    const int64_t late = (int64_t)a.seen[s] - a.recent;
    auto key = [&](int j) {
        const int32_t pos = positions[j];
        if (pos < a.sinks || pos >= late) return 0xffffffffu;
        const float f = scores[j];
        return f != f ? 0u : order_key(f);
    };
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
            if (hole) dst[hi] = j;
            if (move) src[mi] = j;
            tied += n_tie;
            holes += n_hole;
            movers += n_move;
        }
        __syncthreads();
    }
    if (tid == 0) a.count[head] = holes;
    // the entries that stay, then the ones that move (their sources lie at or past the budget)
    for (int j = tid; j < kept; j += kPlan) {
        const float f = scores[j];
        const int32_t p = positions[j];
        scores_out[j] = f;
        positions_out[j] = p;
    }
    __syncthreads();
    for (int j = tid; j < holes; j += kPlan) {
        const int32_t from = src[j], to = dst[j];
        scores_out[to] = scores[from];
        positions_out[to] = positions[from];
    }
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
    evict_plan_kernel<<<dim3((uint32_t)a.heads, (uint32_t)a.num_seqs), kPlan, 0, st>>>(a);
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
