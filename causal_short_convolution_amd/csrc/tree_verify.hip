// The ShortConv K/V step for a tree of drafted tokens (shortconv_kv_verify_tree). The row math and
// the cache row formats are those of the chain (device_common.h), so a tree that is a chain gives
// the same bits. Bound by the rows' bytes: 256 trees of 4-32 tokens, 16 heads of 128, bf16, W = 4 in
// 43 us (4.5 TB/s).
#include "cache_device.h"

namespace sc {
namespace {

constexpr int kBlock = 256;

// One token per workgroup row: each lane owns 16 bytes of the token's K or V row, gathers the
// window rows along the ancestors, and writes the cache row and the snapshot.
template <class E, int D, int W, bool MX>
__global__ void __launch_bounds__(kBlock) verify_tree_kernel(StepArgs a, VerifyArgs va,
                                                             TreeArgs ta) {
    constexpr int VEC = E::VEC;
    constexpr int LPH = D / VEC;
    constexpr int R = W - 1;
    const Batch b = {a.cu, nullptr, a.tokens, a.num_seqs};
    const int64_t t = blockIdx.x;
    const int s = seq_of_token(b, t);
    const int64_t start = uniform((int64_t)clamp_tok(a.cu[s], a.tokens));
    const int64_t end = uniform((int64_t)clamp_tok(a.cu[s + 1], a.tokens));
    if (t < start || t >= end) return;
    const int32_t i = (int32_t)(t - start);

    if (ta.mask != nullptr && blockIdx.y == 0 && threadIdx.x == 0) {
        // one walk to the root: a token's ancestors have lower indices
        auto parent = [&](int32_t j) {
            const int32_t p = ta.parents[start + j];
            return p < j ? p : -1;
        };
        int32_t j = i;
        for (int w = ta.words - 1; w >= 0; --w) {
            uint64_t bits = 0;
            while (j >= 0 && (j >> 6) > w) j = parent(j);  // past the mask
            for (; j >= 0 && (j >> 6) == w; j = parent(j)) bits |= 1ull << (j & 63);
            ta.mask[t * ta.words + w] = (int64_t)bits;
        }
    }
    const int lane = blockIdx.y * kBlock + threadIdx.x;
    if (lane >= 2 * a.lanes_per_tensor) return;
    const int tensor = lane >= a.lanes_per_tensor;
    const int c = lane - tensor * a.lanes_per_tensor;
    const int h = c / LPH;
    const int d0 = (c - h * LPH) * VEC;
    const int64_t row_bytes = (int64_t)a.heads * D * E::BYTES;
    const uint32_t lane_off = (uint32_t)(((int64_t)h * D + d0) * E::BYTES);
    const char* x = static_cast<const char*>(pick(a.x, tensor));
    const int64_t stride_bytes = pick(a.x_stride, tensor) * E::BYTES;
    const char* state = static_cast<const char*>(pick(a.state, tensor));
    const int32_t idx = uniform(a.state_idx ? a.state_idx[s] : s);
    const bool slot_ok = R > 0 && state != nullptr && idx >= 0 && idx < a.num_state_slots;

    LaneParams<E, W> p;
    load_params<E, W>(pick(a.taps, tensor), pick(a.gamma, tensor), a.heads, D, h, d0, p);
    uint4 raw[W];
    float win[W][VEC];
    int32_t at = i;
    int32_t left = R;  // state rows not yet used
#pragma unroll
    for (int k = W - 1; k >= 0; --k) {
        raw[k] = make_uint4(0, 0, 0, 0);
        if (at >= 0) {
            raw[k] = ldrow_keep(x + (start + at) * stride_bytes, lane_off);
            const int32_t up = uniform(ta.parents[start + at]);
            at = up < at ? up : -1;
        } else {
            --left;
            if (slot_ok) raw[k] = ldrow_keep(state + ((int64_t)idx * R + left) * row_bytes, lane_off);
        }
        E::widen(raw[k], win[k]);
    }
    float o[VEC];
    fused_row<E, W, LPH>(win, 0, p, a.eps, 1.0f / (float)D, o);
    const typename SinkFor<E, MX>::type sink(a, tensor, h, d0, D);
    sink.put(uniform(a.slot[t]), true, o);
    char* snap = static_cast<char*>(pick(va.snap, tensor));
    if (R > 0 && snap != nullptr && i < va.max_tokens) {
        char* dst = snap + ((int64_t)s * va.max_tokens + i) * R * row_bytes;
#pragma unroll
        for (int k = 0; k < R; ++k) strow(dst + k * row_bytes, lane_off, raw[k + 1]);
    }
}

template <class E, int D, int W, bool MX>
hipError_t launch(const StepArgs& a, const VerifyArgs& va, const TreeArgs& ta, hipStream_t st) {
    const dim3 grid((uint32_t)a.tokens, (uint32_t)a.lane_blocks);
    verify_tree_kernel<E, D, W, MX><<<grid, kBlock, 0, st>>>(a, va, ta);
    return hipGetLastError();
}

template <class E, int D, bool MX>
hipError_t by_width(const StepArgs& a, const VerifyArgs& va, const TreeArgs& ta, int W,
                    hipStream_t st) {
    switch (W) {
        case 1: return launch<E, D, 1, MX>(a, va, ta, st);
        case 2: return launch<E, D, 2, MX>(a, va, ta, st);
        case 3: return launch<E, D, 3, MX>(a, va, ta, st);
        case 4: return launch<E, D, 4, MX>(a, va, ta, st);
        case 5: return launch<E, D, 5, MX>(a, va, ta, st);
        case 6: return launch<E, D, 6, MX>(a, va, ta, st);
        case 7: return launch<E, D, 7, MX>(a, va, ta, st);
        default: return launch<E, D, 8, MX>(a, va, ta, st);
    }
}

template <class E, bool MX>
hipError_t by_dim(const StepArgs& a, const VerifyArgs& va, const TreeArgs& ta, int D, int W,
                  hipStream_t st) {
    if (D == 64) return by_width<E, 64, MX>(a, va, ta, W, st);
    if (D == 128) return by_width<E, 128, MX>(a, va, ta, W, st);
    return by_width<E, 256, MX>(a, va, ta, W, st);
}

}  // namespace

hipError_t launch_verify_tree(const StepArgs& a, const VerifyArgs& va, const TreeArgs& ta, bool mx,
                              int dtype, int D, int W, hipStream_t st) {
    if (dtype == 0)
        return mx ? by_dim<F32, true>(a, va, ta, D, W, st) : by_dim<F32, false>(a, va, ta, D, W, st);
    return mx ? by_dim<BF16, true>(a, va, ta, D, W, st) : by_dim<BF16, false>(a, va, ta, D, W, st);
}

}  // namespace sc
