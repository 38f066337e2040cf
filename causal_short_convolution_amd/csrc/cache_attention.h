// Geometry of the attention kernels that the host (workspace sizes, launches) and the device share.
#pragma once

#include <stdint.h>

namespace sc {

// Workgroups that share out the steps, a multiple of the 8 XCDs: two on each of the 256 CUs; one
// where the workgroup needs more than half of the CU's LDS or registers.
constexpr int kWorkers = 512;
constexpr int wide_workers(int waves, int head_dim) {
    return waves == 4 && head_dim <= 128 ? 768 : 256;
}

// How the query rows of a unit are held: waves = 0, every wave of a workgroup holds all rows, 16 x
// tiles, and takes keys of its own (cache_attention.hip); else the waves split the rows, 16 x
// tiles each, and share the keys (wide_attention.hip).
struct AttnShape {
    int waves;
    int tiles;
    int rows() const { return 16 * tiles * (waves ? waves : 1); }
    int worker_count(int head_dim) const {
        return waves ? wide_workers(waves, head_dim) : kWorkers;
    }
};

// The shape for the rows of an average sequence (or token). Rows past a unit's make another unit,
// which reads the keys again; rows that stay empty cost products and registers.
inline AttnShape attention_shape(bool tree, int64_t rows, int element_bytes, int head_dim) {
    const bool wide = tree && element_bytes == 2;
    if (rows <= 16 || (head_dim > 128 && !wide)) return {0, 1};
    if ((rows <= 32 && head_dim <= 128) || !wide) return {0, 2};
    if (rows <= 64) return {4, 1};
    if (rows <= 128 || head_dim > 128) return {8, 1};
    return rows > 256 && rows <= 384 ? AttnShape{8, 3} : AttnShape{8, 2};
}

}  // namespace sc
