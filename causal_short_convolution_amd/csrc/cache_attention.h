// Geometry of the attention kernels that the host (workspace sizes, launches) and the device share.
#pragma once

#include <stdint.h>

namespace sc {

// Workgroups that share out the steps, a multiple of the 8 XCDs: two on each of the 256 CUs, one
// where a wave needs more than half of a SIMD's registers.
constexpr int workers_per_cu(int head_dim) { return head_dim <= 128 ? 2 : 1; }
constexpr int workers(int head_dim) { return 256 * workers_per_cu(head_dim); }

// Row tiles of 16 per unit, from the rows of an average sequence (or token). Rows that do not fit a
// unit make another, which reads the keys again.
inline int row_tiles(int64_t rows) { return rows <= 16 ? 1 : 2; }

}  // namespace sc
