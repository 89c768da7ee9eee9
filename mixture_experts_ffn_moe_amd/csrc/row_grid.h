// Launches of one workgroup per row.  (Not in moe_common.h: see lds_barrier.h.)
#pragma once

#include <hip/hip_runtime.h>

namespace moe {

// Grids of one workgroup per row (token or route).  A dimension of a launch holds
// fewer than 2^32 work-items, which 2^24 workgroups of 256 reach: rows past
// kGridRows lie along y.  The last y has workgroups past the last row.
constexpr int kGridRows = 1 << 20;
inline dim3 row_grid(long long rows) {
  return dim3((unsigned)(rows < kGridRows ? rows : kGridRows), (unsigned)((rows + kGridRows - 1) / kGridRows));
}
__device__ __forceinline__ int grid_row() { return (int)(blockIdx.y * kGridRows + blockIdx.x); }

}  // namespace moe
