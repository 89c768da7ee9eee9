// Workgroup barrier of the pipelined kernels (4-bit products, router gradients).
// It is not in moe_common.h, whose text the w13 GEMM's traffic counters belong to:
// bench.py reports them only while the sources that GEMM is built from are those
// the counters were taken on.
#pragma once

#include <hip/hip_runtime.h>

namespace moe {

// A barrier that orders LDS accesses and leaves loads in flight (the one of
// __syncthreads waits for them).
__device__ __forceinline__ void lds_barrier() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

}  // namespace moe
