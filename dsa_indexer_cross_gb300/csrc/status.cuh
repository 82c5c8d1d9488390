// The status words of calls that are one kernel: written by a block that checks every item (sole), or
// cleared by a kernel before and added to.
#pragma once

#include <cstdint>

#include "kernels.h"
#include "ptx.cuh"

namespace dsa {

__device__ __forceinline__ void report(uint32_t* status, bool sole, uint32_t bits) {
  if (sole) return;
  atomicOr(status, bits);
  atomicAdd(status + 1, 1u);
}
static __global__ void clear_status_kernel(uint32_t* status) {
  grid_trigger();
  grid_wait();
  status[threadIdx.x] = 0u;
}
static inline cudaError_t clear_status(uint32_t* status, cudaStream_t st) {
  return launch_pdl(clear_status_kernel, dim3(1), 2, 0, st, 1, status);
}
// Block 0 of a call that writes the status words itself: check(i) gives item i's error bits.
template <typename F>
__device__ __forceinline__ void sole_status(uint32_t* status, int n, F check) {
  __shared__ uint32_t s_bits, s_count;
  if (threadIdx.x == 0) s_bits = s_count = 0u;
  __syncthreads();
  uint32_t bits = 0, count = 0;
  int i = threadIdx.x;
  for (; i + 7 * static_cast<int>(blockDim.x) < n; i += 8 * blockDim.x) {
#pragma unroll
    for (int u = 0; u < 8; ++u) {        // (eight items' loads in flight)
      const uint32_t e = check(i + u * blockDim.x);
      bits |= e;
      count += e ? 1u : 0u;
    }
  }
  for (; i < n; i += blockDim.x) {
    const uint32_t e = check(i);
    bits |= e;
    count += e ? 1u : 0u;
  }
  if (bits) {
    atomicOr(&s_bits, bits);
    atomicAdd(&s_count, count);
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    status[0] = s_bits;
    status[1] = s_count;
  }
}

}  // namespace dsa
