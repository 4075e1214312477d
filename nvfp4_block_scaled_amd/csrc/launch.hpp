// Launches of more workgroups than one dimension takes.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace nvfp4 {

// Along one dimension the runtime counts a launch's threads in 32 bits and drops
// the rest without an error, so past 2^22 workgroups (of at most 512 threads) they
// go on along the next.
constexpr int kRowShift = 22;

// A launch of n workgroups, up to 2^31 - 1. Those that it numbers from n on are
// surplus and leave.
inline dim3 row_grid(int64_t n) {
  const int64_t row = int64_t(1) << kRowShift;
  return n <= row ? dim3((unsigned)n) : dim3((unsigned)row, (unsigned)((n + row - 1) / row));
}

// A workgroup's number in it.
__device__ __forceinline__ uint32_t row_workgroup() { return (blockIdx.y << kRowShift) + blockIdx.x; }

}  // namespace nvfp4
