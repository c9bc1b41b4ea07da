// Grids of the decoder operators' kernels.  A launch holds fewer than 2^32 threads
// along an axis, so more workgroups than 2^21 (of up to 1024 threads) are laid out in
// rows of as many; the last row's spare ones return at once.
#pragma once

#include <hip/hip_runtime.h>

namespace lstm {

constexpr long long kGridRow = 1ll << 21;  // a multiple of the 8 XCDs

inline dim3 grid_of(long long blocks) {
  return blocks <= kGridRow ? dim3((unsigned)blocks) : dim3(kGridRow, (unsigned)((blocks + kGridRow - 1) / kGridRow));
}

// This workgroup's number; at least the launch's count of them for a spare one.
__device__ __forceinline__ unsigned grid_block() { return blockIdx.y * gridDim.x + blockIdx.x; }

}  // namespace lstm
