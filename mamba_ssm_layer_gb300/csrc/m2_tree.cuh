// m2_tree.cuh -- trees of drafted tokens (include/mamba2.h): which nodes stand
// above a node, as one 64-bit word.
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

#include "m2_common.cuh"
#include "m2_kernels.h"

namespace m2 {

// The tree of one sequence in a warp: lane l gets the masks of nodes l and l + 32,
// bit j = node j is the node itself or stands above it; 0 for a node that is not
// part of the tree.  A parent's index is below its child's, so the bits of a mask
// in ascending order are the path.  Every step doubles the distance looked up.
// All lanes call it.
__device__ __forceinline__ void tree_masks(const int32_t* parent, int n, int lane, uint64_t (&m)[2]) {
  const int slots = n > 32 ? 2 : 1;
  int up[2];  // the node's ancestor at the current distance, itself at the end of the path; 64: not a path
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int r = lane + 32 * k;
    const int p = r < n ? parent[r] : -2;
    const bool in = p >= -1 && p < r;
    up[k] = !in ? 64 : p < 0 ? r : p;
    m[k] = in ? 1ull << r : 0ull;
  }
  for (int d = 1; d < n; d *= 2) {
    uint64_t nm[2];
    int nu[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      nm[k] = m[k], nu[k] = up[k];
      if (k >= slots) continue;  // (the same for all lanes)
      uint64_t x = __shfl_sync(0xffffffffu, m[0], up[k] & 31);
      int y = __shfl_sync(0xffffffffu, up[0], up[k] & 31);
      if (slots == 2) {
        const uint64_t x1 = __shfl_sync(0xffffffffu, m[1], up[k] & 31);
        const int y1 = __shfl_sync(0xffffffffu, up[1], up[k] & 31);
        if (up[k] & 32) x = x1, y = y1;
      }
      if (up[k] < 64) nm[k] |= x, nu[k] = y;
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) m[k] = nm[k], up[k] = nu[k];
  }
#pragma unroll
  for (int k = 0; k < 2; ++k)
    if (up[k] >= 64) m[k] = 0ull;
}
// The mask of node r, by the warp that holds them (all lanes call it).
__device__ __forceinline__ uint64_t tree_mask_of(const uint64_t (&m)[2], int r) {
  const uint64_t a = __shfl_sync(0xffffffffu, m[0], r & 31), b = __shfl_sync(0xffffffffu, m[1], r & 31);
  return r & 32 ? b : a;
}

}  // namespace m2
