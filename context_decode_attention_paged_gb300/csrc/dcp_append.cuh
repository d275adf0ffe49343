// Device helpers shared by the kernels that append rows to the cache.
#pragma once

#include "dcp_device.cuh"
#include "dcp_internal.h"

namespace dcp {

constexpr int kCopies = 8;         // vectors of a lane in flight while copying

// Tokens of a request that are there (0 for a request whose lengths are out of range).
__device__ __forceinline__ int present(const AppendArgs& a, int b, bool* bad) {
  const int n = a.q_lens ? a.q_lens[b] : a.L;
  *bad = n < 0 || n > a.L || a.seq_lens[b] < n;
  return *bad ? 0 : n;
}

// A warp copies n vectors, vector c from src + at(c) to dst + at(c).
template <typename At>
__device__ __forceinline__ void copy_vectors(const uint4* src, uint4* dst, int n, int lane, At at) {
  uint4 v[kCopies];
  int off[kCopies];
  int c = lane;
  for (; c + 32 * (kCopies - 1) < n; c += 32 * kCopies) {
#pragma unroll
    for (int m = 0; m < kCopies; ++m) {
      off[m] = at(c + 32 * m);
      v[m] = src[off[m]];
    }
#pragma unroll
    for (int m = 0; m < kCopies; ++m) dst[off[m]] = v[m];
  }
  if (c < n) {
    // past the end the last vector again: the same value to the same place
#pragma unroll
    for (int m = 0; m < kCopies; ++m) {
      off[m] = at(min(c + 32 * m, n - 1));
      v[m] = src[off[m]];
    }
#pragma unroll
    for (int m = 0; m < kCopies; ++m) dst[off[m]] = v[m];
  }
}

}  // namespace dcp
