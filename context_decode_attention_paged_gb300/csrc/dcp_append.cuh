// Device helpers shared by the kernels that append rows to the cache.
#pragma once

#include "dcp_device.cuh"
#include "dcp_internal.h"

namespace dcp {

constexpr int kCopies = 8;         // vectors of a lane in flight while copying
constexpr int kScan = 1024;        // requests whose token counts a block sums

// Tokens of a request that are there (0 for a request whose lengths are out of range).
__device__ __forceinline__ int present(const AppendArgs& a, int b, bool* bad) {
  const int n = a.q_lens ? a.q_lens[b] : a.L;
  *bad = n < 0 || n > a.L || a.seq_lens[b] < n;
  return *bad ? 0 : n;
}

// ends[b] = tokens of requests 0 .. b, for all b < B <= kScan (whole block of kThreads).
template <int kThreads>
__device__ __forceinline__ void sum_counts(const AppendArgs& a, int* ends) {
  constexpr int kPer = kScan / kThreads;
  __shared__ int warps[kThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31;
  int sums[kPer], run = 0;
#pragma unroll
  for (int e = 0; e < kPer; ++e) {
    const int b = tid * kPer + e;
    bool bad = false;
    if (b < a.B) run += present(a, b, &bad);
    if (bad && blockIdx.x == 0) set_status(a.status, DCP_ERR_BOUNDS);
    sums[e] = run;
  }
  int inc = run;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += v;
  }
  if (lane == 31) warps[tid >> 5] = inc;
  __syncthreads();
  int before = inc - run;
  for (int w = 0; w < tid >> 5; ++w) before += warps[w];
#pragma unroll
  for (int e = 0; e < kPer; ++e)
    if (tid * kPer + e < a.B) ends[tid * kPer + e] = before + sums[e];
  __syncthreads();
}

// (request, index) of the summed-up token, by bisection of the sums
__device__ __forceinline__ int find_token(const int* ends, int B, unsigned token, int* i) {
  int b = 0;
  for (int hi = B - 1; b < hi;) {
    const int mid = (b + hi) >> 1;
    if ((unsigned)ends[mid] > token) hi = mid;
    else b = mid + 1;
  }
  *i = (int)token - (b > 0 ? ends[b - 1] : 0);
  return b;
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
