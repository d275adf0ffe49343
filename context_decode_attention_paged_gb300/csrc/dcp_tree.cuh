// Device-side helpers of the drafted-tree attention kernels.
//
// Request b holds n_b nodes in its last n_b positions; its context is the
// positions below base = S_b - n_b, seen by every row.  In a shard, tokens are
// dense in global order, so the shard's keys are a run of context keys
// [0, ctx) followed by the nodes it owns.
#pragma once

#include <stdint.h>

#include "dcp_device.cuh"

namespace dcp {

struct TreeReq {
  int n;             // nodes
  long long base;    // first node's position
  bool bad;          // lengths out of range: the request is skipped
};

__device__ __forceinline__ TreeReq tree_request(const int32_t* seq_lens, const int32_t* q_lens, int Lq, int b) {
  const int S = seq_lens[b];
  TreeReq t;
  t.n = q_lens ? q_lens[b] : Lq;
  t.bad = t.n < 0 || t.n > Lq || S < t.n;
  if (t.bad) t.n = 0;
  t.base = t.bad ? 0 : (long long)S - t.n;
  return t;
}

// Whether the mask row (uint32 words) has node j's bit.
__device__ __forceinline__ bool tree_bit(const uint32_t* row, int j) { return (row[j >> 5] >> (j & 31)) & 1u; }

}  // namespace dcp
