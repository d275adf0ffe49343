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

// Which of the shard's keys [j0, j0 + 32) a row sees, as bits: its context
// keys, and the nodes that the row's mask words have (row null: none); keys at
// or past ke are not there.  A shard's keys come in runs of I consecutive
// positions, so the bits of a run are one cut out of the mask words.
__device__ __forceinline__ uint32_t tree_sees32(const uint32_t* row, int words, int ctx, int ke, long long base, int r,
                                                int I, int N, int j0) {
  const int c = min(max(min(ctx, ke) - j0, 0), 32), e = min(max(ke - j0, 0), 32);   // context below c, nodes in [c, e)
  uint32_t sees = c == 32 ? 0xffffffffu : (1u << c) - 1u;
  if (row == nullptr) return sees;
  int left = 0, node = 0;                    // of the run at k
  for (int k = c; k < e;) {
    if (left == 0) {
      const int jj = j0 + k;
      node = (int)(global_pos(jj, r, I, N) - base);
      left = N == 1 ? e - k : min(I - jj % I, e - k);
    }
    const int wi = node >> 5;
    const uint32_t lo = __ldg(row + wi), hi = wi + 1 < words ? __ldg(row + wi + 1) : 0u;
    uint32_t bits = __funnelshift_r(lo, hi, node & 31);
    if (left < 32) bits &= (1u << left) - 1u;
    sees |= bits << k;
    k += left;
    left = 0;
  }
  return sees;
}

// Replace the entries of a 16-byte piece of bf16 values that are not finite by
// 0; true if there were any.
__device__ __forceinline__ bool drop_non_finite(uint4& x) {
  uint32_t* w = &x.x;
  bool any = false;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if ((w[e] & 0x7f80u) == 0x7f80u) w[e] &= 0xffff0000u, any = true;
    if ((w[e] & 0x7f800000u) == 0x7f800000u) w[e] &= 0x0000ffffu, any = true;
  }
  return any;
}

}  // namespace dcp
