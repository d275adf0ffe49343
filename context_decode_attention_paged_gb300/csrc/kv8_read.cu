// Reading rows of the 8-bit cache back as bf16: value = code * 2^(s - 127), the
// product exact for every scale that dcp_kv8_append writes.
//
// Bound by HBM: one byte read and two written per value.  A warp takes a token
// and walks its row (every KV head, keys then values), a lane 8 codes at a time;
// the token's table entry and its scales come first, the codes of up to kAhead
// vectors of a lane together.  Measured (GB300, in a graph): 29,000 rows of 2 x 4
// heads of 128 (90 MB) 24 us, 3.7 TB/s; 2,700 latent rows 4.4 us.  Keys and values
// in one loop: 29 to 24 us; two tokens a warp: 27.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "dcp_device.cuh"
#include "dcp_internal.h"

namespace dcp {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kAhead = 4;          // vectors of a lane in flight

__global__ void __launch_bounds__(kThreads) kv8_read_kernel(const ReadArgs a) {
  const int lane = threadIdx.x & 31;
  const long long token = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (token >= (long long)a.B * a.n) return;
  const int b = (int)(token / a.n), i = (int)(token % a.n);
  const int S = a.seq_lens[b], start = a.starts ? a.starts[b] : 0;
  if (S < 0 || start < 0) {
    if (lane == 0) set_status(a.status, DCP_ERR_BOUNDS);
    return;
  }
  const long long t = (long long)start + i;
  if (t >= S) return;
  const int r = (int)((t / a.I) % a.N);
  const long long j = (t / ((long long)a.I * a.N)) * a.I + t % a.I, jb = j / a.bs;
  const int blk = jb < a.max_lb ? a.block_tables[((long long)r * a.B + b) * a.max_lb + jb] : -1;
  if ((unsigned)blk >= (unsigned)a.num_blocks) {
    if (lane == 0) set_status(a.status, DCP_ERR_BOUNDS);
    return;
  }
  const int per_head = a.D / 8, vecs = a.Hkv * per_head;
  const long long pool = (long long)a.num_blocks * a.bs * a.Hkv * a.D;
  const int first = a.out_k != nullptr ? 0 : vecs, last = a.out_v != nullptr ? 2 * vecs : vecs;   // keys, then values
  const long long cell = ((long long)blk * a.bs + j % a.bs) * a.Hkv * a.D;
  for (int c0 = first + lane; c0 < last; c0 += 32 * kAhead) {
    uint2 u[kAhead];
    float f[kAhead];
#pragma unroll
    for (int m = 0; m < kAhead; ++m) {
      const int c = min(c0 + 32 * m, last - 1), kind = c >= vecs, v = kind ? c - vecs : c;
      u[m] = __ldcs(reinterpret_cast<const uint2*>(a.cache + kind * pool + cell) + v);
      f[m] = scale_factor(a.scales[((long long)kind * a.num_blocks + blk) * a.Hkv + v / per_head]);
    }
#pragma unroll
    for (int m = 0; m < kAhead; ++m) {
      const int c = c0 + 32 * m, kind = c >= vecs, v = kind ? c - vecs : c;
      const uint32_t w[2] = {u[m].x, u[m].y};
      uint32_t o[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        uint32_t pair;
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(pair) : "h"((uint16_t)(w[k / 2] >> (16 * (k & 1)))));
        const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&pair));
        const __nv_bfloat162 q = __floats2bfloat162_rn(x.x * f[m], x.y * f[m]);
        o[k] = *reinterpret_cast<const uint32_t*>(&q);
      }
      if (c < last) {
        uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(kind ? a.out_v : a.out_k) + token * a.Hkv * a.D);
        __stcs(dst + v, make_uint4(o[0], o[1], o[2], o[3]));
      }
    }
  }
}

}  // namespace

cudaError_t launch_kv8_read(const ReadArgs& a) {
  const long long blocks = ((long long)a.B * a.n + kWarps - 1) / kWarps;
  kv8_read_kernel<<<(unsigned)blocks, kThreads, 0, a.stream>>>(a);
  return cudaGetLastError();
}

}  // namespace dcp
