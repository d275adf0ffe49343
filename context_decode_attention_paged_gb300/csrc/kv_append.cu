// Appending keys and values to the sharded cache with the rotary position
// applied on the way, and rotating the queries of the same tokens.
//
// "Context Parallel Guide", section "Overview": a token's KV is stored once, by
// the shard that owns its position (interleave rule, section "Decode Context
// Parallel"); the cell is found as in kv_write.cu.
//
// Mathematics.  Pair k of a row at position p turns by p f_k.  The table holds
// steps[k] = frac(f_k / 2 pi) 2^64, so the 64-bit product p * steps[k] wraps at
// whole turns and its top 32 bits are the phase to 2^-32 of a turn, at any
// position; cos and sin are evaluated in fp32 from it (about 1e-7), the
// rotation runs in fp32 and each value is rounded to bf16 once.
//
// The bound is HBM (every row read and written once) or, for a decode step,
// the launch and three dependent loads.  One block takes one token and up to
// kThreads * kUnits units of its rows; a unit is what one thread loads, turns
// and stores at a time: a 16-byte vector of 8 unrotated values, a vector of 4
// interleaved pairs, or the two vectors of 8 pairs in the half layout.  A
// thread issues all of its loads before the block meets to share the token's
// cos and sin (computed once per block, in shared memory), so the arithmetic
// of the angles hides under the loads.
#include <cuda_bf16.h>

#include <algorithm>

#include "dcp_device.cuh"
#include "dcp_internal.h"

namespace dcp {
namespace {

constexpr int kThreads = 256;
constexpr int kUnits = 4;          // units of a thread, all in flight at once
constexpr int kMaxPairs = 512;     // rotated pairs of a head (shared memory)

enum Mode { kHalf = 0, kInterleaved = 1, kScalar = 2 };

struct Params {
  AppendArgs a;
  int units_rot;        // units of a rotated head
  int units_total;      // units of a token: queries, keys, then values
  int lead;             // 16-byte vectors before the rotated part
  int turned;           // units of the rotated part
  __nv_bfloat16 *pool_k, *pool_v;
};

// (x0, x1) of 32-bit words holding two bf16 values each, turned by (c, s)
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<uint32_t*>(&v);
}

// the half layout: word w of the first vector holds x0 of pairs 2w, 2w + 1, of
// the second their x1
__device__ __forceinline__ void turn_half(uint4& u, uint4& v, const float* c, const float* s) {
  uint32_t* x = &u.x;
  uint32_t* y = &v.x;
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    const float a0 = bf16_lo(x[w]), a1 = bf16_hi(x[w]), b0 = bf16_lo(y[w]), b1 = bf16_hi(y[w]);
    const float c0 = c[2 * w], c1 = c[2 * w + 1], s0 = s[2 * w], s1 = s[2 * w + 1];
    x[w] = pack2(a0 * c0 - b0 * s0, a1 * c1 - b1 * s1);
    y[w] = pack2(b0 * c0 + a0 * s0, b1 * c1 + a1 * s1);
  }
}

// the interleaved layout: word w holds pair w
__device__ __forceinline__ void turn_interleaved(uint4& u, const float* c, const float* s) {
  uint32_t* x = &u.x;
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    const float a = bf16_lo(x[w]), b = bf16_hi(x[w]);
    x[w] = pack2(a * c[w] - b * s[w], b * c[w] + a * s[w]);
  }
}

template <int kMode>
__global__ void __launch_bounds__(kThreads) kv_append_kernel(const Params p, int units_per_block) {
  __shared__ __align__(16) float cs[kMaxPairs], sn[kMaxPairs];
  const AppendArgs& a = p.a;
  const int b = blockIdx.x / a.L, i = blockIdx.x % a.L;
  const int n = a.q_lens ? a.q_lens[b] : a.L;
  const int S = a.seq_lens[b];
  if (n < 0 || n > a.L || S < n) {
    if (threadIdx.x == 0) set_status(a.status, DCP_ERR_BOUNDS);
    return;
  }
  if (i >= n) return;
  const long long base = (long long)S - n, t = base + i;
  const long long pos = base + (a.pos_offsets ? a.pos_offsets[b * a.pos_stride + i] : i);

  // the cache cell of position t
  const int r = (int)((t / a.I) % a.N);
  const long long j = (t / ((long long)a.I * a.N)) * a.I + t % a.I;
  const long long jb = j / a.bs;
  const int blk = jb < a.max_lb ? a.block_tables[((long long)r * a.B + b) * a.max_lb + jb] : -1;
  const bool stored = (unsigned)blk < (unsigned)a.num_blocks;
  if (!stored && threadIdx.x == 0) set_status(a.status, DCP_ERR_BOUNDS);
  const long long cell = ((long long)blk * a.bs + j % a.bs) * a.Hkv * a.D;

  const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q) + b * a.q_batch + i * a.q_token;
  const __nv_bfloat16* k = static_cast<const __nv_bfloat16*>(a.k) + b * a.k_batch + i * a.k_token;
  const __nv_bfloat16* v = static_cast<const __nv_bfloat16*>(a.v) + b * a.v_batch + i * a.v_token;
  __nv_bfloat16* q_out = static_cast<__nv_bfloat16*>(a.q_out) + ((long long)b * a.L + i) * a.Hq * a.D;
  const int heads = a.Hq + a.Hkv;                       // rotated heads of the token

  auto turns = [&]() {
    for (int e = threadIdx.x; e < a.rot_dim / 2; e += kThreads) {
      const unsigned long long phase = (unsigned long long)pos * a.steps[e];
      const float half_turns = (float)(int)(phase >> 32) * 0x1p-31f;
      float s, c;
      sincospif(half_turns, &s, &c);
      cs[e] = c * a.mscale;
      sn[e] = s * a.mscale;
    }
    __syncthreads();
  };
  const int u0 = blockIdx.y * units_per_block;
  const int u1 = min(p.units_total, u0 + units_per_block);

  if constexpr (kMode == kScalar) {
    // rotated parts that do not fall on 16-byte vectors: a unit is a pair or one value
    turns();
    for (int u = u0 + (int)threadIdx.x; u < u1; u += kThreads) {
      if (u < heads * p.units_rot) {
        const int h = u / p.units_rot, w = u % p.units_rot;
        const bool key = h >= a.Hq;
        if (key && !stored) continue;
        const __nv_bfloat16* src = key ? k + (h - a.Hq) * a.D : q + h * a.D;
        __nv_bfloat16* dst = key ? p.pool_k + cell + (h - a.Hq) * a.D : q_out + h * a.D;
        if (w < a.rot_dim / 2) {
          const int d0 = a.rot_offset + (a.interleaved ? 2 * w : w);
          const int d1 = d0 + (a.interleaved ? 1 : a.rot_dim / 2);
          const float x = __bfloat162float(src[d0]), y = __bfloat162float(src[d1]);
          dst[d0] = __float2bfloat16_rn(x * cs[w] - y * sn[w]);
          dst[d1] = __float2bfloat16_rn(y * cs[w] + x * sn[w]);
        } else {
          int e = w - a.rot_dim / 2;                     // an unrotated value
          if (e >= a.rot_offset) e += a.rot_dim;
          dst[e] = src[e];
        }
      } else if (stored) {
        const int e = u - heads * p.units_rot;
        p.pool_v[cell + e] = v[e];
      }
    }
  } else {
    uint4 x[kUnits], y[kUnits];
    uint4 *dx[kUnits], *dy[kUnits];
    int pair[kUnits];                                    // first pair of the unit, -1: a copy
#pragma unroll
    for (int m = 0; m < kUnits; ++m) {
      const int u = u0 + m * kThreads + (int)threadIdx.x;
      dx[m] = dy[m] = nullptr;
      pair[m] = -1;
      if (u >= u1) continue;
      if (u < heads * p.units_rot) {
        const int h = u / p.units_rot, w = u % p.units_rot;
        const bool key = h >= a.Hq;
        if (key && !stored) continue;
        const uint4* src = reinterpret_cast<const uint4*>(key ? k + (h - a.Hq) * a.D : q + h * a.D);
        uint4* dst = reinterpret_cast<uint4*>(key ? p.pool_k + cell + (h - a.Hq) * a.D : q_out + h * a.D);
        int vec = w;                                     // 16-byte vector of the head
        if (w >= p.lead && w < p.lead + p.turned) {
          pair[m] = (w - p.lead) * (kMode == kHalf ? 8 : 4);
          if constexpr (kMode == kHalf) {
            y[m] = src[w + p.turned];
            dy[m] = dst + w + p.turned;
          }
        } else if (kMode == kHalf && w >= p.lead + p.turned) {
          vec = w + p.turned;
        }
        x[m] = src[vec];
        dx[m] = dst + vec;
      } else if (stored) {
        const int e = u - heads * p.units_rot;
        x[m] = reinterpret_cast<const uint4*>(v)[e];
        dx[m] = reinterpret_cast<uint4*>(p.pool_v + cell) + e;
      }
    }
    turns();
#pragma unroll
    for (int m = 0; m < kUnits; ++m) {
      if (dx[m] == nullptr) continue;
      if (pair[m] >= 0) {
        if constexpr (kMode == kHalf) {
          turn_half(x[m], y[m], cs + pair[m], sn + pair[m]);
          *dy[m] = y[m];
        } else {
          turn_interleaved(x[m], cs + pair[m], sn + pair[m]);
        }
      }
      *dx[m] = x[m];
    }
  }
}

}  // namespace

cudaError_t launch_kv_append(const AppendArgs& a) {
  Params p;
  p.a = a;
  if (a.q == nullptr) p.a.Hq = 0;
  const long long tokens = (long long)a.B * a.L;
  p.pool_k = static_cast<__nv_bfloat16*>(a.cache);
  p.pool_v = a.v ? p.pool_k + (long long)a.num_blocks * a.bs * a.Hkv * a.D : nullptr;
  // 16-byte vectors hold whole units of the rotated part: 4 interleaved pairs,
  // or 8 first and 8 second halves; other offsets go value by value
  const bool vec = a.rot_offset % 8 == 0 && a.rot_dim % (a.interleaved ? 8 : 16) == 0;
  if (vec) {
    p.lead = a.rot_offset / 8;
    p.turned = a.interleaved ? a.rot_dim / 8 : a.rot_dim / 16;
    p.units_rot = a.interleaved ? a.D / 8 : a.D / 8 - p.turned;
  } else {
    p.lead = p.turned = 0;
    p.units_rot = a.D - a.rot_dim / 2;
  }
  p.units_total = (p.a.Hq + a.Hkv) * p.units_rot + (a.v ? a.Hkv * (vec ? a.D / 8 : a.D) : 0);
  // few tokens: fewer units to a block, so that the step spreads over the SMs
  int per = kThreads * kUnits;
  while (per > kThreads && tokens * ((p.units_total + per - 1) / per) < 2 * device_sm_count()) per /= 2;
  const dim3 grid((unsigned)tokens, (unsigned)((p.units_total + per - 1) / per));
  if (!vec)
    kv_append_kernel<kScalar><<<grid, kThreads, 0, a.stream>>>(p, per);
  else if (a.interleaved)
    kv_append_kernel<kInterleaved><<<grid, kThreads, 0, a.stream>>>(p, per);
  else
    kv_append_kernel<kHalf><<<grid, kThreads, 0, a.stream>>>(p, per);
  return cudaGetLastError();
}

}  // namespace dcp
