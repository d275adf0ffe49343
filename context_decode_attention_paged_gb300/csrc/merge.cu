// Step a6 (LSE merge + head-slice return) and step a5 (combine of the KV
// splits of one shard, the same rule one level down).
//
// vLLM DCP blog, "DCP 執行流程" (AllGather + ReduceScatter): partial outputs
// and their log-sum-exp values are shared, reweighted with the online-softmax
// rule and summed; each rank keeps only its slice of heads.
//   LSE = m + log sum_r exp(lse_r - m),  m = max_r lse_r
//   o   = sum_r exp(lse_r - LSE) * o_r
// HBM-bound: one warp per output row streams the N partial rows with 16-byte
// loads; the N weights come from one lse load per lane and warp shuffles.  A warp
// has four sources in flight, the first four requested before the weights are
// known.  Measured (GB300): 512 x 128 rows of 8 sources of 512 floats (1.14 GB)
// 0.166 ms, 6.9 TB/s; source after source it was 0.201 ms.  Sources behind the last
// that counts are not read: with 2 of the 8 holding keys (requests of a few tokens)
// 0.065 ms, 0.166 if all are read.  Five blocks an SM (48 registers) matter: with
// 60 registers, four, 1024 x 64 rows of 4 sources of 128 floats take 35 us, not 31.
#include "dcp_device.cuh"
#include "dcp_internal.h"

namespace dcp {
namespace {

constexpr int kWarpsPerBlock = 8;

// Weights for up to 32 sources, one per lane: returns this lane's weight and
// writes the merged LSE.  lane_lse is -inf for lanes >= n; a NaN makes the
// merged row NaN, also where every other source is empty.
__device__ __forceinline__ float lse_weights(float lane_lse, float* merged_lse) {
  float m = lane_lse;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if (m == -INFINITY) {
    const bool nan = __any_sync(0xffffffffu, lane_lse != lane_lse);
    *merged_lse = nan ? NAN : -INFINITY;
    return nan ? NAN : 0.f;
  }
  float e = (lane_lse == -INFINITY) ? 0.f : expf(lane_lse - m);
  float s = e;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  *merged_lse = m + logf(s);
  return e / s;
}

constexpr int kBatch = 4;          // sources of a lane in flight

// Vector c of sources k0 .. k0 + kBatch - 1 (those below n).
__device__ __forceinline__ void load_batch(const float* __restrict__ src, long long src_stride, int n, int k0, int c,
                                           float4 (&v)[kBatch]) {
#pragma unroll
  for (int k = 0; k < kBatch; ++k)
    if (k0 + k < n) v[k] = __ldcs(reinterpret_cast<const float4*>(src + (k0 + k) * src_stride) + c);
}

// out row = sum over n sources (stride src_stride floats) of w_k * src_k.
// Dv4 = Dv / 4 float4 per row.  Loads go out kBatch sources at a time, the first
// ones (in `v`, vector `lane`) before the weights are known.  `counts`: this lane's
// source does.  A source of weight 0 does not, whatever it holds; with kLight it
// does where it has keys, and what is not finite shows however small its weight.
template <bool kBf16Out, bool kLight = false>
__device__ __forceinline__ void weighted_row(const float* __restrict__ src, long long src_stride,
                                             int n, float w_lane, bool counts, int Dv4, float4 (&v)[kBatch],
                                             void* dst_row) {
  const int lane = threadIdx.x & 31;
  // tokens and splits are dealt from the first source on, so those without keys are
  // the last ones
  // (a NaN LSE makes the weights of lanes without a source NaN too)
  n = 32 - __clz(__ballot_sync(0xffffffffu, lane < n && counts));
  for (int c = lane; c - lane < Dv4; c += 32) {
    const bool in = c < Dv4;                         // (the shuffles below take the whole warp)
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k0 = 0; k0 < n; k0 += kBatch) {
      if (in && (c != lane || k0 > 0)) load_batch(src, src_stride, n, k0, c, v);
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        if (k0 + k >= n) break;
        const float w = __shfl_sync(0xffffffffu, w_lane, k0 + k);
        if (w == 0.f) {
          if constexpr (kLight) {                      // (a source without keys holds zeros)
            acc.x = fabsf(v[k].x) < INFINITY ? acc.x : acc.x + v[k].x;
            acc.y = fabsf(v[k].y) < INFINITY ? acc.y : acc.y + v[k].y;
            acc.z = fabsf(v[k].z) < INFINITY ? acc.z : acc.z + v[k].z;
            acc.w = fabsf(v[k].w) < INFINITY ? acc.w : acc.w + v[k].w;
          }
          continue;
        }
        acc.x = fmaf(w, v[k].x, acc.x);
        acc.y = fmaf(w, v[k].y, acc.y);
        acc.z = fmaf(w, v[k].z, acc.z);
        acc.w = fmaf(w, v[k].w, acc.w);
      }
    }
    if (!in) continue;
    if (kBf16Out) {
      __nv_bfloat162 lo = __floats2bfloat162_rn(acc.x, acc.y);
      __nv_bfloat162 hi = __floats2bfloat162_rn(acc.z, acc.w);
      uint2 pk;
      pk.x = *reinterpret_cast<uint32_t*>(&lo);
      pk.y = *reinterpret_cast<uint32_t*>(&hi);
      reinterpret_cast<uint2*>(dst_row)[c] = pk;
    } else {
      reinterpret_cast<float4*>(dst_row)[c] = acc;
    }
  }
}

// One warp per (b, i, h): merge N shard partials; write rank h / (Hq/N)'s slice.
__global__ void __launch_bounds__(kWarpsPerBlock * 32, 5)
merge_kernel(const float* __restrict__ partial_out, const float* __restrict__ lse, int N, int B,
             int Lq, int Hq, int Dv, __nv_bfloat16* __restrict__ out, float* __restrict__ out_lse) {
  const long long row = (long long)blockIdx.x * kWarpsPerBlock + (threadIdx.x >> 5);
  const long long rows = (long long)B * Lq * Hq;
  if (row >= rows) return;
  const int lane = threadIdx.x & 31;
  // row = (b * Lq + i) * Hq + h ; partial rows of shard r at r * rows + row
  const float lane_lse = lane < N ? lse[(long long)lane * rows + row] : -INFINITY;
  const float* src = partial_out + row * Dv;
  const long long stride = rows * (long long)Dv;
  float4 v[kBatch];
  if (lane < Dv / 4) load_batch(src, stride, N, 0, lane, v);
  float merged;
  const float w = lse_weights(lane_lse, &merged);
  const int h = (int)(row % Hq);
  const long long bi = row / Hq;
  const int hs = Hq / N;
  const int r = h / hs;
  const long long dst = (((long long)r * B * Lq + bi) * hs + (h % hs));
  weighted_row<true>(src, stride, N, w, w != 0.f, Dv / 4, v, out + dst * Dv);
  if (out_lse && lane == 0) out_lse[dst] = merged;
}

// One warp per (r, b, i, h): merge n_split workspace partials into partial_out (kLight: the
// 8-bit cache's, where a NaN value shows in every row that sees it, wherever splits begin).
template <bool kLight>
__global__ void __launch_bounds__(kWarpsPerBlock * 32, 5)
split_combine_kernel(const float* __restrict__ ws_o, const float* __restrict__ ws_lse, int n_split,
                     long long rows, int Hq, int Dv, float* __restrict__ partial_out,
                     float* __restrict__ lse) {
  const long long row = (long long)blockIdx.x * kWarpsPerBlock + (threadIdx.x >> 5);
  if (row >= rows) return;
  const int lane = threadIdx.x & 31;
  // row = ((r * B + b) * Lq + i) * Hq + h ; ws rows: (unit * n_split + s) * Hq + h
  const long long unit = row / Hq;
  const int h = (int)(row % Hq);
  const long long base = unit * n_split * Hq + h;
  const float lane_lse = lane < n_split ? ws_lse[base + (long long)lane * Hq] : -INFINITY;
  const float* src = ws_o + base * Dv;
  const long long stride = (long long)Hq * Dv;
  float4 v[kBatch];
  if (lane < Dv / 4) load_batch(src, stride, n_split, 0, lane, v);
  float merged;
  const float w = lse_weights(lane_lse, &merged);
  weighted_row<false, kLight>(src, stride, n_split, w, kLight ? lane_lse != -INFINITY : w != 0.f, Dv / 4, v,
                              partial_out + row * Dv);
  if (lane == 0) lse[row] = merged;
}

}  // namespace

cudaError_t launch_merge(const float* partial_out, const float* lse, int N, int B, int Lq, int Hq,
                         int Dv, void* out, float* out_lse, cudaStream_t stream) {
  const long long rows = (long long)B * Lq * Hq;
  if (rows == 0) return cudaSuccess;
  const long long blocks = (rows + kWarpsPerBlock - 1) / kWarpsPerBlock;
  merge_kernel<<<(unsigned)blocks, kWarpsPerBlock * 32, 0, stream>>>(
      partial_out, lse, N, B, Lq, Hq, Dv, static_cast<__nv_bfloat16*>(out), out_lse);
  return cudaGetLastError();
}

cudaError_t launch_split_combine(const AttnArgs& a, const SplitPlan& p) {
  const long long rows = (long long)a.N * a.B * a.Lq * a.Hq;
  if (rows == 0 || p.n_split <= 1) return cudaSuccess;
  const float* ws_o = static_cast<const float*>(a.workspace);
  const size_t o_bytes = (size_t)rows * p.n_split * a.Dv * sizeof(float);
  const float* ws_lse = reinterpret_cast<const float*>(static_cast<const char*>(a.workspace) +
                                                       ((o_bytes + 255) & ~size_t(255)));
  const long long blocks = (rows + kWarpsPerBlock - 1) / kWarpsPerBlock;
  auto* kernel = a.kv_scales ? split_combine_kernel<true> : split_combine_kernel<false>;
  kernel<<<(unsigned)blocks, kWarpsPerBlock * 32, 0, a.stream>>>(ws_o, ws_lse, p.n_split, rows, a.Hq, a.Dv, a.partial_out,
                                                                 a.lse);
  return cudaGetLastError();
}

}  // namespace dcp
