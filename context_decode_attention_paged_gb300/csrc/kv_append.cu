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
// the launch and the chain of dependent loads.  A warp takes tasks in turn, a
// task being one token and some of its heads.  A lane always holds the same
// pairs of a head, so it finds their cos and sin once per task, in registers,
// and turns head after head: 16-byte vectors of 4 interleaved pairs, or the two
// vectors of 8 pairs in the half layout.  The first loads go out as soon as the
// lengths say that the token is there; position, angles and cache cell are
// found under them.  With lengths of their own, absent tokens have no tasks:
// every block first sums the counts (up to kScan requests; when there are more
// tasks than the SMs hold at once) and a warp finds its token in the sums.
// Rotated parts whose vectors do not divide a warp (rot_dim 96 in the half
// layout, say) or do not fall on vectors, and heads of 65,000 dims and more, go
// unit by unit with the angles in shared memory, one block a token.
//
// Measured (GB300; one of five in a graph): 64 tokens of 64 + 4 + 4 heads of 128
// (2.4 MB moved) 4.8 us, launch and dependent loads; 512 tokens of 128 + 1 heads of
// 576 (152 MB) 27.3 us, 5.6 TB/s; 6 ragged prompt chunks of up to 2,048 tokens (79
// MB) 15.9 us (L2 holds part of them by then; 20.6 as calls of their own, 3.9 TB/s).
#include <cuda_bf16.h>

#include <algorithm>

#include "dcp_device.cuh"
#include "dcp_internal.h"

namespace dcp {
namespace {

constexpr int kThreads = 256;
constexpr int kBlocks = 3;         // resident blocks of an SM
constexpr int kAhead = 4;          // heads of a lane whose loads are in flight
constexpr int kCopies = 8;         // vectors of a lane in flight while copying
constexpr int kTaskBytes = 8192;   // rows of a task, at most (when tokens abound)
constexpr int kMaxPairs = DCP_ROPE_MAX_DIM / 2;   // rotated pairs of a head (shared memory)
constexpr int kScan = 1024;        // requests whose token counts a block sums

enum Mode { kHalf = 0, kInterleaved = 1, kScalar = 2 };

struct Params {
  AppendArgs a;
  int units_rot;        // units of a rotated head
  int units_total;      // units of a token: queries, keys, then values
  int lead;             // 16-byte vectors before the rotated part
  int turned;           // units of the rotated part
  bool summed;          // tasks are numbered over the tokens that are there
  unsigned per_copies;  // ceil(2^32 / copies): quotients of small numbers by a multiplication
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

// Tokens of a request that are there (0 for a request whose lengths are out of range).
__device__ __forceinline__ int present(const AppendArgs& a, int b, bool* bad) {
  const int n = a.q_lens ? a.q_lens[b] : a.L;
  *bad = n < 0 || n > a.L || a.seq_lens[b] < n;
  return *bad ? 0 : n;
}

// ends[b] = tokens of requests 0 .. b, for all b < B <= kScan (whole block).
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

// cos and sin (times mscale) of position pos in pair e
__device__ __forceinline__ void turn_of(const AppendArgs& a, long long pos, int e, float& c, float& s) {
  const unsigned long long phase = (unsigned long long)pos * a.steps[e];
  sincospif((float)(int)(phase >> 32) * 0x1p-31f, &s, &c);
  c *= a.mscale;
  s *= a.mscale;
}

// First element of the cache cell of position t of request b, -1 (and
// DCP_ERR_BOUNDS) where the table has none.
__device__ __forceinline__ long long cell_of(const AppendArgs& a, int b, long long t, bool reports) {
  const int r = (int)((t / a.I) % a.N);
  const long long j = (t / ((long long)a.I * a.N)) * a.I + t % a.I;
  const long long jb = j / a.bs;
  const int blk = jb < a.max_lb ? a.block_tables[((long long)r * a.B + b) * a.max_lb + jb] : -1;
  if ((unsigned)blk < (unsigned)a.num_blocks) return ((long long)blk * a.bs + j % a.bs) * a.Hkv * a.D;
  if (reports) set_status(a.status, DCP_ERR_BOUNDS);
  return -1;
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

template <bool kHalfLayout>
__global__ void __launch_bounds__(kThreads, kBlocks) kv_append_kernel(const Params p, int parts, int part_heads,
                                                                      unsigned tasks) {
  constexpr int kPairs = kHalfLayout ? 8 : 4;            // pairs of a lane
  __shared__ int ends[kScan];
  const AppendArgs& a = p.a;
  const int lane = threadIdx.x & 31;
  const int heads = a.Hq + a.Hkv, turned = p.turned, copies = p.units_rot - turned, row16 = a.D / 8;
  const int skip = kHalfLayout ? 2 * turned : turned;    // vectors of the rotated part
  const int unit = lane % turned, first = lane / turned, step = 32 / turned;   // this lane's vector; heads of a pass
  if (p.summed) {
    sum_counts(a, ends);
    tasks = (unsigned)ends[a.B - 1] * (unsigned)parts;
  }
  for (unsigned task = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); task < tasks;
       task += gridDim.x * (kThreads / 32)) {
    const unsigned token = task / (unsigned)parts;
    const int part = (int)(task - token * (unsigned)parts);
    int b = (int)(token / (unsigned)a.L), i = (int)(token % (unsigned)a.L);
    if (p.summed) b = find_token(ends, a.B, token, &i);
    bool bad;
    const int n = present(a, b, &bad);
    if (bad && lane == 0) set_status(a.status, DCP_ERR_BOUNDS);
    if (i >= n) continue;
    const uint4* q = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.q) + b * a.q_batch + i * a.q_token);
    const uint4* k = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.k) + b * a.k_batch + i * a.k_token);
    uint4* q_out = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.q_out) + ((long long)b * a.L + i) * a.Hq * a.D);
    const int h0 = part * part_heads, h1 = min(heads, h0 + part_heads);
    auto row_in = [&](int h) { return h < a.Hq ? q + h * row16 : k + (h - a.Hq) * row16; };
    uint4 x[kAhead], y[kHalfLayout ? kAhead : 1];
    auto load = [&](int h) {
#pragma unroll
      for (int m = 0; m < kAhead; ++m)
        if (h + m * step < h1) {
          const uint4* src = row_in(h + m * step) + p.lead + unit;
          x[m] = src[0];                                 // (q_out may be q: no read-only path)
          if constexpr (kHalfLayout) y[m] = src[turned];
        }
    };
    load(h0 + first);

    const long long base = (long long)a.seq_lens[b] - n, t = base + i;
    const long long pos = base + (a.pos_offsets ? a.pos_offsets[b * a.pos_stride + i] : i);
    float cs[kPairs], sn[kPairs];
#pragma unroll
    for (int e = 0; e < kPairs; ++e) turn_of(a, pos, unit * kPairs + e, cs[e], sn[e]);
    uint4 *cell_k = nullptr, *cell_v = nullptr;
    if (h1 > a.Hq) {
      const long long cell = cell_of(a, b, t, lane == 0);
      if (cell >= 0) {
        cell_k = reinterpret_cast<uint4*>(p.pool_k + cell);
        cell_v = reinterpret_cast<uint4*>(p.pool_v + cell);
      }
    }
    auto row_out = [&](int h) -> uint4* {
      return h < a.Hq ? q_out + h * row16 : cell_k != nullptr ? cell_k + (h - a.Hq) * row16 : nullptr;
    };

    for (int h = h0 + first; h < h1; h += kAhead * step) {
#pragma unroll
      for (int m = 0; m < kAhead; ++m) {
        if (h + m * step >= h1) break;
        uint4* dst = row_out(h + m * step);
        if (dst == nullptr) continue;
        dst += p.lead + unit;
        if constexpr (kHalfLayout) {
          turn_half(x[m], y[m], cs, sn);
          dst[turned] = y[m];
        } else {
          turn_interleaved(x[m], cs, sn);
        }
        dst[0] = x[m];
      }
      load(h + kAhead * step);
    }
    // the dims that do not turn (queries rotated in place have them already),
    // and with the last heads the values
    if (copies > 0) {
      const int q1 = min(h1, a.Hq), k0 = max(h0, a.Hq) - a.Hq, k1 = h1 - a.Hq;
      auto around = [&](int c) {                           // vector c of the unrotated ones, head by head
        const int h = copies == 1 ? c : (int)__umulhi((unsigned)c, p.per_copies);
        const int vec = c - h * copies;
        return h * row16 + (vec < p.lead ? vec : vec + skip);
      };
      if (q != q_out) copy_vectors(q + h0 * row16, q_out + h0 * row16, (q1 - h0) * copies, lane, around);
      if (cell_k != nullptr) copy_vectors(k + k0 * row16, cell_k + k0 * row16, (k1 - k0) * copies, lane, around);
    }
    if (a.v != nullptr && h1 == heads && cell_v != nullptr)
      copy_vectors(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.v) + b * a.v_batch + i * a.v_token),
                   cell_v, a.Hkv * row16, lane, [](int c) { return c; });
  }
}

// Any rotated part, one block a token: a unit is a vector of unrotated values,
// the vectors of a group of pairs, or (kScalar) one pair or value.
template <int kMode>
__global__ void __launch_bounds__(kThreads) kv_append_any_kernel(const Params p) {
  __shared__ __align__(16) float cs[kMaxPairs], sn[kMaxPairs];
  const AppendArgs& a = p.a;
  const int b = (int)(blockIdx.x / (unsigned)a.L), i = (int)(blockIdx.x % (unsigned)a.L);
  bool bad;
  const int n = present(a, b, &bad);
  if (bad && threadIdx.x == 0) set_status(a.status, DCP_ERR_BOUNDS);
  if (i >= n) return;
  const long long base = (long long)a.seq_lens[b] - n, t = base + i;
  const long long pos = base + (a.pos_offsets ? a.pos_offsets[b * a.pos_stride + i] : i);
  for (int e = threadIdx.x; e < a.rot_dim / 2; e += kThreads) turn_of(a, pos, e, cs[e], sn[e]);
  const long long cell = cell_of(a, b, t, threadIdx.x == 0);
  __syncthreads();
  const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q) + b * a.q_batch + i * a.q_token;
  const __nv_bfloat16* k = static_cast<const __nv_bfloat16*>(a.k) + b * a.k_batch + i * a.k_token;
  const __nv_bfloat16* v = static_cast<const __nv_bfloat16*>(a.v) + b * a.v_batch + i * a.v_token;
  __nv_bfloat16* q_out = static_cast<__nv_bfloat16*>(a.q_out) + ((long long)b * a.L + i) * a.Hq * a.D;
  const int rotated = (a.Hq + a.Hkv) * p.units_rot;
  for (int u = (int)threadIdx.x; u < p.units_total; u += kThreads) {
    if (u >= rotated) {
      if (cell < 0) continue;
      if constexpr (kMode == kScalar)
        p.pool_v[cell + u - rotated] = v[u - rotated];
      else
        reinterpret_cast<uint4*>(p.pool_v + cell)[u - rotated] = reinterpret_cast<const uint4*>(v)[u - rotated];
      continue;
    }
    const int h = u / p.units_rot, w = u % p.units_rot;
    const bool key = h >= a.Hq;
    if (key && cell < 0) continue;
    const __nv_bfloat16* src = key ? k + (h - a.Hq) * a.D : q + h * a.D;
    __nv_bfloat16* dst = key ? p.pool_k + cell + (h - a.Hq) * a.D : q_out + h * a.D;
    if constexpr (kMode == kScalar) {
      if (w < a.rot_dim / 2) {
        const int d0 = a.rot_offset + (a.interleaved ? 2 * w : w);
        const int d1 = d0 + (a.interleaved ? 1 : a.rot_dim / 2);
        const float x0 = __bfloat162float(src[d0]), x1 = __bfloat162float(src[d1]);
        dst[d0] = __float2bfloat16_rn(x0 * cs[w] - x1 * sn[w]);
        dst[d1] = __float2bfloat16_rn(x1 * cs[w] + x0 * sn[w]);
      } else {
        int e = w - a.rot_dim / 2;                         // an unrotated value
        if (e >= a.rot_offset) e += a.rot_dim;
        dst[e] = src[e];
      }
    } else {
      const uint4* src16 = reinterpret_cast<const uint4*>(src);
      uint4* dst16 = reinterpret_cast<uint4*>(dst);
      if (w >= p.lead && w < p.lead + p.turned) {
        uint4 x = src16[w];
        if constexpr (kMode == kHalf) {
          uint4 y = src16[w + p.turned];
          turn_half(x, y, cs + (w - p.lead) * 8, sn + (w - p.lead) * 8);
          dst16[w + p.turned] = y;
        } else {
          turn_interleaved(x, cs + (w - p.lead) * 4, sn + (w - p.lead) * 4);
        }
        dst16[w] = x;
      } else {
        const int at = kMode == kHalf && w >= p.lead + p.turned ? w + p.turned : w;
        dst16[at] = src16[at];
      }
    }
  }
}

}  // namespace

cudaError_t launch_kv_append(const AppendArgs& a) {
  Params p;
  p.a = a;
  if (a.q == nullptr) p.a.Hq = 0;
  p.summed = false;
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
  const int copies = p.units_rot - p.turned;
  p.per_copies = copies > 1 ? (unsigned)(((1ull << 32) + copies - 1) / copies) : 0u;
  p.units_total = (p.a.Hq + a.Hkv) * p.units_rot + (a.v ? a.Hkv * (vec ? a.D / 8 : a.D) : 0);
  // per_copies finds the quotient of a vector number below 2^32 / copies; a task has
  // at most about two passes of heads, or kTaskBytes, of vectors
  auto quotients_fit = [&]() { return (2LL * (32 / p.turned) * copies + kTaskBytes / 8) * copies < (1LL << 32); };
  if (vec && p.turned <= 32 && 32 % p.turned == 0 && quotients_fit()) {
    // heads of a task: up to kTaskBytes of rows, fewer when the tokens alone
    // would not fill the SMs' warps (a pass of 32 / turned heads at the least)
    const int sms = device_sm_count(), heads = p.a.Hq + a.Hkv, step = 32 / p.turned;
    const int passes = (heads + step - 1) / step;
    const long long warps = (long long)sms * kBlocks * (kThreads / 32);
    const long long wanted = std::max((warps + tokens - 1) / tokens, ((long long)heads * a.D * 2 + kTaskBytes - 1) / kTaskBytes);
    int parts = (int)std::min<long long>(std::max<long long>(wanted, 1), passes);
    const int part_heads = (passes + parts - 1) / parts * step;
    parts = (heads + part_heads - 1) / part_heads;
    const long long tasks = tokens * parts;
    if (tasks >= (1LL << 31)) return cudaErrorInvalidValue;        // (terabytes of rows)
    // more tasks than the SMs hold at once, some of them absent tokens': the
    // blocks sum the counts and stay for several tasks
    p.summed = a.q_lens != nullptr && a.B <= kScan && tasks > warps;
    const long long blocks = (tasks + kThreads / 32 - 1) / (kThreads / 32);
    const unsigned grid = (unsigned)(p.summed ? (long long)kBlocks * sms : blocks);
    if (a.interleaved)
      kv_append_kernel<false><<<grid, kThreads, 0, a.stream>>>(p, parts, part_heads, (unsigned)tasks);
    else
      kv_append_kernel<true><<<grid, kThreads, 0, a.stream>>>(p, parts, part_heads, (unsigned)tasks);
  } else if (!vec) {
    kv_append_any_kernel<kScalar><<<(unsigned)tokens, kThreads, 0, a.stream>>>(p);
  } else if (a.interleaved) {
    kv_append_any_kernel<kInterleaved><<<(unsigned)tokens, kThreads, 0, a.stream>>>(p);
  } else {
    kv_append_any_kernel<kHalf><<<(unsigned)tokens, kThreads, 0, a.stream>>>(p);
  }
  return cudaGetLastError();
}

}  // namespace dcp
