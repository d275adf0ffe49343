// Appending keys and values to the sharded cache with RMS norms of the heads and
// the rotary position applied on the way, into the bf16 cache or into the 8-bit
// one, and the same for the queries of these tokens.
//
// "Context Parallel Guide", section "Overview": a token's KV is stored once, by
// the shard that owns its position (interleave rule, section "Decode Context
// Parallel").
//
// Mathematics.  y = x w / sqrt(mean x^2 + eps) over the first norm_dim dims of a
// head; pair k at position p then turns by p f_k.  As in kv_append.cu the table
// holds frac(f_k / 2 pi) 2^64, so the top 32 bits of the wrapped product are the
// phase at any position; what is left of the nearest quarter turn goes through
// the Taylor series of sin and cos (|x| <= pi / 4: the first terms left out are
// below 2e-9), about 1e-7 in all.
// The 8-bit cache has one scale 2^e per block, KV head and K or V: the new rows'
// largest magnitude a sets it where the block was empty (a <= 112 2^e), it stays
// while a <= 448 2^e and otherwise the block's earlier codes are rounded to the
// scale that a wants.  A quarter of the range is left free at first, so a later
// row seldom makes a block read and written again; codes have exponents of their
// own, so what that costs is two of the 15 binades below the largest value.
//
// Layout.  SG lanes hold a row of one head, SLOTS 16-byte vectors each (128 dims:
// 16 lanes, two rows a warp), so a norm is one pass of shuffles in the group.
// Pairs of the interleaved layout lie in a lane; in the half layout the partner
// vector is another lane's (a shuffle); any other rotated part goes through
// shared memory.  Queries: a warp takes a token's heads in turn, its angles and
// weights in registers; vectors that neither norm nor rotation touch are copied.
// Rows of the 8-bit cache: a team takes all new rows of one block and KV head: norm,
// rotation and maximum, then the codes from what it kept in shared memory (rows that
// do not fit are read, from L2, and made again).  Up to kWarpRows rows a team is a
// warp, in one launch with the queries; more take a CTA, and the queries' kernel runs
// beside that one (a programmatic launch; one launch for both held the queries to the
// rows' registers).
//
// Bound: for latent rows HBM; for prompts loads that 24 warps an SM wait for and a
// second wave of tasks that is not full (issue slots at 0.56 and, in 8 bits, 0.43:
// about 190 instructions a pass of two rows of 128); for a decode step the launch
// and dependent loads.  Measured (GB300, in a
// graph; 64 + 4 heads of 128 unless said): 64 tokens 5.5 us into either cache; 2,154
// tokens of ragged prompts into the bf16 cache 26 us (79 MB, 3.1 TB/s), into the
// 8-bit one 31; 400 drafted tokens of 40 + 8 heads 11; 1,352 latent rows with 128
// query heads of 576 84 (401 MB, 4.8 TB/s).  Packed two-value arithmetic and a
// fourth CTA an SM gained nothing (26.5 and 28.8 us for 26).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <float.h>

#include <algorithm>
#include <climits>

#include "dcp_append.cuh"
#include "dcp_device.cuh"
#include "dcp_internal.h"

namespace dcp {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kAhead = 4;          // heads of a lane whose loads are in flight
// Rows of a query task, at most (when tokens abound).  Rows that are mostly copied take the larger one (latent
// prompt rows 83 us; at 8192 88), rows that are worked on the smaller (prompt chunks 26 us; at 16384 34).
constexpr int kTaskBytes = 8192, kCopyTaskBytes = 16384;
constexpr int kKeptBytes = 96 * 1024;   // shared memory of a CTA for made rows (of 16 warps: half as much again)
constexpr int kSmemBytes = 220 * 1024;  // of a CTA in all (the counts' sums are beside it)
constexpr int kWarpRows = 32;      // rows of a block that a warp takes alone (drafted tokens, 12 rows: 11 us; by a CTA 22)

enum Rot { kPair = 0, kSwap = 1, kAny = 2 };

// Vectors of a head that norm and rotation touch; the `rest` others are copied as they are.
struct Window {
  int first, count, rest;
  unsigned per_rest;               // ceil(2^32 / rest): quotients of small numbers by a multiplication
};

struct Params {
  NormAppendArgs a;
  __nv_bfloat16 *pool_k, *pool_v;  // bf16 cache
  uint8_t *codes_k, *codes_v;      // 8-bit cache
  int groups;                      // (block, shard) groups of a request, or its tokens
  int nblk;                        // blocks of a shard that may get rows; 0: groups are tokens
  unsigned kv_blocks;              // CTAs of the 8-bit cache's rows, before the queries'
  long long kv_tasks;
  int parts, part_heads;           // query heads of a token in parts
  long long q_tasks;
  int kept_rows, kept_floats;      // rows that a group of lanes keeps in shared memory; floats of a warp for them
  bool keys;                       // the token tasks store the bf16 cache's rows too
  bool summed;                     // tasks are numbered over the tokens that are there
  Window q, k;
};

__device__ __forceinline__ uint32_t pack2(float a, float b) {
  __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<uint32_t*>(&v);
}

// cos and sin (times mscale) of position pos in pair k
__device__ __forceinline__ void turn_of(const AppendArgs& a, long long pos, int k, float& c, float& s) {
  const uint32_t phase = (uint32_t)(((unsigned long long)pos * a.steps[k]) >> 32);   // 2^-32 turns
  const uint32_t quarter = (phase + 0x20000000u) >> 30;
  const float x = (float)(int32_t)(phase - (quarter << 30)) * (0x1p-31f * 3.14159265358979f);
  const float z = x * x;
  const float sn = x * fmaf(z, fmaf(z, fmaf(z, fmaf(z, 1.f / 362880, -1.f / 5040), 1.f / 120), -1.f / 6), 1.f);
  const float cs = fmaf(z, fmaf(z, fmaf(z, fmaf(z, fmaf(z, -1.f / 3628800, 1.f / 40320), -1.f / 720), 1.f / 24), -0.5f), 1.f);
  const bool odd = quarter & 1u;
  c = (odd ? sn : cs) * ((quarter + 1) & 2u ? -a.mscale : a.mscale);
  s = (odd ? cs : sn) * (quarter & 2u ? -a.mscale : a.mscale);
}

__device__ __forceinline__ void unpack(const uint4& u, float (&x)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) x[2 * k] = bf16_lo(w[k]), x[2 * k + 1] = bf16_hi(w[k]);
}

__device__ __forceinline__ uint4 pack(const float (&x)[8]) {
  return make_uint4(pack2(x[0], x[1]), pack2(x[2], x[3]), pack2(x[4], x[5]), pack2(x[6], x[7]));
}

// Floats of shared memory that a warp needs to rotate.
__host__ __device__ constexpr int scratch_floats(int rot, int sg, int rot_dim) {
  return rot == kAny ? 2 * (32 / sg) * rot_dim : 0;
}

// A lane's part of a row of one head: dims 8 (first + sl + SG s) .. + 7, s < SLOTS, of the vectors
// [first, first + vecs) that norm and rotation touch (all of the head where it is quantised).
template <int SG, int SLOTS, int kRot>
struct Rows {
  static constexpr int kAngles = kRot == kPair ? 4 : kRot == kSwap ? 8 : 1;
  const AppendArgs& a;
  int sl, vecs, norm_vecs, dim0;   // dim0: first dim of the window
  float eps, per_dim;              // 1 / norm_dim
  bool normed;
  float w[SLOTS][8];
  float c[SLOTS][kAngles], s[SLOTS][kAngles];
  uint32_t turns;                  // kPair: bit 4 slot + pair; kSwap: 1 where the lane turns
  int partner;                     // kSwap: lane of the partner vector
  float *values, *angles;          // kAny: this group's shared memory

  __device__ __forceinline__ Rows(const NormAppendArgs& n, int lane, float* scratch, int first, int count)
      : a(n), sl(lane % SG), vecs(count), norm_vecs(n.norm_dim / 8), dim0(8 * first), eps(n.eps),
        per_dim(1.f / (float)n.norm_dim), normed(false), turns(0), partner(lane), values(nullptr), angles(nullptr) {
    if constexpr (kRot == kPair) {
#pragma unroll
      for (int m = 0; m < SLOTS; ++m)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int d = dim0 + 8 * (sl + SG * m) + 2 * e - a.rot_offset;
          if (d >= 0 && d < a.rot_dim) turns |= 1u << (4 * m + e);
        }
    } else if constexpr (kRot == kSwap) {
      const int half = a.rot_dim / 16, v = sl + (dim0 - a.rot_offset) / 8;
      if (v >= 0 && v < 2 * half) {
        turns = 1;
        partner = lane + (v < half ? half : -half);
      }
    } else {
      values = scratch + (lane / SG) * 2 * a.rot_dim;
      angles = values + a.rot_dim;
    }
  }

  __device__ __forceinline__ void set_weights(const float* weight) {
    normed = weight != nullptr;
#pragma unroll
    for (int m = 0; m < SLOTS; ++m)
#pragma unroll
      for (int e = 0; e < 8; ++e) w[m][e] = normed && sl + SG * m < norm_vecs ? weight[8 * (sl + SG * m) + e] : 1.f;
  }

  __device__ __forceinline__ void set_position(long long pos) {
    if constexpr (kRot == kPair) {
#pragma unroll
      for (int m = 0; m < SLOTS; ++m)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (turns >> (4 * m + e) & 1u) turn_of(a, pos, (dim0 + 8 * (sl + SG * m) + 2 * e - a.rot_offset) / 2, c[m][e], s[m][e]);
    } else if constexpr (kRot == kSwap) {
      // the lanes of both halves need the same 8 angles: each finds 4 and gets the others from its partner
      const int half = a.rot_dim / 16, v = sl + (dim0 - a.rot_offset) / 8;
      const bool second = v >= half;
      float mc[4], ms[4];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (turns) turn_of(a, pos, second ? 8 * (v - half) + 4 + e : 8 * v + e, mc[e], ms[e]);
        else mc[e] = ms[e] = 0.f;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float oc = __shfl_sync(0xffffffffu, mc[e], partner), os = __shfl_sync(0xffffffffu, ms[e], partner);
        c[0][e] = second ? oc : mc[e], c[0][e + 4] = second ? mc[e] : oc;
        s[0][e] = second ? os : -ms[e], s[0][e + 4] = second ? ms[e] : -os;
      }
    } else {
      __syncwarp();                 // (the last row's angles have been read)
      for (int k = sl; k < a.rot_dim / 2; k += SG) turn_of(a, pos, k, angles[2 * k], angles[2 * k + 1]);
      __syncwarp();
    }
  }

  // a row of zeros where src is null
  __device__ __forceinline__ void load(const __nv_bfloat16* src, uint4 (&raw)[SLOTS]) const {
#pragma unroll
    for (int m = 0; m < SLOTS; ++m)
      raw[m] = src != nullptr && sl + SG * m < vecs ? reinterpret_cast<const uint4*>(src + dim0)[sl + SG * m]
                                                    : make_uint4(0, 0, 0, 0);
  }

  __device__ __forceinline__ float group_sum(float v) const {
#pragma unroll
    for (int o = SG / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
  }

  // norm and rotation of the row, in place (whole warp)
  __device__ __forceinline__ void turn(float (&x)[SLOTS][8]) const {
    if (normed) {
      float sum = 0.f;
#pragma unroll
      for (int m = 0; m < SLOTS; ++m)
        if (sl + SG * m < norm_vecs)
#pragma unroll
          for (int e = 0; e < 8; ++e) sum = fmaf(x[m][e], x[m][e], sum);
      sum = group_sum(sum);
      float r = rsqrtf(fmaf(sum, per_dim, eps));
      if (__any_sync(0xffffffffu, sum > FLT_MAX)) {
        // squares past fp32's range (or an infinity): the sum from values scaled down; eps is below rounding then
        const float by = sum > FLT_MAX ? 0x1p-70f : 1.f;
        float small = 0.f;
#pragma unroll
        for (int m = 0; m < SLOTS; ++m)
          if (sl + SG * m < norm_vecs)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const float y = x[m][e] * by;
              small = fmaf(y, y, small);
            }
        small = group_sum(small);
        if (sum > FLT_MAX) r = rsqrtf(small * per_dim) * by;
      }
#pragma unroll
      for (int m = 0; m < SLOTS; ++m)
        if (sl + SG * m < norm_vecs)
#pragma unroll
          for (int e = 0; e < 8; ++e) x[m][e] = x[m][e] * r * w[m][e];
    }
    if constexpr (kRot == kPair) {
#pragma unroll
      for (int m = 0; m < SLOTS; ++m)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (turns >> (4 * m + e) & 1u) {
            const float x0 = x[m][2 * e], x1 = x[m][2 * e + 1];
            x[m][2 * e] = x0 * c[m][e] - x1 * s[m][e];
            x[m][2 * e + 1] = x1 * c[m][e] + x0 * s[m][e];
          }
    } else if constexpr (kRot == kSwap) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float other = __shfl_sync(0xffffffffu, x[0][e], partner);
        if (turns) x[0][e] = x[0][e] * c[0][e] + other * s[0][e];
      }
    } else {
#pragma unroll
      for (int m = 0; m < SLOTS; ++m)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int d = dim0 + 8 * (sl + SG * m) + e - a.rot_offset;
          if (d >= 0 && d < a.rot_dim) values[d] = x[m][e];
        }
      __syncwarp();
      const int half = a.rot_dim / 2;
#pragma unroll
      for (int m = 0; m < SLOTS; ++m)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int d = dim0 + 8 * (sl + SG * m) + e - a.rot_offset;
          if (d < 0 || d >= a.rot_dim) continue;
          const bool second = a.interleaved ? d & 1 : d >= half;
          const int k = a.interleaved ? d >> 1 : second ? d - half : d;
          const float other = values[a.interleaved ? d ^ 1 : second ? d - half : d + half];
          x[m][e] = x[m][e] * angles[2 * k] + other * (second ? angles[2 * k + 1] : -angles[2 * k + 1]);
        }
      __syncwarp();
    }
  }

  __device__ __forceinline__ void store_bf16(__nv_bfloat16* dst, const float (&x)[SLOTS][8]) const {
    if (dst == nullptr) return;
#pragma unroll
    for (int m = 0; m < SLOTS; ++m)
      if (sl + SG * m < vecs) reinterpret_cast<uint4*>(dst + dim0)[sl + SG * m] = pack(x[m]);
  }
};

__device__ __forceinline__ long long position_of(const AppendArgs& a, int b, int i, long long base) {
  return base + (a.pos_offsets ? a.pos_offsets[b * a.pos_stride + i] : i);
}

// Block of local token l of request b on shard r; -1 (and DCP_ERR_BOUNDS) where the table has none.
__device__ __forceinline__ int block_of(const AppendArgs& a, int b, int r, int jb, bool reports) {
  const int blk = jb < a.max_lb ? a.block_tables[((long long)r * a.B + b) * a.max_lb + jb] : -1;
  if ((unsigned)blk < (unsigned)a.num_blocks) return blk;
  if (reports) set_status(a.status, DCP_ERR_BOUNDS);
  return -1;
}

// Heads [h0, h1) of a token at position pos: src + h D -> dst + h D, in turn over the warp's groups.
template <int SG, int SLOTS, int kRot>
__device__ __forceinline__ void head_rows(Rows<SG, SLOTS, kRot>& rows, const __nv_bfloat16* src, __nv_bfloat16* dst, int h0,
                                          int h1, int lane, int D, long long pos, const float* weight) {
  constexpr int kStep = 32 / SG, kDeep = SLOTS > 1 ? 2 : kAhead;
  uint4 raw[kDeep][SLOTS];
  rows.set_position(pos);
  rows.set_weights(weight);
  const int mine = lane / SG;
  auto row = [&](int h) { return h < h1 ? src + (long long)h * D : nullptr; };
#pragma unroll
  for (int m = 0; m < kDeep; ++m) rows.load(row(h0 + m * kStep + mine), raw[m]);
  for (int h = h0; h < h1; h += kDeep * kStep) {             // (whole warps: the norms shuffle)
#pragma unroll
    for (int m = 0; m < kDeep; ++m) {
      if (h + m * kStep >= h1) break;
      float x[SLOTS][8];
#pragma unroll
      for (int k = 0; k < SLOTS; ++k) unpack(raw[m][k], x[k]);
      const int hh = h + m * kStep + mine;
      rows.load(row(hh + kDeep * kStep), raw[m]);
      rows.turn(x);
      rows.store_bf16(hh < h1 ? dst + (long long)hh * D : nullptr, x);
    }
  }
}

// The vectors around the window of heads [h0, h1).
__device__ __forceinline__ void copy_rest(const Window& w, const __nv_bfloat16* src, __nv_bfloat16* dst, int h0, int h1,
                                          int row16, int lane) {
  if (w.rest == 0 || src == dst) return;
  copy_vectors(reinterpret_cast<const uint4*>(src) + (long long)h0 * row16, reinterpret_cast<uint4*>(dst) + (long long)h0 * row16,
               (h1 - h0) * w.rest, lane, [&](int c) {
                 const int h = w.rest == 1 ? c : (int)__umulhi((unsigned)c, w.per_rest), v = c - h * w.rest;
                 return h * row16 + (v < w.first ? v : v + w.count);
               });
}

// Task (token, part of its query heads, or (with `keys`) behind them its keys and values into the bf16 cache).
template <int SG, int SLOTS, int QSG, int QSLOTS, int kRot>
__device__ __forceinline__ void token_task(const Params& p, int b, int i, int part, int lane, float* scratch) {
  const NormAppendArgs& a = p.a;
  bool bad;
  const int n = present(a, b, &bad);
  if (bad && lane == 0) set_status(a.status, DCP_ERR_BOUNDS);
  if (i >= n) return;
  const long long base = (long long)a.seq_lens[b] - n;
  const int row16 = a.D / 8;
  if (part < p.parts) {
    const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(a.q) + b * a.q_batch + i * a.q_token;
    __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(a.q_out) + ((long long)b * a.L + i) * a.Hq * a.D;
    const int h0 = part * p.part_heads, h1 = min(a.Hq, h0 + p.part_heads);
    if (p.q.count > 0) {
      Rows<QSG, QSLOTS, kRot> rows(a, lane, scratch, p.q.first, p.q.count);
      head_rows(rows, src, dst, h0, h1, lane, a.D, position_of(a, b, i, base), a.q_weight);
    }
    copy_rest(p.q, src, dst, h0, h1, row16, lane);
    return;
  }
  const long long t = base + i;
  const int r = (int)((t / a.I) % a.N);
  const long long j = (t / ((long long)a.I * a.N)) * a.I + t % a.I;
  const int blk = block_of(a, b, r, (int)(j / a.bs), lane == 0);
  if (blk < 0) return;
  const long long cell = ((long long)blk * a.bs + j % a.bs) * a.Hkv * a.D;
  const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(a.k) + b * a.k_batch + i * a.k_token;
  if (p.k.count > 0) {
    Rows<SG, SLOTS, kRot> rows(a, lane, scratch, p.k.first, p.k.count);
    head_rows(rows, src, p.pool_k + cell, 0, a.Hkv, lane, a.D, position_of(a, b, i, base), a.k_weight);
  }
  copy_rest(p.k, src, p.pool_k + cell, 0, a.Hkv, row16, lane);
  if (a.v != nullptr)
    copy_vectors(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.v) + b * a.v_batch + i * a.v_token),
                 reinterpret_cast<uint4*>(p.pool_v + cell), a.Hkv * row16, lane, [](int c) { return c; });
}

// The token tasks of blocks [0, blocks), a warp each in turn.
template <int SG, int SLOTS, int QSG, int QSLOTS, int kRot>
__device__ __forceinline__ void token_tasks(const Params& p, int* ends, unsigned block, unsigned blocks, float* scratch) {
  const NormAppendArgs& a = p.a;
  const unsigned parts = p.parts + (p.keys ? 1 : 0);
  long long tasks = p.q_tasks;
  if (p.summed) {
    sum_counts<kThreads>(a, ends);
    tasks = (long long)ends[a.B - 1] * parts;
  }
#pragma unroll 1
  for (long long task = (long long)block * kWarps + (threadIdx.x >> 5); task < tasks; task += (long long)blocks * kWarps) {
    const unsigned token = (unsigned)task / parts, part = (unsigned)task - token * parts;
    int b = (int)(token / (unsigned)a.L), i = (int)(token % (unsigned)a.L);
    if (p.summed) b = find_token(ends, a.B, token, &i);
    token_task<SG, SLOTS, QSG, QSLOTS, kRot>(p, b, i, (int)part, threadIdx.x & 31, scratch);
  }
}

// Queries, and (with `keys`) the bf16 cache's rows.  Beside kv8_rows_kernel (`beside`) it starts while that
// one runs and ends behind it.
template <int SG, int SLOTS, int QSG, int QSLOTS, int kRot>
__global__ void __launch_bounds__(kThreads, SLOTS == 1 ? 3 : 2) token_kernel(const Params p, bool beside) {
  extern __shared__ float4 scratch[];
  __shared__ int ends[kScan];
  token_tasks<SG, SLOTS, QSG, QSLOTS, kRot>(p, ends, blockIdx.x, gridDim.x,
                                            reinterpret_cast<float*>(scratch) +
                                                (threadIdx.x >> 5) * scratch_floats(kRot, QSG < SG ? QSG : SG, p.a.rot_dim));
  if (beside) asm volatile("griddepcontrol.wait;" ::: "memory");
}

// Codes of a vector: y / 2^e to nearest (y by = 2^-e), NaN where y is not finite.
__device__ __forceinline__ uint2 codes_of(const float (&y)[8], float by) {
  uint32_t out[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    uint16_t half[2];
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      float v[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float x = y[4 * k + 2 * m + e];
        v[e] = fabsf(x) <= FLT_MAX ? x * by : NAN;
      }
      asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(half[m]) : "f"(v[1]), "f"(v[0]));
    }
    out[k] = (uint32_t)half[0] | (uint32_t)half[1] << 16;
  }
  return make_uint2(out[0], out[1]);
}

__device__ __forceinline__ void values_of(const uint2& u, float (&y)[8]) {
  const uint32_t w[2] = {u.x, u.y};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    uint32_t pair;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(pair) : "h"((uint16_t)(w[k / 2] >> (16 * (k & 1)))));
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&pair));
    y[2 * k] = f.x, y[2 * k + 1] = f.y;
  }
}

// 2^e, e within the exponents of normal numbers
__device__ __forceinline__ float power(int e) { return __int_as_float((127 + e) << 23); }

// Exponent of the scale that a largest magnitude wants: the smallest e with most <= 112 2^e.
__device__ __forceinline__ int exponent_for(float most) {
  const uint32_t bits = __float_as_uint(most);
  const int e = (int)(bits >> 23) - 127 - 6 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0);   // 112 = 1.75 2^6
  return min(max(e, -DCP_KV8_MAX_EXP), DCP_KV8_MAX_EXP);
}

// The new rows of one block, KV head and K or V, by a team of kTeam warps.
template <int SG, int SLOTS, int kRot, int kTeam>
__device__ __forceinline__ void block_rows(const Params& p, long long task, int team_warp, int lane, float* scratch,
                                           float* shared, float4* kept) {
  constexpr int kGroups = kTeam * 32 / SG;                    // rows at a time
  constexpr int kLoads = SLOTS > 1 ? 2 : 4;                   // rows of a group whose loads are in flight
  const NormAppendArgs& a = p.a;
  const int kinds = a.v != nullptr ? 2 : 1;
  const bool values = kinds == 2 && (task & 1);
  long long rest = kinds == 2 ? task >> 1 : task;
  const int h = (int)(rest % a.Hkv);
  rest /= a.Hkv;
  const int g = (int)(rest % p.groups), b = (int)(rest / p.groups);
  bool bad;
  const int n = present(a, b, &bad);
  if (bad && lane == 0 && team_warp == 0) set_status(a.status, DCP_ERR_BOUNDS);
  if (n == 0 || (p.nblk == 0 && g >= n)) return;
  const int S = a.seq_lens[b], base = S - n;
  // local tokens [lo, hi) of shard r, in block jb of its table
  int r, jb, lo, hi;
  if (p.nblk == 0) {
    // token g leads a block's new rows: it is the first of them
    const int t = base + g;
    r = (int)(((unsigned)t / (unsigned)a.I) % (unsigned)a.N);
    lo = local_len(t, r, a.I, a.N);
    if (lo != local_len(base, r, a.I, a.N) && lo % a.bs) return;
    jb = lo / a.bs;
  } else {
    r = g / p.nblk;
    const int from = local_len(base, r, a.I, a.N);
    jb = from / a.bs + g % p.nblk;
    lo = max(from, (int)min((long long)jb * a.bs, (long long)INT_MAX));
  }
  hi = (int)min((long long)local_len(S, r, a.I, a.N), ((long long)jb + 1) * a.bs);
  if (lo >= hi) return;
  const int count = hi - lo, before = lo % a.bs;              // new rows, slots of earlier ones
  const int group = (team_warp * 32 + lane) / SG;
  const __nv_bfloat16* src = values ? static_cast<const __nv_bfloat16*>(a.v) + b * a.v_batch + (long long)h * a.D
                                    : static_cast<const __nv_bfloat16*>(a.k) + b * a.k_batch + (long long)h * a.D;
  const long long token = values ? a.v_token : a.k_token;
  Rows<SG, SLOTS, kRot> rows(a, lane, scratch, 0, a.D / 8);
  auto index_of = [&](int k) { return (int)(global_pos(lo + min(k, count - 1), r, a.I, a.N) - base); };
  auto load = [&](int k, uint4 (&raw)[SLOTS]) { rows.load(k < count ? src + index_of(k) * token : nullptr, raw); };
  auto make = [&](int k, const uint4 (&raw)[SLOTS], float (&y)[SLOTS][8]) {
#pragma unroll
    for (int m = 0; m < SLOTS; ++m) unpack(raw[m], y[m]);
    if (!values) {
      rows.set_position(position_of(a, b, index_of(k), base));
      rows.turn(y);
    }
  };
  // A lane keeps its part of the made rows in shared memory (its own alone: two float4 a vector, lanes side by
  // side), as far as there is room; rows behind that are read and made again.
  const int room = p.kept_rows;
  auto keep = [&](int step, int m, int half) -> float4& { return kept[((step * SLOTS + m) * 2 + half) * 32 + lane]; };
  float most = 0.f;
  uint4 raw[kLoads][SLOTS];
#pragma unroll
  for (int m = 0; m < kLoads; ++m) load(m * kGroups + group, raw[m]);
  if (!values) rows.set_weights(a.k_weight);
  for (int k0 = 0, step = 0; k0 < count; k0 += kLoads * kGroups) {
#pragma unroll
    for (int q = 0; q < kLoads; ++q, ++step) {
      const int k = k0 + q * kGroups;
      if (k >= count) break;
      float y[SLOTS][8];
      make(k + group, raw[q], y);
      load(k + kLoads * kGroups + group, raw[q]);
#pragma unroll
      for (int m = 0; m < SLOTS; ++m) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float x = fabsf(y[m][e]);
          if (x <= FLT_MAX) most = fmaxf(most, x);
        }
        if (step < room) {
          keep(step, m, 0) = make_float4(y[m][0], y[m][1], y[m][2], y[m][3]);
          keep(step, m, 1) = make_float4(y[m][4], y[m][5], y[m][6], y[m][7]);
        }
      }
    }
  }
  const int blk = block_of(a, b, r, jb, lane == 0 && team_warp == 0);
  const long long scale_at = ((values ? (long long)a.num_blocks : 0) + max(blk, 0)) * a.Hkv + h;
  const uint32_t old = a.scales[scale_at];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
  if constexpr (kTeam > 1) {
    if (lane == 0) shared[team_warp] = most;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kTeam; ++k) most = fmaxf(most, shared[k]);
  }
  if (blk < 0) return;
  uint8_t* pool = (values ? p.codes_v : p.codes_k) + ((long long)blk * a.bs * a.Hkv + h) * a.D;
  const long long pitch = (long long)a.Hkv * a.D;
  uint32_t byte = old;
  if (before == 0 || !(most <= 448.f * scale_factor(old))) {  // (a factor of NaN holds nothing)
    byte = (uint32_t)(127 + exponent_for(most));
    if (lane == 0 && team_warp == 0) a.scales[scale_at] = (uint8_t)byte;
    // the earlier rows' codes, to the new scale (2^-126 of a code is 0, as less of it is)
    const float ratio = old == 255 ? NAN : power(min(max((int)old - (int)byte, -126), 127));
    const int vecs = a.D / 8, total = before * vecs;
    for (int c0 = team_warp * 32 + lane; c0 < total; c0 += kTeam * 32 * 4) {
      uint2 u[4];
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        const int c = c0 + m * kTeam * 32;
        if (c < total) u[m] = *reinterpret_cast<const uint2*>(pool + (c / vecs) * pitch + (c % vecs) * 8);
      }
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        const int c = c0 + m * kTeam * 32;
        float v[8];
        values_of(u[m], v);
        if (c < total) *reinterpret_cast<uint2*>(pool + (c / vecs) * pitch + (c % vecs) * 8) = codes_of(v, ratio);
      }
    }
  }
  const float by = scale_factor(254 - byte);                  // 1 / the factor
  auto store = [&](int k, const float (&v)[SLOTS][8]) {
    if (k >= count) return;
#pragma unroll
    for (int m = 0; m < SLOTS; ++m)
      if (rows.sl + SG * m < rows.vecs)
        *reinterpret_cast<uint2*>(pool + (before + k) * pitch + (rows.sl + SG * m) * 8) = codes_of(v[m], by);
  };
  for (int k = 0, step = 0; k < count; k += kGroups, ++step) {
    float v[SLOTS][8];
    if (step < room) {
#pragma unroll
      for (int m = 0; m < SLOTS; ++m) {
        const float4 lo = keep(step, m, 0), up = keep(step, m, 1);
        v[m][0] = lo.x, v[m][1] = lo.y, v[m][2] = lo.z, v[m][3] = lo.w;
        v[m][4] = up.x, v[m][5] = up.y, v[m][6] = up.z, v[m][7] = up.w;
      }
    } else {
      load(k + group, raw[0]);
      make(k + group, raw[0], v);
    }
    store(k + group, v);
  }
}

// Few rows a block: a warp a block's rows, and the queries behind them in the same launch.
template <int SG, int SLOTS, int QSG, int QSLOTS, int kRot>
__global__ void __launch_bounds__(kThreads, SLOTS == 1 ? 3 : 2) kv8_step_kernel(const Params p) {
  extern __shared__ float4 scratch[];
  __shared__ int ends[kScan];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float* kept = reinterpret_cast<float*>(scratch);             // (16-byte aligned: first)
  float* mine = kept + kWarps * p.kept_floats + warp * scratch_floats(kRot, QSG < SG ? QSG : SG, p.a.rot_dim);
  if (blockIdx.x < p.kv_blocks) {
    const long long task = (long long)blockIdx.x * kWarps + warp;
    if (task < p.kv_tasks)
      block_rows<SG, SLOTS, kRot, 1>(p, task, 0, lane, mine, nullptr, reinterpret_cast<float4*>(kept + warp * p.kept_floats));
  } else {
    token_tasks<SG, SLOTS, QSG, QSLOTS, kRot>(p, ends, blockIdx.x - p.kv_blocks, gridDim.x - p.kv_blocks, mine);
  }
}

// Many rows a block: a CTA a block's rows.  The queries' kernel runs beside it.
template <int SG, int SLOTS, int kRot, int kTeam>
__global__ void __launch_bounds__(32 * kTeam, kTeam == 16 ? 1 : 2) kv8_rows_kernel(const Params p) {
  extern __shared__ float4 scratch[];
  __shared__ float shared[kTeam];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float* kept = reinterpret_cast<float*>(scratch);
  block_rows<SG, SLOTS, kRot, kTeam>(p, blockIdx.x, warp, lane, kept + kTeam * p.kept_floats + warp * scratch_floats(kRot, SG, p.a.rot_dim),
                                     shared, reinterpret_cast<float4*>(kept + warp * p.kept_floats));
}

template <typename Kernel, typename... Args>
cudaError_t start(Kernel kernel, unsigned grid, int threads, size_t smem, cudaStream_t stream, bool beside, Args... args) {
  if (smem > 40 * 1024) {
    const cudaError_t e = allow_smem(kernel, kSmemBytes);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = beside ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <int SG, int SLOTS, int QSG, int QSLOTS, int kRot>
cudaError_t launch_rot(const Params& p, int team, unsigned q_blocks, cudaStream_t stream) {
  const size_t turning = scratch_floats(kRot, SG, p.a.rot_dim), q_turning = scratch_floats(kRot, std::min(QSG, SG), p.a.rot_dim);
  const size_t q_smem = kWarps * q_turning * sizeof(float);
  if (p.a.scales == nullptr)
    return start(token_kernel<SG, SLOTS, QSG, QSLOTS, kRot>, q_blocks, kThreads, q_smem, stream, false, p, false);
  if (team == 1)
    return start(kv8_step_kernel<SG, SLOTS, QSG, QSLOTS, kRot>, p.kv_blocks + q_blocks, kThreads,
                 kWarps * (q_turning + p.kept_floats) * sizeof(float), stream, false, p);
  constexpr int kTeam = SLOTS == 1 ? 8 : 16;
  const cudaError_t e = start(kv8_rows_kernel<SG, SLOTS, kRot, kTeam>, p.kv_blocks, 32 * kTeam,
                              kTeam * (turning + p.kept_floats) * sizeof(float), stream, false, p);
  if (e != cudaSuccess || q_blocks == 0) return e;
  // (without keys: the instance of the queries' own shape)
  return start(token_kernel<QSG, QSLOTS, QSG, QSLOTS, kRot>, q_blocks, kThreads, kWarps * scratch_floats(kRot, QSG, p.a.rot_dim) * sizeof(float),
               stream, true, p, true);
}

template <int SG, int SLOTS, int QSG, int QSLOTS>
cudaError_t launch(const Params& p, int rot, int team, unsigned q_blocks, cudaStream_t stream) {
  if (rot == kPair) return launch_rot<SG, SLOTS, QSG, QSLOTS, kPair>(p, team, q_blocks, stream);
  if constexpr (SLOTS == 1)
    if (rot == kSwap) return launch_rot<SG, SLOTS, QSG, QSLOTS, kSwap>(p, team, q_blocks, stream);
  return launch_rot<SG, SLOTS, QSG, QSLOTS, kAny>(p, team, q_blocks, stream);
}

Window window_of(const NormAppendArgs& a, bool normed) {
  const int row16 = a.D / 8, lo = a.rot_dim ? a.rot_offset / 8 : 0, hi = a.rot_dim ? (a.rot_offset + a.rot_dim + 7) / 8 : 0;
  Window w;
  w.first = normed ? 0 : lo;
  w.count = (normed ? std::max(hi, a.norm_dim / 8) : hi) - w.first;
  w.rest = row16 - w.count;
  w.per_rest = w.rest > 1 ? (unsigned)(((1ull << 32) + w.rest - 1) / w.rest) : 0u;
  return w;
}

}  // namespace

cudaError_t launch_kv_append_norm(const NormAppendArgs& a) {
  Params p{};
  p.a = a;
  p.q = window_of(a, a.q_weight != nullptr);
  p.k = window_of(a, a.k_weight != nullptr);
  const long long pool = (long long)a.num_blocks * a.bs * a.Hkv * a.D;
  const long long tokens = (long long)a.B * a.L;
  const int sms = device_sm_count();
  const int sg = a.D <= 64 ? 8 : a.D <= 128 ? 16 : 32;
  // queries without a norm have their rotated vectors turned alone, by 8 lanes where they are 8 at most
  const bool narrow = sg > 8 && p.q.count <= 8;
  const int qsg = narrow ? 8 : sg;
  // interleaved pairs within a lane's vector; whole vectors of halves; anything else
  const int rot = a.rot_dim == 0 || (a.interleaved && a.rot_offset % 2 == 0) ? kPair
                  : !a.interleaved && a.rot_offset % 8 == 0 && a.rot_dim % 16 == 0 && a.D <= 256 ? kSwap
                                                                                                : kAny;
  int team = 1;
  if (a.scales == nullptr) {
    p.pool_k = static_cast<__nv_bfloat16*>(a.cache);
    p.pool_v = a.v ? p.pool_k + pool : nullptr;
  } else {
    p.codes_k = static_cast<uint8_t*>(a.cache);
    p.codes_v = a.v ? p.codes_k + pool : nullptr;
    // rows that L tokens in a row can bring a shard, and the blocks they can fall in; for few
    // tokens each of them looks whether it is the first of its block instead
    const long long period = (long long)a.I * a.N;
    const long long most = std::min<long long>(a.L, a.L / period * a.I + std::min<long long>(a.I, a.L % period));
    const long long nblk = (most + a.bs - 2) / a.bs + 1;
    const bool by_token = a.L <= nblk * a.N;
    p.nblk = by_token ? 0 : (int)nblk;
    p.groups = by_token ? a.L : (int)(nblk * a.N);
    // long rows: 16 warps (and all of an SM's registers and memory); else 8
    team = std::min<long long>(most, a.bs) <= kWarpRows ? 1 : a.D <= 256 ? 8 : 16;
    // made rows that a warp's groups of lanes keep, up to kKeptBytes of a CTA
    const int cta = team == 1 ? kWarps : team, at_once = team * 32 / sg, slots = a.D <= 256 ? 1 : 3;
    const long long steps = (std::min<long long>(most, a.bs) + at_once - 1) / at_once;
    // (beside what the rotation takes, within an SM's memory)
    const int turning = cta * scratch_floats(rot, qsg, a.rot_dim) * (int)sizeof(float);
    const int room = team == 16 ? std::min(kKeptBytes + kKeptBytes / 2, kSmemBytes - turning) : kKeptBytes;
    p.kept_rows = (int)std::min<long long>(steps, room / (cta * 32 * slots * 32));
    p.kept_floats = p.kept_rows * 32 * slots * 8;
    p.kv_tasks = (long long)a.B * p.groups * a.Hkv * (a.v ? 2 : 1);
    if (p.kv_tasks >= (1LL << 31)) return cudaErrorInvalidValue;
    p.kv_blocks = (unsigned)(team == 1 ? (p.kv_tasks + cta - 1) / cta : p.kv_tasks);
  }
  // query heads of a task: up to kTaskBytes of rows, fewer when the tokens alone would not
  // fill the SMs' warps
  const int resident = a.D <= 256 || (team > 1 && narrow) ? 3 : 2;
  const long long warps = (long long)sms * resident * kWarps;
  if (a.Hq > 0) {
    const int task_bytes = 2 * p.q.rest > a.D / 8 ? kCopyTaskBytes : kTaskBytes;
    const int step = 32 / qsg, passes = (a.Hq + step - 1) / step;
    const long long wanted = std::max((warps + tokens - 1) / tokens, ((long long)a.Hq * a.D * 2 + task_bytes - 1) / task_bytes);
    p.parts = (int)std::min<long long>(std::max<long long>(wanted, 1), passes);
    p.part_heads = (passes + p.parts - 1) / p.parts * step;
    p.parts = (a.Hq + p.part_heads - 1) / p.part_heads;
  }
  p.keys = a.scales == nullptr;
  p.q_tasks = tokens * (p.parts + (p.keys ? 1 : 0));
  // (quotients by per_rest: numbers below 2^32 / rest)
  if (p.q_tasks >= (1LL << 31) || (long long)std::max(p.part_heads, a.Hkv) * p.q.rest * p.q.rest >= (1LL << 32) ||
      (long long)a.Hkv * p.k.rest * p.k.rest >= (1LL << 32))
    return cudaErrorInvalidValue;
  // more tasks than the SMs hold at once, some of them absent tokens': the blocks sum the counts
  // and stay for several tasks
  p.summed = a.q_lens != nullptr && a.B <= kScan && p.q_tasks > warps;
  const long long q_blocks = p.summed ? (long long)sms * resident : (p.q_tasks + kWarps - 1) / kWarps;
  if (a.D <= 64) return launch<8, 1, 8, 1>(p, rot, team, (unsigned)q_blocks, a.stream);
  if (a.D <= 128)
    return narrow ? launch<16, 1, 8, 1>(p, rot, team, (unsigned)q_blocks, a.stream) : launch<16, 1, 16, 1>(p, rot, team, (unsigned)q_blocks, a.stream);
  if (a.D <= 256)
    return narrow ? launch<32, 1, 8, 1>(p, rot, team, (unsigned)q_blocks, a.stream) : launch<32, 1, 32, 1>(p, rot, team, (unsigned)q_blocks, a.stream);
  return narrow ? launch<32, 3, 8, 1>(p, rot, team, (unsigned)q_blocks, a.stream) : launch<32, 3, 32, 3>(p, rot, team, (unsigned)q_blocks, a.stream);
}

}  // namespace dcp
