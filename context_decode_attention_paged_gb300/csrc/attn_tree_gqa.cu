// Drafted-tree attention for GQA on tcgen05 tensor cores.
//
// Compute step of the vLLM DCP blog ("DCP 執行流程") for a tree of drafted
// tokens ("未來發展藍圖", speculative decoding): every shard attends the nodes'
// queries to its local keys and returns a partial output with its LSE.
//
// Mathematics, for one row (node i, query head h) over the shard's keys:
//   m = max_t x_t,  l = sum_t 2^(x_t - m),  o = sum_t 2^(x_t - m) v_t,
//   x_t = scale log2(e) q . k_t  for the keys the row sees, -inf for the others,
// in one pass with a running m that moves lazily (only past 2^8), so that o is
// rescaled a few times in all; partial = o / l, lse = (m + log2 l) ln 2.
//
// A tree of n nodes puts n * Hq / Hkv query rows against each KV head: 64
// nodes of a 16-head group are 1024 rows, 1024 flop per cache byte, four times
// the ridge.  So rows sit on the 128 lanes of the MMA (M), unlike the decode
// kernel, which has few rows and puts the keys there:
//   S = Q K^T   (M = 128 rows, N = 64 keys, K = D; both K-major in shared memory)
//   O += P V    (M = 128 rows, N = D, K = 64 keys; P from TMEM, V MN-major)
// in steps of 64 keys, two to a tile of 128.
// A probability is rounded to bf16 once unless it is heavy, above 2^-3 of its
// row's sum so far: then bf16(p - bf16(p)) goes along as a second term, so that
// 16 bits of it reach the product.  Of a row at most a few probabilities are
// heavy at any time, and they alone could lose half a bf16 step of the output; a
// warp that holds none skips the second term, its half of the PV product too.
//
// Work unit = (shard, request, KV head, row block, KV split).  A CTA holds an SM
// and takes units in turn (longest requests first, forth and back over the CTAs),
// so that the next unit's tiles load while the last one ends.  It runs two
// streams, each two 64-key score/probability buffers and an output tile in
// TMEM, an MMA issuer warp, and a warpgroup of 128 threads (thread = row):
//   more than 128 rows: stream w takes rows [128 w, +128) of the block of 256
//     and both go over every key tile, so each tile in shared memory serves
//     256 rows;
//   128 rows or fewer: both streams hold the same rows and take the key tiles
//     in turn, each through half of the ring, two independent running softmaxes
//     joined at the end.
// A tile of 128 keys is two steps of 64: S(s + 1) is issued while the
// probabilities of step s are made, and the other stream's MMAs fill what is
// left.  P(s) overwrites S(s) in TMEM (its first 32 columns the first terms, its
// last 32 the second); a thread's MMAs complete in order, so the commit behind
// PV(s) also says that O is at rest and may be rescaled.
//
// Masks.  A shard's keys are dense in global order: context keys, then the
// nodes it owns.  Tiles of context keys alone take no mask; in the others a
// thread builds its row's 128 visibility bits from the mask words.  The value
// product mixes all rows of a tile, so a value no row may see must not be
// there: rows past the key range are zeroed in shared memory, and entries of
// node values that are not finite are replaced by 0 and added in the epilogue
// to the rows that see them.
//
// Warp roles (384 threads; setmaxnreg moves registers to the softmax warps):
// warps 0 and 3 TMA producers (ring of K and V tiles; warp 0 also makes the
// units), warps 1 and 2 the streams' MMA issuers (whole warps on uniform values,
// one elected lane issues: 30-37 cycles an MMA instead of 65-90 from one lane's
// branch), warps 4-7 and 8-11 the two streams; warps without a row skip the
// softmax.  Every wait is bounded; on expiry the kernel records DCP_ERR_TIMEOUT,
// drains its copies and MMAs and returns.
//
// Measured (GB300, 2.07 GHz, D = 128, 64 query and 4 KV heads, 4 shards):
//   64 requests of 8,192 to 32,768 tokens, 5 nodes: 379 us, 6.2 TB/s (HBM);
//   16 of them, 64 nodes (1024 rows a KV head): 534 us in a graph, 1.13 PFLOP/s
//     (559 as a call of its own; the merge is part of both): a step of
//     both streams takes ~1,740 cycles, ~1,260 of them tensor time (the scores'
//     operands come out of shared memory, 47 cycles an MMA of 32); a unit's
//     start and end are ~14,000 of ~128,000 cycles;
//   64 of 1,000 to 16,384 tokens, 1 node: 149 us, 4.9 TB/s: start and end are
//     ~12,000 of a unit's ~38,000 cycles, and the last CTAs end ~8 us after the
//     rest.
// Slower when tried: two threads a row (no gain for 640 threads), exponentials
// before the maximum is known (745 us against 624 at the time), one issuer for
// both streams with two score buffers (869 against 581), the second term for
// every probability (3% on the first of these cases, 18% on the second, 5 to 20% on
// small batches of 128 rows or fewer).
#include <cuda.h>
#include <cuda_bf16.h>

#include <algorithm>

#include "dcp_device.cuh"
#include "dcp_internal.h"
#include "dcp_sm100.cuh"
#include "dcp_tma.h"
#include "dcp_tree.cuh"

namespace dcp {
namespace {

using namespace sm100;

constexpr int kNt = 128;                      // keys per tile, rows per stream
constexpr int kNs = 64;                       // keys per step: half a tile
constexpr int kMaxSlots = 12;                 // K or V tiles in the ring
constexpr int kThreads = 384;
constexpr int kLaunchRegs = 168, kCtrlRegs = 72, kSoftRegs = 216;
static_assert(128 * kCtrlRegs + 256 * kSoftRegs <= kThreads * kLaunchRegs, "register split exceeds the launch");
constexpr size_t kSmemLimit = 232448;         // dynamic shared memory per CTA
constexpr float kLazyLog2 = 8.0f;             // m moves when scores pass it by more than this
constexpr float kHeavyLog2 = 3.0f;            // a probability above 2^-3 of its row's sum so far takes its second term
constexpr uint32_t kBarEpi = 1;               // named barrier of the two streams
constexpr int kLptMaxBatch = 128;             // longest-first unit order up to this batch
// TMEM columns (512 allocated): scores of step s of stream w, and P over them,
// at 128 w + 64 (s & 1); O at 256 + 128 w
constexpr uint32_t kColO = 256;

struct Params {
  const __nv_bfloat16* q;
  const __nv_bfloat16* v_pool;
  const int32_t *block_tables, *seq_lens, *q_lens;
  const uint32_t* mask;
  long long mask_stride;
  float* dst_o;
  float* dst_lse;
  int* status;
  int B, Lq, Hq, Hkv, N, I, max_lb, bs, num_blocks, n_split, split_tokens, words;
  int row_blocks, block_rows;      // row blocks of a KV head and their rows (128 or 256)
  bool turns;                      // 128 rows: the streams take the key tiles in turn
  int units, slots, q_bytes;
  float scale_log2;
  unsigned long long wait_ns;
  int skip_tile;
};

// One unit: which rows and which keys of the shard.
struct Unit {
  int b, r, g, s_idx;
  int row0, R, R_out;      // first row, rows that attend, rows to write
  int kb, ke, ctx;         // keys [kb, ke), context keys of the shard
  int L, T;                // keys of the shard, key tiles of the unit
  bool turns, bad;
  long long base;
  // key tile n of stream w, how many it has, and its steps (the last half tile may be empty)
  __device__ __forceinline__ int tile(int w, int n) const { return turns ? 2 * n + w : n; }
  __device__ __forceinline__ int tiles(int w) const { return turns ? (T + 1 - w) / 2 : T; }
  __device__ __forceinline__ int steps(int w) const {
    const int n = tiles(w);
    return n > 0 && kb + tile(w, n - 1) * kNt + kNs >= ke ? 2 * n - 1 : 2 * n;
  }
  // first key of step s
  __device__ __forceinline__ int key(int w, int s) const { return kb + tile(w, s >> 1) * kNt + (s & 1) * kNs; }
};

// Ring.  A tile is two items, K then V, numbered through the CTA's units.  In
// turn each stream has its own items in its half of the slots, else both read
// every item: either way a stream that waits for an item has consumed the last
// one in that slot (a barrier a whole lap behind its waiter would look done).
struct Ring {
  int first, len;          // slots of the stream
  __device__ __forceinline__ Ring(const Params& p, int w)
      : first(p.turns ? w * (p.slots / 2) : 0), len(p.turns ? p.slots / 2 : p.slots) {}
  __device__ __forceinline__ int slot(unsigned item) const { return first + (int)(item % (unsigned)len); }
  __device__ __forceinline__ uint32_t lap(unsigned item) const { return item / (unsigned)len; }
};

struct Smem {
  uint64_t full[kMaxSlots], empty[kMaxSlots];
  uint64_t s_full[2][2], p_full[2][2], pv_done[2], o_full[2], drain[2];   // [stream][step parity]
  uint64_t q_full[2];              // by unit parity: see the issuers
  uint64_t unit_full[2], unit_free[2];
  uint32_t tmem_base;
  int abort;
  Unit unit[2];                    // by turns: the unit at hand and the next
  uint32_t odd[2][8];              // node keys of the unit whose values are not all finite (bit: key - first)
  unsigned heavy[2][2];            // per stream and step parity: 1 + the last step with a heavy probability
  uint8_t order[kLptMaxBatch];     // requests, longest first
};

// Unit n of this CTA, -1 past the last.  CTAs take the units back and forth, so
// that each gets long and short ones.
__device__ __forceinline__ int unit_of(const Params& p, int n) {
  const long long at = (long long)n * gridDim.x + ((n & 1) ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
  return at < p.units ? (int)at : -1;
}

__device__ __forceinline__ Unit make_unit(const Params& p, const Smem& sm, int unit) {
  Unit u;
  const int per_req = p.N * p.Hkv * p.row_blocks * p.n_split;       // (units fit in 32 bits)
  const int k_req = unit / per_req, rest = unit % per_req;
  u.b = p.B <= kLptMaxBatch ? sm.order[k_req] : k_req;
  u.s_idx = rest % p.n_split;
  const int mb = rest / p.n_split % p.row_blocks;
  u.g = rest / (p.n_split * p.row_blocks) % p.Hkv;
  u.r = rest / (p.n_split * p.row_blocks * p.Hkv);
  const int gsize = p.Hq / p.Hkv;
  const TreeReq tr = tree_request(p.seq_lens, p.q_lens, p.Lq, u.b);
  u.base = tr.base;
  u.turns = p.turns;
  u.row0 = mb * p.block_rows;
  u.R_out = min(p.block_rows, p.Lq * gsize - u.row0);
  u.R = min(max(tr.n * gsize - u.row0, 0), u.R_out);
  u.L = tr.bad ? 0 : local_len(p.seq_lens[u.b], u.r, p.I, p.N);
  u.bad = tr.bad || (long long)u.L > (long long)p.max_lb * p.bs;     // (a short table: what it has)
  u.L = (int)min((long long)u.L, (long long)p.max_lb * p.bs);
  u.ctx = local_count_upto(tr.base - 1, u.r, p.I, p.N);
  u.kb = min(u.L, u.s_idx * p.split_tokens);
  u.ke = min(u.L, u.kb + p.split_tokens);
  u.T = u.R > 0 ? (u.ke - u.kb + kNt - 1) / kNt : 0;
  return u;
}

template <int D>
constexpr size_t tile_bytes() { return (size_t)kNt * D * 2; }

template <int D>
size_t smem_bytes(int q_bytes, int slots) {
  return 1024 + q_bytes + slots * tile_bytes<D>() + sizeof(Smem) + 16;
}

template <int D>
int ring_slots(int q_bytes) {
  const int n = (int)((kSmemLimit - smem_bytes<D>(q_bytes, 0)) / tile_bytes<D>());
  return std::min(n, kMaxSlots);
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float fmax3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// Paired fp32 arithmetic (each half rounds as the scalar operation does).
__device__ __forceinline__ float2 ffma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 ra, rb, rc, rd;\n\t"
      "mov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\tmov.b64 rc, {%6, %7};\n\t"
      "fma.rn.f32x2 rd, ra, rb, rc;\n\tmov.b64 {%0, %1}, rd;\n\t}"
      : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}

__device__ __forceinline__ float2 fadd2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 ra, rb, rd;\n\t"
      "mov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\t"
      "add.rn.f32x2 rd, ra, rb;\n\tmov.b64 {%0, %1}, rd;\n\t}"
      : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}

// Keep non-finite values out of the product: half `hf` of the row of key j at
// `v` (chunks of 64 dims, 128-byte rows).  Past the range the row becomes 0; a
// node's row loses the entries that are not finite and is marked.
template <int D>
__device__ __forceinline__ void clean_value_row(const Unit& u, uint32_t* odd_keys, uint8_t* v, int jj, int hf) {
  const bool past = jj >= u.ke;
  if (!past && jj < u.ctx) return;
  bool odd = false;
#pragma unroll 4
  for (int i = 0; i < D / 16; ++i) {
    // 16-byte pieces of the row, whatever their place under the swizzle
    // (threads start at different pieces, so that their rows do not meet in a bank)
    const int c = hf * (D / 16) + i;
    uint4* p = reinterpret_cast<uint4*>(v + (c >> 3) * (kNt * 128) + (D == 64 ? (c ^ jj) & 3 | c & 4 : (c ^ jj) & 7) * 16);
    uint4 x = *p;
    if (past) {
      if ((x.x | x.y | x.z | x.w) != 0u) *p = make_uint4(0u, 0u, 0u, 0u);
      continue;
    }
    if (drop_non_finite(x)) *p = x, odd = true;
  }
  if (odd) {
    const int bit = jj - max(u.kb, u.ctx);
    atomicOr(&odd_keys[bit >> 5], 1u << (bit & 31));
  }
}

// What a stream's softmax carries from unit to unit.
struct StreamState {
  unsigned item = 0, step = 0;     // ring items and steps so far
  uint32_t o_par = 0;              // parity of the next unit's o_full
};

// Softmax of one stream (128 threads, thread = row) over one unit, and its share
// of the output; false: the unit was aborted (its rows are 0 and -inf).
template <int D>
__device__ __forceinline__ bool stream(const Params& p, Smem& sm, const Unit& u, uint32_t* odd_keys, StreamState& st,
                                       uint8_t* qs, uint8_t* ring, uint32_t tmem, int warp, int lane) {
  const int w = (warp - 4) >> 2, quad = warp & 3, lrow = quad * 32 + lane;
  const uint32_t lanes = tmem + ((uint32_t)(quad * 32) << 16);
  const uint32_t tS = lanes + 128u * w, tO = lanes + kColO + 128u * w;
  const float sl2 = p.scale_log2;
  volatile int* abort_flag = &sm.abort;
  const int steps = u.steps(w);
  // steps whose first key is at most this one hold context keys alone
  const int plain = min(u.ctx, u.ke) - kNs;
  auto row_of = [&]() { return u.turns ? lrow : 128 * w + lrow; };             // row of the block
  auto mask_of = [&]() -> const uint32_t* {                                     // null: a row without a node
    const int row = row_of();
    if (row >= u.R) return nullptr;
    return p.mask + u.b * p.mask_stride + (long long)((u.row0 + row) / (p.Hq / p.Hkv)) * p.words;
  };

  const bool idle = (u.turns ? quad * 32 : 128 * w + quad * 32) >= u.R;
  float m = -INFINITY, l = 0.f;
  float heavy_at = -INFINITY;            // a score above it is heavy, or moves the reference
  bool bad = false;
#pragma unroll 1
  for (int s = 0; s < steps; ++s) {
    const unsigned gs = st.step + s;
    const int buf = gs & 1;
    const uint32_t tB = tS + kNs * buf;
    if (!__all_sync(0xffffffffu, *abort_flag == 0 && mbar_wait(smem_u32(&sm.s_full[w][buf]), (gs >> 1) & 1u, p.wait_ns))) {
      bad = true;
      break;
    }
    uint32_t x[kNs];
    tc_fence_after();
#pragma unroll
    for (int c = 0; c < 2; ++c) tmem_ld32(tB + 32 * c, *reinterpret_cast<uint32_t(*)[32]>(&x[32 * c]));
    tmem_wait_ld();
    {
      // the second terms are zero unless this warp finds a heavy probability
      // below (another warp of the stream may have one)
      const uint32_t zero[16] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u};
      tmem_st16(tB + 32, zero);
      tmem_st16(tB + 48, zero);
    }
    const int j0 = u.key(w, s);
    if (j0 > plain) {
      // nodes or the end of the range
      const uint32_t* mask_row = mask_of();
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const uint32_t sees = tree_sees32(mask_row, p.words, u.ctx, u.ke, u.base, u.r, p.I, p.N, j0 + 32 * c);
        if (__any_sync(0xffffffffu, sees != 0xffffffffu)) {
#pragma unroll
          for (int k = 0; k < 32; ++k)
            if (!((sees >> k) & 1u)) x[32 * c + k] = 0xff800000u;
        }
      }
      // the values, before this stream's product reads them (on a tile that
      // both streams use, each cleans it: the second finds nothing to do)
      const Ring rg(p, w);
      const unsigned item = st.item + (unsigned)(s | 1);
      const int slot = rg.slot(item);
      if (!__all_sync(0xffffffffu, mbar_wait(smem_u32(&sm.full[slot]), rg.lap(item) & 1u, p.wait_ns))) {
        bad = true;
        break;
      }
      const int k = (s & 1) * kNs + (lrow & 63);
      clean_value_row<D>(u, odd_keys, ring + slot * tile_bytes<D>() + k * 128, j0 + (lrow & 63), lrow >> 6);
      fence_proxy_async_smem();
    }
    if (idle) {
      // no row of this warp attends: its probabilities are the scores' own bits,
      // which meet no other row
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&sm.p_full[w][buf]));
      continue;
    }
    auto f = [&](int k) { return __uint_as_float(x[k]); };
    float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
    for (int k = 0; k < kNs; k += 8)
#pragma unroll
      for (int e = 0; e < 4; ++e) mx[e] = fmax3(mx[e], f(k + e), f(k + 4 + e));
    const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * sl2;
    const bool heavy = __any_sync(0xffffffffu, top > heavy_at);
    if (heavy) {
      const bool moves = top > m + kLazyLog2;
      if (__any_sync(0xffffffffu, moves)) {
        const float to = moves ? top : m;
        const float alpha = !moves ? 1.f : m == -INFINITY ? 0.f : ex2(m - to);
        m = to;
        l *= alpha;
        if (s > 0) {
          // O moves with the reference, once the previous product has landed
          // (the one before it did before this step's scores went out, so the
          // parity is unambiguous)
          if (!__all_sync(0xffffffffu, mbar_wait(smem_u32(&sm.pv_done[w]), (gs - 1) & 1u, p.wait_ns))) {
            bad = true;
            break;
          }
          tc_fence_after();
#pragma unroll 1
          for (int c = 0; c < D; c += 32) {
            uint32_t o[32];
            tmem_ld32(tO + c, o);
            tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * alpha);
            tmem_st32(tO + c, o);
          }
        }
      }
    }
    const float ref = m == -INFINITY ? 0.f : -m;
    float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
    uint32_t hi[32];
#pragma unroll
    for (int k = 0; k < 32; ++k) {
      const float2 y = ffma2(make_float2(f(2 * k), f(2 * k + 1)), make_float2(sl2, sl2), make_float2(ref, ref));
      const float2 e = make_float2(ex2(y.x), ex2(y.y));
      sum[k & 1] = fadd2(sum[k & 1], e);
      hi[k] = pack_bf16x2(e.x, e.y);
      x[2 * k] = __float_as_uint(e.x);
      x[2 * k + 1] = __float_as_uint(e.y);
    }
    tmem_st32(tB, hi);
    if (heavy) {
#pragma unroll
      for (int k = 0; k < 32; ++k)
        hi[k] = pack_bf16x2(f(2 * k) - bf16_lo(hi[k]), f(2 * k + 1) - bf16_hi(hi[k]));
      tmem_st32(tB + 32, hi);
      if (lane == 0) *(volatile unsigned*)&sm.heavy[w][buf] = gs + 1;
    }
    tmem_wait_st();
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&sm.p_full[w][buf]));
    l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
    heavy_at = fminf(m + __log2f(l) - kHeavyLog2, m + kLazyLog2);
  }
  bool have = !bad;
  if (have && steps > 0)
    have = __all_sync(0xffffffffu, mbar_wait(smem_u32(&sm.o_full[w]), st.o_par, p.wait_ns));
  if (!have) {
    set_status(p.status, DCP_ERR_TIMEOUT);
    *abort_flag = 1;
  }
  // one decision for the CTA: every product landed (the query's shared memory
  // is idle from here on: it carries m and l across the streams, then stages O)
  have = !bar_red_or(kBarEpi, 256, !have);
  tc_fence_after();
  st.step += (unsigned)steps;
  st.item += 2u * (unsigned)u.tiles(w);
  st.o_par ^= steps > 0 ? 1u : 0u;

  const int gsize = p.Hq / p.Hkv;
  const int row = row_of();
  const uint32_t* mask_row = mask_of();
  // in turn, both streams hold the row: each writes half of its dims
  float w0 = 1.f, w1 = 0.f;             // weights of this stream's and the other's O
  const bool other = u.turns && u.steps(w ^ 1) > 0;
  if (u.turns) {
    float* share = reinterpret_cast<float*>(qs);
    share[(2 * w) * kNt + lrow] = m;
    share[(2 * w + 1) * kNt + lrow] = l;
    named_bar_sync(kBarEpi, 256);
    const float m2 = share[(2 * (w ^ 1)) * kNt + lrow], l2 = share[(2 * (w ^ 1) + 1) * kNt + lrow];
    named_bar_sync(kBarEpi, 256);
    const float top = fmaxf(m, m2);
    const float ref = top == -INFINITY ? 0.f : top;
    w0 = ex2(m - ref);
    w1 = ex2(m2 - ref);
    l = l * w0 + l2 * w1;
    m = top;
  }
  const bool live = have && row < u.R && !(l == 0.f);
  const float inv = live ? 1.f / l : 0.f;
  w0 *= inv;
  w1 *= inv;
  const int d0 = u.turns ? w * (D / 2) : 0;
  const uint32_t tOther = lanes + kColO + 128u * (w ^ 1);
  auto dst_row = [&](int rr) {
    const int i = rr / gsize, head = u.g * gsize + rr % gsize;
    return ((((long long)u.r * p.B + u.b) * p.Lq + i) * p.n_split + u.s_idx) * p.Hq + head;
  };
  bool any_odd = false;
  for (int k = 0; k < 8; ++k) any_odd |= odd_keys[k] != 0;
  const bool writes = row < u.R_out;
  const unsigned long long out = writes ? (unsigned long long)(p.dst_o + dst_row(u.row0 + row) * D) : 0ull;
  // 32 dims at a time through 4 KB of the query's memory, so that a row's part
  // goes out as one 128-byte line (a rolled loop: the code runs once a unit, and
  // fetching it is what it costs)
  const int chunks = (u.turns ? D / 2 : D) / 32;
  uint8_t* mine = qs + (warp - 4) * 4096;
#pragma unroll 1
  for (int i = 0; i < chunks; ++i) {
    if (have) {
      const int c = d0 + 32 * i;
      uint32_t o[32];
      if (steps > 0) {
        tmem_ld32(tO + c, o);
        tmem_wait_ld();
      }
#pragma unroll
      for (int k = 0; k < 32; ++k) o[k] = live && steps > 0 ? __float_as_uint(__uint_as_float(o[k]) * w0) : 0u;
      if (other) {
        uint32_t o2[32];
        tmem_ld32(tOther + c, o2);
        tmem_wait_ld();
        if (live) {
#pragma unroll
          for (int k = 0; k < 32; ++k)
            o[k] = __float_as_uint(fmaf(__uint_as_float(o2[k]), w1, __uint_as_float(o[k])));
        }
      }
      if (any_odd && live) {
        // values of nodes that are not finite: added to the rows that see them
#pragma unroll 1
        for (int bit = 0; bit < DCP_TREE_MAX_NODES; ++bit) {
          if (!((odd_keys[bit >> 5] >> (bit & 31)) & 1u)) continue;
          const int jj = max(u.kb, u.ctx) + bit;
          if (!tree_bit(mask_row, (int)(global_pos(jj, u.r, p.I, p.N) - u.base))) continue;
          const int blk = p.block_tables[((long long)u.r * p.B + u.b) * p.max_lb + jj / p.bs];
          const __nv_bfloat16* v = p.v_pool + (((long long)blk * p.bs + jj % p.bs) * p.Hkv + u.g) * D + c;
#pragma unroll
          for (int k = 0; k < 32; ++k) {
            const float e = __bfloat162float(v[k]);
            if (!(fabsf(e) < INFINITY)) o[k] = __float_as_uint(__uint_as_float(o[k]) + e);
          }
        }
      }
#pragma unroll
      for (int k = 0; k < 8; ++k)
        *reinterpret_cast<uint4*>(mine + lane * 128 + ((k ^ (lane & 7)) << 4)) =
            make_uint4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
    }
    __syncwarp();
    // (all reads before the first store: branch by branch they took 170 cycles each)
    uint4 v[8];
#pragma unroll
    for (int it = 0; it < 8; ++it) {
      const int rr = it * 4 + (lane >> 3), k = lane & 7;
      v[it] = *reinterpret_cast<const uint4*>(mine + rr * 128 + ((k ^ (rr & 7)) << 4));
    }
#pragma unroll
    for (int it = 0; it < 8; ++it) {
      const int rr = it * 4 + (lane >> 3), k = lane & 7;
      const unsigned long long to = __shfl_sync(0xffffffffu, out, rr);
      if (!have) v[it] = make_uint4(0u, 0u, 0u, 0u);
      if (to != 0ull) *reinterpret_cast<uint4*>(reinterpret_cast<float*>(to) + d0 + 32 * i + 4 * k) = v[it];
    }
    __syncwarp();
  }
  if (writes && (!u.turns || w == 0))
    p.dst_lse[dst_row(u.row0 + row)] = live ? (m + log2f(l)) * 0.69314718055994531f : -INFINITY;
  return have;
}

// Zeros and -inf for a unit that is not run (256 threads).
template <int D>
__device__ __forceinline__ void write_empty(const Params& p, const Unit& u, int warp, int lane) {
  const int gsize = p.Hq / p.Hkv;
  for (int rr = warp - 4; rr < u.R_out; rr += 8) {
    const int i = (u.row0 + rr) / gsize, head = u.g * gsize + (u.row0 + rr) % gsize;
    const long long to = ((((long long)u.r * p.B + u.b) * p.Lq + i) * p.n_split + u.s_idx) * p.Hq + head;
    for (int c = 4 * lane; c < D; c += 128)
      *reinterpret_cast<uint4*>(p.dst_o + to * D + c) = make_uint4(0u, 0u, 0u, 0u);
    if (lane == 0) p.dst_lse[to] = -INFINITY;
  }
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
tree_gqa_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v, const Params p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* qs = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  constexpr uint32_t kTile = (uint32_t)tile_bytes<D>();
  uint8_t* ring = qs + p.q_bytes;
  Smem& sm = *reinterpret_cast<Smem*>(ring + p.slots * kTile);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    prefetch_tmap(&tm_k);
    prefetch_tmap(&tm_v);
    for (int k = 0; k < p.slots; ++k) {
      mbar_init(smem_u32(&sm.full[k]), 1);
      mbar_init(smem_u32(&sm.empty[k]), p.turns ? 1 : 2);   // streams that read the tile
    }
    for (int k = 0; k < 2; ++k) {
      for (int b = 0; b < 2; ++b) {
        mbar_init(smem_u32(&sm.s_full[k][b]), 1);
        mbar_init(smem_u32(&sm.p_full[k][b]), 4);    // warps of the stream
        sm.heavy[k][b] = 0;
      }
      mbar_init(smem_u32(&sm.pv_done[k]), 1);
      mbar_init(smem_u32(&sm.o_full[k]), 1);
      mbar_init(smem_u32(&sm.drain[k]), 1);
      mbar_init(smem_u32(&sm.q_full[k]), 8);         // softmax warps
      mbar_init(smem_u32(&sm.unit_full[k]), 1);
      mbar_init(smem_u32(&sm.unit_free[k]), 11);     // a producer, two issuers, eight softmax warps
    }
    sm.abort = 0;
    fence_mbar_init();
  }
  if (warp == 1) tmem_alloc(smem_u32(&sm.tmem_base), 512);
  if (p.B <= kLptMaxBatch) {
    // units go longest request first: rank the requests by counting
    int* lens = reinterpret_cast<int*>(ring);              // idle until the first load
    const int sj = tid < p.B ? p.seq_lens[tid] : 0;
    if (tid < p.B) lens[tid] = sj;
    __syncthreads();
    if (tid < p.B) {
      int rank = 0;
#pragma unroll 8
      for (int i = 0; i < p.B; ++i) {
        const int si = lens[i];
        rank += (si > sj) || (si == sj && i < tid);
      }
      sm.order[rank] = (uint8_t)tid;
    }
    fence_proxy_async_smem();                              // before the loads into the ring
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem_base;
  volatile int* abort_flag = &sm.abort;
  auto fail = [&](void) {
    set_status(p.status, DCP_ERR_TIMEOUT);
    *abort_flag = 1;
  };
  // unit n, once warp 0 has put it there
  auto unit_ready = [&](int n) {
    return *abort_flag == 0 && mbar_wait(smem_u32(&sm.unit_full[n & 1]), (uint32_t)(n >> 1) & 1u, p.wait_ns);
  };
  auto unit_done = [&](int n) { mbar_arrive(smem_u32(&sm.unit_free[n & 1])); };

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" :: "n"(kCtrlRegs));
    if (warp == 0 || warp == 3) {
      // ---------------- TMA producers; warp 0 also makes the units ----------------
      // in turn: warp 0 loads stream 0's tiles, warp 3 stream 1's; else warp 0 K, warp 3 V
      const int w = warp == 0 ? 0 : 1;
      const int box_rows = p.bs < kNt ? p.bs : kNt;
      const int from = p.turns ? 0 : w, by = p.turns ? 1 : 2;
      const Ring rg(p, w);
      unsigned item0 = 0, end = 0;                         // items before this unit; one past the last loaded
      bool ok = true;
      for (int n = 0; ok; ++n) {
        const int index = unit_of(p, n);
        if (index < 0) break;
        Unit& u = sm.unit[n & 1];
        if (warp == 0) {
          if (n >= 2 && !__all_sync(0xffffffffu, *abort_flag == 0 && mbar_wait(smem_u32(&sm.unit_free[n & 1]),
                                                                             (uint32_t)((n >> 1) - 1) & 1u, p.wait_ns))) {
            ok = false;
            break;
          }
          Unit v = make_unit(p, sm, index);
          // a block id past the pool among the shard's keys skips the unit, and with
          // it every row of the request in the shard (without a row to attend, as in
          // a padded request, the table is not read)
          const int32_t* bt = p.block_tables + ((long long)v.r * p.B + v.b) * p.max_lb;
          bool bad_blk = false;
          for (int jb = lane; v.R > 0 && jb < (v.L + p.bs - 1) / p.bs; jb += 32) bad_blk |= (unsigned)bt[jb] >= (unsigned)p.num_blocks;
          bad_blk = __any_sync(0xffffffffu, bad_blk);
          if (bad_blk) v.T = 0;
          if (lane < 8) sm.odd[n & 1][lane] = 0;
          if (lane == 0) {
            if (v.bad || bad_blk) set_status(p.status, DCP_ERR_BOUNDS);
            u = v;
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&sm.unit_full[n & 1]));
        } else if (!__all_sync(0xffffffffu, unit_ready(n))) {
          ok = false;
          break;
        }
        const int items = 2 * u.tiles(w);
        const int32_t* bt = p.block_tables + ((long long)u.r * p.B + u.b) * p.max_lb;
        const int kb = u.kb, ke = u.ke, g = u.g;
        // pool row of box `lane` of key tile t (boxes past the key range read row
        // 0: masked, values zeroed), found a tile ahead
        auto row_of = [&](int t) {
          const int j = kb + t * kNt + lane * box_rows;
          return lane * box_rows < kNt && j < ke ? bt[j / p.bs] * p.bs + j % p.bs : 0;
        };
        int next = from < items ? row_of(u.tile(w, from >> 1)) : 0, row = 0;
        for (int at = from; at < items; at += by) {
          const unsigned item = item0 + (unsigned)at;
          const int slot = rg.slot(item);
          const uint32_t lap = rg.lap(item);
          if (by == 2 || !(at & 1)) {                       // (V's rows are K's)
            row = next;
            if ((at >> 1) + 1 < items / 2) next = row_of(u.tile(w, (at >> 1) + 1));
          }
          if (!__all_sync(0xffffffffu, *abort_flag == 0 && (lap == 0 || mbar_wait(smem_u32(&sm.empty[slot]), (lap - 1) & 1u,
                                                                                   p.wait_ns)))) {
            ok = false;
            break;
          }
          if (u.tile(w, at >> 1) == p.skip_tile && !(at & 1)) continue;    // test hook: a tile that never comes
          const CUtensorMap* tm = (at & 1) ? &tm_v : &tm_k;
          const uint32_t full = smem_u32(&sm.full[slot]);
          uint8_t* dst = ring + slot * kTile;
          if (lane == 0) mbar_arrive_expect_tx(full, kTile);
          for (int k = 0; k < kNt; k += box_rows) {
            const int to = __shfl_sync(0xffffffffu, row, k / box_rows);
            if (lane == 0) {
#pragma unroll
              for (int c = 0; c < D / 64; ++c)
                tma_load_3d(smem_u32(dst + c * (kNt * 128) + k * 128), tm, 64 * c, g, to, full);
            }
          }
          end = item + 1;
        }
        item0 += (unsigned)items;
        if (warp == 3 && lane == 0) unit_done(n);
      }
      if (!ok) fail();
      if (lane == 0 && *abort_flag) {
        // let every copy this thread issued land before the CTA exits (the last lap of each slot)
        for (unsigned back = 1; back <= (unsigned)rg.len && back <= end; ++back) {
          const unsigned item = end - back;
          if (p.turns || (item & 1u) == (unsigned)w)
            mbar_wait(smem_u32(&sm.full[rg.slot(item)]), rg.lap(item) & 1u, p.wait_ns);
        }
      }
    } else {
      // ---------------- MMA issuers, warp 1 + w for stream w ----------------
      // PV(s), then the scores of step s + 2, whose buffer P(s) leaves.  The
      // whole warp runs the loop on uniform values and one lane issues: with a
      // single lane in the loop each MMA cost 65-90 clocks to issue, as long as
      // it runs.
      // The query's barrier goes by the unit's parity.  In turn a stream may have
      // no step in a unit (one tile) and pass it while its query is still being
      // staged; on one barrier its next wait would then be a phase ahead of the
      // open one and pass at once, and if it waited for the unit it has no part
      // in, the other stream could be two phases on before it looks.  A unit is
      // published only when the one two before it has left, so on its own barrier
      // every earlier phase is over, and the next one needs this stream's output.
      const int w = (int)uniform((uint32_t)warp - 1u);
      constexpr uint32_t id_qk = idesc_bf16(128, kNs, false);
      constexpr uint32_t id_pv = idesc_bf16(128, D, true);
      const bool turns = p.turns, lead = elect_one();
      const Ring rg(p, w);
      const int first = (int)uniform((uint32_t)rg.first), limit = first + (int)uniform((uint32_t)rg.len);
      const uint32_t tm = uniform(tmem);
      const uint32_t ring_addr = uniform(smem_u32(ring)), qt = uniform(smem_u32(qs) + (turns ? 0u : w * kTile));
      const uint32_t full = uniform(smem_u32(&sm.full[0])), empty = uniform(smem_u32(&sm.empty[0]));
      const uint32_t s_full = uniform(smem_u32(&sm.s_full[w][0])), p_full = uniform(smem_u32(&sm.p_full[w][0]));
      const uint32_t pv_done = uniform(smem_u32(&sm.pv_done[w])), o_full = uniform(smem_u32(&sm.o_full[w]));
      const uint32_t q_full = uniform(smem_u32(&sm.q_full[0]));
      // cursors over the K and the V tiles: slot and lap parity (a tile serves two steps)
      struct Cursor {
        int slot;
        uint32_t par;
      };
      auto wait = [&](uint32_t bar, uint32_t par) {
        return __all_sync(0xffffffffu, *abort_flag == 0 && mbar_wait(bar, par, p.wait_ns));
      };
      auto next = [&](Cursor& c) {          // two items on
        c.slot += 2;
        if (c.slot >= limit) {
          c.slot -= limit - first;
          c.par ^= 1u;
        }
      };
      Cursor kc = {first, 0u}, vc = {first + 1, 0u};
      unsigned step0 = 0;                   // steps before this unit
      uint32_t q_par = 0;                   // bit n & 1: parity of that barrier's next phase
      bool ok = true;
      for (int n = 0; ok; ++n) {
        if (unit_of(p, n) < 0) break;
        if (!__all_sync(0xffffffffu, unit_ready(n))) {
          ok = false;
          break;
        }
        const int steps = (int)uniform((uint32_t)sm.unit[n & 1].steps(w));
        const bool runs = uniform((uint32_t)sm.unit[n & 1].T) > 0;
        if (lead) unit_done(n);
        // scores of step s into their buffer
        auto qk = [&](int s) -> bool {
          if (!(s & 1) && !wait(full + 8 * kc.slot, kc.par)) return false;
          const uint32_t kt = ring_addr + kc.slot * kTile + (s & 1) * (kNs * 128), buf = (step0 + s) & 1u;
          const bool done = (s & 1) || s + 1 == steps;      // the tile's last step
          if (lead) {
            tc_fence_after();
#pragma unroll
            for (int k = 0; k < D / 16; ++k)
              mma_ss(tm + 128u * w + kNs * buf, smem_desc(qt + (k >> 2) * (kNt * 128) + (k & 3) * 32, 16, 1024, kSw128),
                     smem_desc(kt + (k >> 2) * (kNt * 128) + (k & 3) * 32, 16, 1024, kSw128), id_qk, k > 0 ? 1u : 0u);
            mma_commit(s_full + 8 * buf);
            if (done) mma_commit(empty + 8 * kc.slot);
          }
          if (done) next(kc);
          return true;
        };
        auto pv = [&](int s) -> bool {
          const uint32_t gs = step0 + s, buf = gs & 1u;
          if ((!(s & 1) && !wait(full + 8 * vc.slot, vc.par)) || !wait(p_full + 8 * buf, (gs >> 1) & 1u)) return false;
          tc_fence_after();
          const uint32_t vt = ring_addr + vc.slot * kTile + (s & 1) * (kNs * 128), pt = tm + 128u * w + kNs * buf;
          const bool heavy = __any_sync(0xffffffffu, *(volatile unsigned*)&sm.heavy[w][buf] == gs + 1);
          const bool done = (s & 1) || s + 1 == steps;
          if (lead) {
#pragma unroll
            for (int k = 0; k < kNs / 16; ++k)
              mma_ts(tm + kColO + 128u * w, pt + 8 * k, smem_desc(vt + k * 2048, kNt * 128, 1024, kSw128), id_pv,
                     (s > 0 || k > 0) ? 1u : 0u);
            if (heavy) {
#pragma unroll
              for (int k = 0; k < kNs / 16; ++k)
                mma_ts(tm + kColO + 128u * w, pt + 32 + 8 * k, smem_desc(vt + k * 2048, kNt * 128, 1024, kSw128), id_pv, 1u);
            }
            mma_commit(pv_done);
            if (s + 1 == steps) mma_commit(o_full);
            if (done) mma_commit(empty + 8 * vc.slot);
          }
          if (done) next(vc);
          return true;
        };
        if (steps > 0) ok = wait(q_full + 8 * (n & 1), (q_par >> (n & 1)) & 1u) && qk(0) && (steps < 2 || qk(1));
        for (int s = 0; s < steps && ok; ++s) ok = pv(s) && (s + 2 >= steps || qk(s + 2));
        step0 += (unsigned)steps;
        q_par ^= runs ? 1u << (n & 1) : 0u;
      }
      if (!ok) fail();
      if (lead) mma_commit(smem_u32(&sm.drain[w]));
      if (!mbar_wait(smem_u32(&sm.drain[w]), 0, p.wait_ns)) fail();
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" :: "n"(kSoftRegs));
    StreamState st;
    const int gsize = p.Hq / p.Hkv;
    bool ok = true;
    int n = 0;
    for (; unit_of(p, n) >= 0; ++n) {
      // the last unit's output has left the query's memory; the streams leave
      // the loop together
      const bool ready = unit_ready(n);
      if (bar_red_or(kBarEpi, 256, !ready)) {
        ok = false;
        break;
      }
      const Unit& u = sm.unit[n & 1];
      if (u.T > 0) {
        // query rows -> shared memory, K-major with the 128-byte swizzle (rows
        // past R are zero), while the first tiles are on their way
        const int rows = p.turns ? kNt : 2 * kNt;
        constexpr int kPer = D / 8;                        // 16-byte pieces of a row
        constexpr int kStep = 256 / kPer;
        const int c = (tid - 128) % kPer;
        int i = (u.row0 + (tid - 128) / kPer) / gsize, hh = (u.row0 + (tid - 128) / kPer) % gsize;   // node and head of row rr
        const int di = kStep / gsize, dh = kStep % gsize;
        const __nv_bfloat16* q = p.q + (((long long)u.b * p.Lq) * p.Hq + u.g * gsize) * D + 8 * c;
#pragma unroll 2
        for (int rr = (tid - 128) / kPer; rr < rows; rr += kStep) {
          const int lr = rr & 127;
          const uint32_t dst = smem_u32(qs + (rr >> 7) * kTile + (c >> 3) * (kNt * 128) + lr * 128 + (((c & 7) ^ (lr & 7)) << 4));
          // (a row past R: zero bytes from an address inside the query)
          const bool there = rr < u.R;
          cp_async_16(dst, there ? q + ((long long)i * p.Hq + hh) * D : q, there ? 16u : 0u);
          i += di;
          hh += dh;
          if (hh >= gsize) hh -= gsize, ++i;
        }
        cp_async_wait_all();
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sm.q_full[n & 1]));
      }
      ok = stream<D>(p, sm, u, sm.odd[n & 1], st, qs, ring, tmem, warp, lane);
      __syncwarp();
      if (lane == 0) unit_done(n);
      if (!ok) {
        ++n;
        break;
      }
    }
    // after an abort: the CTA's other units are empty
    if (!ok)
      for (int index; (index = unit_of(p, n)) >= 0; ++n) write_empty<D>(p, make_unit(p, sm, index), warp, lane);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

int rows_of(const AttnArgs& a) { return a.Lq * (a.Hq / a.Hkv); }
// Rows of a block.  Pairs of 128 share a key tile; an odd one holds an SM for a
// pair's time, which counts for most where there are few; in turn there are twice the
// units, which fill the SMs better.  Time in turn against in pairs, over 25 to 40
// shapes each (1 to 64 requests of unlike lengths up to 60,000, 1 to 8 KV heads, 1
// to 4 shards), geometric mean and range: two blocks 0.94 (0.67-1.46), three 0.84
// (0.51-1.18), four 0.94 (0.68-1.22), five 0.86 (0.57-1.15), six 0.96 (0.68-1.45),
// seven 0.90 (0.62-1.26).  Where many equal units fill the SMs either way the passes
// over the cache decide (64 requests of 2,048 tokens, 64 and 4 heads, 4 shards):
// three blocks 1.00, five 1.06, seven 1.12, even ones 1.20 and more, 15 to 31 1.21 to
// 1.28; 16 requests of 8,192: three and five 0.91, seven 1.00, 9 to 31 1.02 to 1.13.
// So three and five go in turn, where the gain is the largest and the loss small.
int block_rows_of(const AttnArgs& a) {
  const int n = (rows_of(a) + kNt - 1) / kNt;
  return n == 1 || n == 3 || n == 5 ? kNt : 2 * kNt;
}
int row_blocks_of(const AttnArgs& a) { return (rows_of(a) + block_rows_of(a) - 1) / block_rows_of(a); }

template <int D>
cudaError_t launch(const CUtensorMap& tm_k, const CUtensorMap& tm_v, Params& p, cudaStream_t stream) {
  // (the query's memory also stages the output: 4 KB a softmax warp at the least)
  p.q_bytes = std::max(p.block_rows / kNt * (int)tile_bytes<D>(), 8 * 4096);
  p.slots = ring_slots<D>(p.q_bytes);
  const size_t smem = smem_bytes<D>(p.q_bytes, p.slots);
  // the register split assumes the compiled launch count; refuse to launch
  // otherwise (setmaxnreg.inc would wait for registers that do not exist)
  cudaFuncAttributes fa;
  cudaError_t e = cudaFuncGetAttributes(&fa, tree_gqa_kernel<D>);
  if (e != cudaSuccess) return e;
  if (fa.numRegs * kThreads < 128 * kCtrlRegs + 256 * kSoftRegs) return cudaErrorInvalidConfiguration;
  e = allow_smem(tree_gqa_kernel<D>);
  if (e != cudaSuccess) return e;
  const int grid = std::min(p.units, device_sm_count());
  tree_gqa_kernel<D><<<(unsigned)grid, kThreads, smem, stream>>>(tm_k, tm_v, p);
  return cudaGetLastError();
}

}  // namespace

// Head dim 64 or 128; block sizes as the decode kernel takes them.
bool tree_gqa_supported(const AttnArgs& a) {
  if (a.kind != DCP_ATTN_GQA || (a.Dqk != 64 && a.Dqk != 128) || a.Dv != a.Dqk) return false;
  if (a.bs % 8 || (a.bs >= kNt ? a.bs % kNt : kNt % a.bs)) return false;
  if ((long long)a.Lq * (a.Hq / a.Hkv) > (1LL << 20)) return false;
  return (long long)a.num_blocks * a.bs < (1LL << 31);
}

SplitPlan plan_tree_gqa(const AttnArgs& a, int sm_count) {
  return plan_splits(a, sm_count, kNt, a.Hkv * row_blocks_of(a));
}

cudaError_t launch_tree_gqa(const AttnArgs& a, const SplitPlan& plan) {
  CUtensorMap tm_k, tm_v;
  const uint64_t rows = (uint64_t)a.num_blocks * a.bs;
  const uint64_t dims[3] = {(uint64_t)a.Dqk, (uint64_t)a.Hkv, rows};
  const uint64_t strides[2] = {(uint64_t)a.Dqk * 2, (uint64_t)a.Hkv * a.Dqk * 2};
  const uint32_t box[3] = {64, 1, (uint32_t)(a.bs < kNt ? a.bs : kNt)};
  const char* k_pool = static_cast<const char*>(a.kv);
  const char* v_pool = k_pool + rows * a.Hkv * a.Dqk * 2;
  if (!make_tensor_map_bf16(&tm_k, k_pool, 3, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !make_tensor_map_bf16(&tm_v, v_pool, 3, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B))
    return cudaErrorInvalidValue;
  Params p{};
  p.q = static_cast<const __nv_bfloat16*>(a.q);
  p.v_pool = reinterpret_cast<const __nv_bfloat16*>(v_pool);
  p.block_tables = a.block_tables;
  p.seq_lens = a.seq_lens;
  p.q_lens = a.q_lens;
  p.mask = a.tree_mask;
  p.mask_stride = a.tree_mask_stride;
  p.words = a.tree_words;
  p.status = a.status;
  p.B = a.B, p.Lq = a.Lq, p.Hq = a.Hq, p.Hkv = a.Hkv, p.N = a.N, p.I = a.I;
  p.max_lb = a.max_lb, p.bs = a.bs, p.num_blocks = a.num_blocks;
  p.n_split = plan.n_split, p.split_tokens = plan.split_tokens;
  p.row_blocks = row_blocks_of(a), p.block_rows = block_rows_of(a);
  p.scale_log2 = a.scale * 1.4426950408889634f;
  p.wait_ns = test_hooks().wait_ns;
  p.skip_tile = test_hooks().skip_tile;
  p.dst_o = a.partial_out;
  p.dst_lse = a.lse;
  if (plan.n_split > 1) {
    const size_t o_bytes = (size_t)a.N * a.B * a.Lq * a.Hq * plan.n_split * a.Dv * sizeof(float);
    p.dst_o = static_cast<float*>(a.workspace);
    p.dst_lse = reinterpret_cast<float*>(static_cast<char*>(a.workspace) + ((o_bytes + 255) & ~size_t(255)));
  }
  const long long units = (long long)a.N * a.B * a.Hkv * p.row_blocks * plan.n_split;
  if (units > INT32_MAX) return cudaErrorInvalidValue;
  p.units = (int)units;
  p.turns = p.block_rows == kNt;
  const cudaError_t e = a.Dqk == 128 ? launch<128>(tm_k, tm_v, p, a.stream) : launch<64>(tm_k, tm_v, p, a.stream);
  if (e != cudaSuccess || plan.n_split <= 1) return e;
  return launch_split_combine(a, plan);
}

}  // namespace dcp
