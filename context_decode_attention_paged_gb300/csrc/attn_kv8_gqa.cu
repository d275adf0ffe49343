// Step a3 over the 8-bit cache: per-shard partial attention for GQA on tcgen05
// tensor cores, e4m3 keys and values with a power-of-two scale per block and KV
// head.
//
// vLLM DCP blog, "DCP 執行流程", Compute step (each shard attends the full
// query to its local KV slice and returns a partial output with its LSE).
//
// Mathematics, per query row and key t (log2 domain):
//   x_t = scale log2 e * 2^ek_t q.k8_t,   y_t = x_t + ev_t
//   l = sum 2^(x_t - R),  o = sum 2^(y_t - R) v8_t / l,  lse = (R + log2 l) ln 2
// with ek, ev the exponents of the scales of t's block.  The value's scale goes
// into the probability's exponent, so what the value product multiplies by is
// P_t = 2^(y_t - R), and R follows the largest y, lazily: P stays below 2^15 and
// the row's largest one above 2^7.  fp16 then holds P to 2^-11 of itself down to
// 2^-21 of the row's largest.
//
// Products.  Few query rows, many keys: the keys sit on the MMA's 128 rows.
//   S^T = K8 Q^T     kind::f8f6f4.  A bf16 query value has 8 significant bits and
//                    is the sum of two e4m3 values (4 bits each) once its row is
//                    scaled to at most 256, so q.k8 takes two products on codes
//                    as they are: no key is converted.
//   O^T += V^T P^T   kind::f16.  P in e4m3 would need three terms, and rows whose
//                    weights lie far below the largest (a sink beside a hundred
//                    thousand others) more; instead a tile's values turn into fp16
//                    (exact), once for all rows: ldmatrix transposes their bytes
//                    (keys x dims -> dims x keys), and they go to tensor memory as
//                    the A operand.  Through shared memory (values written as fp16
//                    and read by the MMA) 256 requests took 1,300 us, so 1,140.
// Roles: warp 0 TMA producer (K and V tiles of 128 keys in rings of their own, the
// tile's scale bytes beside them), 1 QK issuer, 2 PV issuer, 3 scheduler, 4-7 query
// split and value conversion, 8 and up softmax and epilogue (a thread owns one key
// of the tile and 16 rows).  16 rows: 4 softmax warps and three CTAs an SM, 32: 8
// and two, 64: 16 and one; a CTA that starts or ends a unit leaves the SM to the
// others (one CTA an SM with 16 softmax warps: 1,546 us, two with 8: 906, three: 791).
//
// Work.  A unit is (request, shard, KV head, row tile); its tiles and a constant
// for its start and end are its weight.  A CTA takes an equal share of the summed
// weight, whatever the lengths: units that a border cuts leave partial rows in the
// workspace (two at most per CTA), joined by kv8_join_kernel.  CTAs go from unit
// to unit without a stop: the scheduler warp reads lengths and tables ahead and
// publishes unit descriptors, O has two TMEM buffers.
//
// Bound: HBM (128 bytes of a key and of a value a token and KV head; TMA fetches
// exactly these: with 256-byte L2 fetches the next head's row came along, 1.39 of
// the bytes and 1,142 against 906 us).  Measured (GB300, in a graph, with the merge):
//   256 requests of 8,192 - 32,768 tokens, 64 + 4 heads (4.66 GB)  769-790 us, 5.9-6.1 TB/s
//   one request of 200,000 tokens, 64 + 8 heads (410 MB)            93-99 us, 4.1-4.4 TB/s
//   33 requests, 4 ragged queries, blocks of 16 (370 MB)            104-106 us, 3.5 TB/s
//   one request of 1,024 tokens, 8 + 2 heads of 64                  15 us
// What is left of the first: unit ends (about 15,000 cycles, the others' time on the
// SM), of the second and third the first tiles (code fetched behind the rings' first
// copies) and the last CTAs.  Code counts: all roles share the instruction cache, and
// compact waits, ragged tiles masked by a loop and the rest of it took 139 to 96 KB
// and the ragged queries from 181 to 124 us.  A unit of nothing that warms the cache
// up before the first copies measured 1 to 5% slower, softmax warps that leave out absent
// rows (a loop of their own, of barriers alone) 3%.
//
// Few units are cut into up to a part a CTA, which one CTA joins: one request of 50,000
// tokens, 1 KV head and 16 rows takes 187 us, of 200,000 and 8 KV heads 116.
//
// Every wait is bounded; when one runs out the CTA records DCP_ERR_TIMEOUT, goes
// through its remaining units without work and leaves zeros and -inf for them.  So
// no warp that may give up alone meets others at a barrier, and nothing is written
// without the wait for where it goes.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <float.h>

#include <algorithm>
#include <climits>

#include "dcp_device.cuh"
#include "dcp_internal.h"
#include "dcp_sm100.cuh"
#include "dcp_tma.h"

namespace dcp {
namespace {

using namespace sm100;

constexpr int kNt = 128;                       // keys per tile (MMA M of S^T)
constexpr int kMaxStages = 6;
constexpr int kMaxBoxes = 16;                  // blocks of 8 tokens
constexpr int kMeta = 8;                       // tiles whose scale bytes are kept (K stages and 2 more at least)
constexpr int kConvWarp = 4, kSoftWarp = 8, kConvWarps = 4;
constexpr float kTop = 15.0f, kStart = 7.0f;   // log2 of the largest P, and of it after a move
constexpr float kNoRef = FLT_MAX;              // -R of a row that has seen no key: any y + kNoRef is above kTop, -inf stays
constexpr uint32_t kBarSoftmax = 1;            // (the one barrier where warps meet, and they leave it with one answer)
constexpr int kMaxCols = 64;
constexpr uint32_t kWCols = kNt / 2;           // TMEM columns of an fp16 value tile

struct Params {
  const __nv_bfloat16* q;
  const uint8_t* codes_v;                      // (NaN codes of hidden tokens)
  const uint8_t* scales;
  const int32_t *block_tables, *seq_lens, *q_lens;
  float *out, *lse;
  float *ws_o, *ws_lse;                        // partial rows: slots 2c (head) and 2c + 1 (tail) of CTA c
  long long* cut;                              // [2 grid] unit of a slot, -1
  int* status;
  int B, Lq, Hq, Hkv, N, I, max_lb, bs, num_blocks, m_tiles, gsize;
  int box_shift;                               // log2 of the tokens of a TMA box
  float scale_log2;
  uint32_t wait_ns;                            // limit of a wait, below 2^32
  int skip_tile;
};

template <int NCOL>
struct Unit {
  int b, r, g, row0, rows;                     // rows: query rows of the tile
  int n, first, keys;                          // queries of the request, position of the first; keys of the shard
  int t0, tiles;                               // first tile, tiles (-1: no more units)
  int ke, lim_min;                             // keys that some row sees; those below lim_min every live row sees
  int slot;                                    // partial slot, -1: final rows
  int nan_values;                              // hidden or ragged keys hold NaN values
  // written by the warps that split the query
  alignas(16) int lim[NCOL];                   // keys that a row sees (0: no such query)
  alignas(16) float qf[NCOL];                  // scale of the split query row
  long long at[NCOL];                          // where its output goes, in rows
};

template <int NCOL, int D>
struct Cfg {
  // a softmax thread holds 16 rows of its key: 4, 8 or 16 softmax warps, three, two or one CTA an SM
  static constexpr int kGroups = NCOL / 16, kCtas = NCOL == 16 ? 3 : NCOL == 32 ? 2 : 1;
  static constexpr int kSoftWarps = 4 * kGroups, kWarps = kSoftWarp + kSoftWarps;
  static constexpr uint32_t kThreads = 32 * kWarps, kSoftThreads = 32 * kSoftWarps;
  static constexpr int kReleases = 3 + kConvWarps + kSoftWarps;   // warps that read a unit descriptor
  // P^T tiles: a second one costs a stage with 16 rows alone (32 rows, one and two: 110 and 109 us)
  static constexpr int kBufs = NCOL == 16 ? 1 : 2;
  // Start and end of a unit, in tiles.  2, 4, 6: 33 requests of 4 ragged queries 109, 104, 109 us; 64 of one query 90,
  // 83, 82; of 12 queries (64 rows: nobody else on the SM meanwhile) 252, 213, 201; 256 long requests 789, 794, 794.
  static constexpr int kUnitCost = NCOL == 64 ? 6 : 4;
  static constexpr int kWBufs = NCOL == 16 ? 1 : 2;               // fp16 value tiles
  static constexpr size_t kSmemLimit = (kCtas == 1 ? 233472 : kCtas == 2 ? 116736 : 77824) - 1024;
  // registers of a thread at launch, and what setmaxnreg makes of them
  static constexpr int kLaunchRegs = NCOL == 16 ? 56 : NCOL == 32 ? 64 : 80;
  static constexpr int kCtrlRegs = NCOL == 64 ? 48 : 40, kConvRegs = NCOL == 64 ? 48 : 40, kSoftRegs = NCOL == 64 ? 96 : 88;
  static_assert(128 * (kCtrlRegs + kConvRegs) + (int)kSoftThreads * kSoftRegs <= (int)kThreads * kLaunchRegs, "registers");
  static constexpr uint32_t kTile = kNt * D;                      // bytes of a K or V tile
  static constexpr uint32_t kQBytes = 2 * NCOL * D;               // split query: hi rows, lo rows
  static constexpr int kUnits = 2;
  static constexpr uint32_t kPitch = NCOL * 2;                    // bytes of one P^T row (key)
  static constexpr uint32_t kPBytes = kNt * kPitch;
  static constexpr uint32_t kPSwz = NCOL == 16 ? kSw32 : NCOL == 32 ? kSw64 : kSw128;
  static constexpr uint32_t kKSwz = D == 128 ? kSw128 : kSw64;
  static constexpr uint32_t kTmemCols = NCOL == 16 ? 128 : NCOL == 32 ? 256 : 512;   // two S, two O, the value tiles
  __device__ static __forceinline__ uint32_t pchunk(uint32_t c, uint32_t k) {
    return NCOL == 16 ? (c ^ ((k >> 2) & 1u)) : NCOL == 32 ? (c ^ ((k >> 1) & 3u)) : (c ^ (k & 7u));
  }
  // 16-byte chunk c of row k of a tile or query as stored under its swizzle
  __device__ static __forceinline__ uint32_t kchunk(uint32_t c, uint32_t k) {
    return D == 128 ? (c ^ (k & 7u)) : (c ^ ((k >> 1) & 3u));
  }
};

template <int NCOL, int D>
struct Smem {
  uint64_t k_full[kMaxStages], k_empty[kMaxStages], v_full[kMaxStages], v_empty[kMaxStages];
  uint64_t w_full[2], w_empty[2];              // fp16 value tiles
  uint64_t s_full[2], s_free[2], p_full[2], p_free[2], o_free[2], drain[2];
  // (q_full goes by descriptors, so that its next phase needs every reader's release of the unit: with one barrier a
  // unit of few tiles let the query's next phase end too before a softmax warp had looked, and that warp waited on)
  uint64_t unit_full[2], unit_empty[2], q_full[2], q_free;
  uint32_t tmem_base;
  int abort;
  int start_e;                                 // first entry of this CTA's share
  long long start_at;                          // weight before it
  long long sums[Cfg<NCOL, D>::kWarps];
  uint16_t meta[kMeta][kMaxBoxes];             // scale bytes of a tile's boxes: K, V << 8
  alignas(16) float red[4][NCOL];              // maxima and sums of the rows by lane quadrant
  alignas(16) float nref[NCOL];                // references of the rows, negated
  alignas(16) float by[NCOL];                  // what a move of them scales by; at a unit's end 1 / sum (-1: no output)
  Unit<NCOL> unit[Cfg<NCOL, D>::kUnits];
};

template <int NCOL, int D>
constexpr size_t fixed_bytes() {
  using C = Cfg<NCOL, D>;
  return 1024 + C::kBufs * C::kPBytes + C::kQBytes + sizeof(Smem<NCOL, D>);
}

// Ring stages of the K and of the V tiles.
template <int NCOL, int D>
constexpr int stages(bool values) {
  const int all = (int)((Cfg<NCOL, D>::kSmemLimit - fixed_bytes<NCOL, D>()) / Cfg<NCOL, D>::kTile);
  const int n = values ? all - all / 2 : all / 2;             // (a value tile is held longer)
  return n > kMaxStages ? kMaxStages : n;
}

template <int NCOL, int D>
constexpr size_t smem_bytes() {
  return fixed_bytes<NCOL, D>() + (size_t)(stages<NCOL, D>(false) + stages<NCOL, D>(true)) * Cfg<NCOL, D>::kTile;
}

// Instruction descriptors with fp32 accumulation: e4m3 x e4m3, both K-major
// (kind::f8f6f4), and fp16 (TMEM, K-major) x fp16 (MN-major) (kind::f16).
__host__ __device__ constexpr uint32_t idesc_e4m3(int N) {
  return (1u << 4) | ((uint32_t)(N >> 3) << 17) | (8u << 24);
}
__host__ __device__ constexpr uint32_t idesc_fp16_mn(int N) {
  return (1u << 4) | (1u << 16) | ((uint32_t)(N >> 3) << 17) | (8u << 24);
}

// D[tmem] (+)= A[smem] * B[smem] on 8-bit operands
__device__ __forceinline__ void mma_ss_f8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                          uint32_t accumulate) {
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
               "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}"
               :: "r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
               : "memory");
}

// Two transposed 16 x 16 matrices of bytes; lane k gives the address of row k of the 32.  Lane t gets
// bytes 4 (t % 4) .. + 3 of columns t / 4 (r0) and t / 4 + 8 (r1) of the first, r2 and r3 of the second.
__device__ __forceinline__ void ldmatrix_t_b8(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m16n16.x2.trans.shared.b8 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}

// 16 lanes x 32 columns: lane t stores columns 8 k + 2 (t % 4), + 1 of TMEM lanes t / 4 (v[4 k], v[4 k + 1])
// and t / 4 + 8 (v[4 k + 2], v[4 k + 3]).
__device__ __forceinline__ void tmem_st_16x256b_x4(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x256b.x4.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
      "%14, %15, %16};"
      :: "r"(taddr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
         "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}

// v[c] of the 32 lanes joined by op, for every c: lane t returns that of c = t / 2.
template <typename Op>
__device__ __forceinline__ float across_lanes(const float (&v)[16], int lane, Op op) {
  float a[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const bool up = lane & 16;
    a[k] = op(up ? v[k + 8] : v[k], __shfl_xor_sync(0xffffffffu, up ? v[k] : v[k + 8], 16));
  }
#pragma unroll
  for (int half = 4; half > 0; half >>= 1) {
    const bool up = lane & (2 * half);
#pragma unroll
    for (int k = 0; k < half; ++k) {
      const float other = __shfl_xor_sync(0xffffffffu, up ? a[k] : a[k + half], 2 * half);
      a[k] = op(up ? a[k + half] : a[k], other);
    }
  }
  return op(a[0], __shfl_xor_sync(0xffffffffu, a[0], 1));
}

__device__ __forceinline__ uint32_t globaltimer_lo() {
  uint32_t t;
  asm volatile("mov.u32 %0, %%globaltimer_lo;" : "=r"(t));
  return t;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ uint32_t f16x2_of_codes(uint32_t two) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)two));
  return r;
}

__device__ __forceinline__ uint32_t codes_of(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// Tokens of the first `upto` positions that shard r holds (local_len without its 64-bit division).
__device__ __forceinline__ int held_below(int upto, int r, int I, int N) {
  const long long period = (long long)I * N;
  const unsigned full = period > upto ? 0u : (unsigned)upto / (unsigned)period;
  const long long rest = upto - full * period - (long long)r * I;
  return (int)(full * (unsigned)I) + (int)min(max(rest, 0LL), (long long)I);
}

// Queries of request b (0 where its lengths are out of range) and the keys of shard r that they see.
struct Request {
  int S, n, keys;
  bool bad;                                    // lengths out of range, or more keys than the table holds
};

__device__ __forceinline__ Request request_of(const Params& p, int b, int r) {
  Request q;
  q.S = p.seq_lens[b];
  q.n = p.q_lens ? p.q_lens[b] : p.Lq;
  q.bad = q.n < 0 || q.n > p.Lq || q.S < q.n;
  if (q.bad) q.n = 0;
  q.keys = q.n > 0 ? held_below(q.S, r, p.I, p.N) : 0;
  const long long room = (long long)p.max_lb * p.bs;
  if (q.keys > room) q.keys = (int)room, q.bad = true;
  return q;
}

// a / b (a 64-bit division costs several times as much)
__device__ __forceinline__ long long quotient(long long a, unsigned b) {
  return (unsigned long long)a >> 32 ? a / b : (long long)((unsigned)a / b);
}

__device__ __forceinline__ int tiles_of(int keys) { return (int)(((unsigned)keys + kNt - 1) / kNt); }   // (keys up to 2^31 - 1)

// Weight of a unit: its tiles (an empty one still writes its rows), its start and end.
__device__ __forceinline__ int weight_of(const Params& p, int e, int unit_cost) {
  return max(1, tiles_of(request_of(p, e / p.N, e % p.N).keys)) + unit_cost;
}

template <int NCOL, int D>
__global__ void __launch_bounds__(Cfg<NCOL, D>::kThreads, Cfg<NCOL, D>::kCtas)
kv8_gqa_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v, const Params p) {
  using C = Cfg<NCOL, D>;
  constexpr int kWarps = C::kWarps, kSoftWarps = C::kSoftWarps, kBufs = C::kBufs;
  constexpr uint32_t kThreads = C::kThreads, kSoftThreads = C::kSoftThreads;
  constexpr int kKStages = stages<NCOL, D>(false), kVStages = stages<NCOL, D>(true);
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* kring = base;
  uint8_t* vring = kring + kKStages * C::kTile;
  uint8_t* ps = vring + kVStages * C::kTile;
  uint8_t* qs = ps + kBufs * C::kPBytes;
  Smem<NCOL, D>& sm = *reinterpret_cast<Smem<NCOL, D>*>(qs + C::kQBytes);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  volatile int* abort_flag = &sm.abort;
  if (tid == 0) {
    for (int k = 0; k < kMaxStages; ++k) {
      mbar_init(smem_u32(&sm.k_full[k]), 1);
      mbar_init(smem_u32(&sm.k_empty[k]), 1);
      mbar_init(smem_u32(&sm.v_full[k]), 1);
      mbar_init(smem_u32(&sm.v_empty[k]), kConvWarps);
    }
    for (int k = 0; k < 2; ++k) {
      mbar_init(smem_u32(&sm.w_full[k]), kConvWarps);
      mbar_init(smem_u32(&sm.w_empty[k]), 1);
      mbar_init(smem_u32(&sm.s_full[k]), 1);
      mbar_init(smem_u32(&sm.s_free[k]), kSoftWarps);
      mbar_init(smem_u32(&sm.p_full[k]), kSoftWarps);
      mbar_init(smem_u32(&sm.p_free[k]), 1);
      mbar_init(smem_u32(&sm.o_free[k]), kSoftWarps);
      mbar_init(smem_u32(&sm.drain[k]), 1);
    }
    for (int k = 0; k < C::kUnits; ++k) {
      mbar_init(smem_u32(&sm.unit_full[k]), 1);
      mbar_init(smem_u32(&sm.unit_empty[k]), C::kReleases);
      mbar_init(smem_u32(&sm.q_full[k]), kConvWarps);
    }
    mbar_init(smem_u32(&sm.q_free), 1);
    sm.abort = 0;
    sm.start_e = -1;
    fence_mbar_init();
    prefetch_tmap(&tm_k);
    prefetch_tmap(&tm_v);
  }
  if (warp == 1) tmem_alloc(smem_u32(&sm.tmem_base), C::kTmemCols);

  // this CTA's share of the summed weight: entries (request, shard) in order, a run of them per thread
  const int entries = p.B * p.N, per = (entries + (int)kThreads - 1) / (int)kThreads;
  const long long units_per = (long long)p.Hkv * p.m_tiles;
  long long mine = 0;
#pragma unroll 1
  for (int k = 0; k < per; ++k)
    if (tid * (long long)per + k < entries) mine += weight_of(p, tid * per + k, C::kUnitCost);
  mine *= units_per;
  long long upto = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long v = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += v;
  }
  if (lane == 31) sm.sums[warp] = upto;
  __syncthreads();
  long long total = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w == warp) upto += total;
    total += sm.sums[w];
  }
  // (no share is empty, so the parts of a cut unit are neighbours; CTAs past the summed weight have none)
  const long long ctas = min((long long)gridDim.x, total);
  const long long each = quotient(total, (unsigned)ctas), over = total - each * ctas;    // (the first `over` take one more)
  const long long c = min((long long)blockIdx.x, ctas), lo = each * c + min(c, over);
  const long long hi = blockIdx.x < ctas ? lo + each + (c < over ? 1 : 0) : lo;
  if (upto - mine <= lo && lo < upto) {
    long long at = upto - mine;
    int e = tid * per;
#pragma unroll 1
    for (;; ++e) {
      const long long next = at + weight_of(p, e, C::kUnitCost) * units_per;
      if (lo < next) break;
      at = next;
    }
    sm.start_e = e;
    sm.start_at = at;
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem_base;
  if (tid == 0) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  auto fail = [&](void) {
    set_status(p.status, DCP_ERR_TIMEOUT);
    *abort_flag = 1;
  };
  // A whole warp waits for the phase of `parity`; false: it did not come within `limits` times the limit (or,
  // with `heeds`, the CTA has given up).  Compact on purpose: every role's code shares the instruction cache.
  auto wait_at = [&](uint32_t bar, uint32_t parity, bool heeds, int limits) -> bool {
    uint32_t start = 0;
    bool first = true;
#pragma unroll 1
    while (!__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) {
      const uint32_t now = globaltimer_lo();
      if (first) start = now, first = false;
      bool stop = heeds && *abort_flag != 0;
      if (now - start > p.wait_ns) start = now, stop |= --limits == 0;
      if (__any_sync(0xffffffffu, stop)) return false;
    }
    return true;
  };
  auto wait = [&](uint64_t& bar, uint32_t parity) -> bool { return wait_at(smem_u32(&bar), parity, true, 1); };
  // the next unit's descriptor (a whole warp); false: there are no more, or the wait ran out
  auto unit_wait = [&](int u, int limits = 4) -> bool {
    const int slot = u % C::kUnits;
    if (!wait_at(smem_u32(&sm.unit_full[slot]), (uint32_t)(u / C::kUnits) & 1u, false, limits)) {
      fail();
      return false;
    }
    return sm.unit[slot].tiles >= 0;
  };
  auto unit_done = [&](int u) {
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&sm.unit_empty[u % C::kUnits]));
  };

  if (warp < kConvWarp) {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" :: "n"(C::kCtrlRegs));
  if (warp == 3) {
    // ---------------- scheduler ----------------
    if (lane == 0) p.cut[2 * blockIdx.x] = p.cut[2 * blockIdx.x + 1] = -1;
    auto slot_free = [&](int u) -> bool {
      if (u < C::kUnits ||
          wait_at(smem_u32(&sm.unit_empty[u % C::kUnits]), (uint32_t)(u / C::kUnits - 1) & 1u, false, 4))
        return true;
      fail();
      return false;
    };
    int e = sm.start_e, u = 0;
    long long at = sm.start_at;
    bool ok = true;
    if (e >= 0) {
#pragma unroll 1
      for (; ok && e < entries && at < hi; ++e) {
        const int b = e / p.N, r = e % p.N;
        const Request q = request_of(p, b, r);
        const int tiles = tiles_of(q.keys), weight = max(1, tiles) + C::kUnitCost;
        const int32_t* bt = p.block_tables + ((long long)r * p.B + b) * p.max_lb;
        // a block id past the pool among the keys empties the request in this shard
        bool bad_block = false;
        const int blocks = (int)(((unsigned)q.keys + (unsigned)p.bs - 1) / (unsigned)p.bs);
#pragma unroll 1
        for (int k = lane; k < blocks; k += 32 * 8) {
          int blk[8];
#pragma unroll
          for (int m = 0; m < 8; ++m) blk[m] = k + 32 * m < blocks ? bt[k + 32 * m] : 0;
#pragma unroll
          for (int m = 0; m < 8; ++m) bad_block |= (unsigned)blk[m] >= (unsigned)p.num_blocks;
        }
        bad_block = __any_sync(0xffffffffu, bad_block);
        if (lane == 0 && (q.bad || bad_block)) set_status(p.status, DCP_ERR_BOUNDS);
        long long k0 = at < lo ? quotient(lo - at, (unsigned)weight) : 0;      // first unit of the entry in this share
#pragma unroll 1
        for (; k0 < units_per; ++k0) {
          const long long first = at + k0 * weight;
          if (first >= hi) break;
          const int g = (int)((unsigned)k0 / (unsigned)p.m_tiles), mt = (int)k0 - g * p.m_tiles;
          const int row0 = mt * NCOL, rows = min(NCOL, p.Lq * p.gsize - row0);
          const int live = bad_block || row0 / p.gsize >= q.n ? 0 : tiles;      // tiles that count
          const int t0 = (int)min(max(lo - first, 0LL), (long long)live), t1 = (int)min(hi - first, (long long)live);
          if (live > 0 ? t1 <= t0 : first < lo) continue;     // (another CTA's)
          const int slot = u % C::kUnits;
          ok = slot_free(u);
          if (!ok) break;
          Unit<NCOL>& w = sm.unit[slot];
          if (lane == 0) {
            const int slot_at = live == 0 || (t0 == 0 && t1 == live) ? -1 : 2 * (int)blockIdx.x + (t0 > 0 ? 0 : 1);
            w.b = b, w.r = r, w.g = g, w.row0 = row0, w.rows = rows;
            w.n = q.n, w.first = q.S - q.n, w.keys = q.keys;
            w.t0 = t0, w.tiles = t1 - t0;
            w.ke = live == 0 ? 0 : min(q.keys, held_below(w.first + min(q.n, (row0 + rows - 1) / p.gsize + 1), r, p.I, p.N));
            w.lim_min = live == 0 ? 0 : min(w.ke, held_below(w.first + row0 / p.gsize + 1, r, p.I, p.N));
            w.slot = slot_at;
            w.nan_values = 0;
            if (slot_at >= 0) p.cut[slot_at] = (long long)e * units_per + k0;
            mbar_arrive(smem_u32(&sm.unit_full[slot]));
          }
          __syncwarp();
          ++u;
        }
        at += weight * units_per;
      }
    }
    const int slot = u % C::kUnits;
    if (ok && slot_free(u) && lane == 0) {
      sm.unit[slot].tiles = -1;
      mbar_arrive(smem_u32(&sm.unit_full[slot]));
    }
  } else if (warp == 0) {
    // ---------------- TMA producer ----------------
    const int box = 1 << p.box_shift, boxes = kNt >> p.box_shift, window = 32 >> (7 - p.box_shift);   // tiles of a window
    int kst = 0, vst = 0, tt = 0;
    uint32_t kph = 1, vph = 1;
    int k_issued = 0, v_issued = 0;
#pragma unroll 1
    for (int u = 0; unit_wait(u); ++u) {
      const Unit<NCOL>& w = sm.unit[u % C::kUnits];
      const int tiles = *abort_flag ? 0 : w.tiles, t0 = w.t0, ke = w.ke, g = w.g;
      const int32_t* bt = p.block_tables + ((long long)w.r * p.B + w.b) * p.max_lb;
      // A lane's box of a window of tiles: pool block and scale bytes.  The next window's bytes and the table
      // entries of the one behind it are on their way meanwhile.
      auto entry = [&](int t) {
        const unsigned j = (unsigned)(t0 + t) * kNt + (unsigned)(lane * box);      // (may pass 2^31 behind the last tile)
        return t < tiles && j < (unsigned)ke ? bt[j / (unsigned)p.bs] : -1;
      };
      auto scale_bytes = [&](int blk) {
        if (blk < 0) return 127u | 127u << 8;
        const uint8_t* s = p.scales + (long long)blk * p.Hkv + g;
        return (uint32_t)s[0] | (uint32_t)s[(long long)p.num_blocks * p.Hkv] << 8;
      };
      int blk = entry(0), blk1 = entry(window), blk2 = entry(2 * window);
      uint32_t sc = scale_bytes(blk), sc1 = scale_bytes(blk1);
#pragma unroll 1
      for (int t = 0; t < tiles; ++t) {
        const int in = t & (window - 1);
        if (in == 0 && t > 0) {
          blk = blk1, sc = sc1;
          blk1 = blk2, sc1 = scale_bytes(blk1);
          blk2 = entry(t + 2 * window);
        }
        if (!wait(sm.k_empty[kst], kph)) {
          fail();
          break;
        }
        const int k = lane - in * boxes;                      // this lane's box of the tile
        const bool has = k >= 0 && k < boxes;
        const int row = has && blk >= 0 ? blk * p.bs + ((t0 + t) * kNt + k * box) % p.bs : 0;
        const bool loads = t0 + t != p.skip_tile;             // (test hook: a tile that is never loaded)
        if (has && loads) tma_load_3d(smem_u32(kring + kst * C::kTile + k * box * D), &tm_k, 0, g, row, smem_u32(&sm.k_full[kst]));
        // the scale bytes arrive behind the copies' start; the barrier's one arrival follows both
        if (has) sm.meta[tt & (kMeta - 1)][k] = (uint16_t)sc;
        __syncwarp();
        if (loads) {
          if (lane == 0) mbar_arrive_expect_tx(smem_u32(&sm.k_full[kst]), C::kTile);
          ++k_issued;
          if (++kst == kKStages) kst = 0, kph ^= 1;
          if (!wait(sm.v_empty[vst], vph)) {
            fail();
            break;
          }
          if (lane == 0) mbar_arrive_expect_tx(smem_u32(&sm.v_full[vst]), C::kTile);
          __syncwarp();
          if (has) tma_load_3d(smem_u32(vring + vst * C::kTile + k * box * D), &tm_v, 0, g, row, smem_u32(&sm.v_full[vst]));
          ++v_issued;
          if (++vst == kVStages) vst = 0, vph ^= 1;
        }
        ++tt;
      }
      unit_done(u);
    }
    // Copies in flight land before the CTA leaves.  (They have, where it did not give up; another role may do that behind
    // the last copy, and the CTA leaves then without having waited for it elsewhere.)
#pragma unroll 1
    for (int k = max(0, k_issued - kKStages); k < k_issued; ++k)
      wait_at(smem_u32(&sm.k_full[k % kKStages]), (uint32_t)(k / kKStages) & 1u, false, 1);
#pragma unroll 1
    for (int k = max(0, v_issued - kVStages); k < v_issued; ++k)
      wait_at(smem_u32(&sm.v_full[k % kVStages]), (uint32_t)(k / kVStages) & 1u, false, 1);
  } else if (warp == 1) {
    // ---------------- QK issuer: S^T(t) = K(t) (Q_hi + Q_lo)^T ----------------
    constexpr uint32_t id = idesc_e4m3(NCOL);
    const bool lead = elect_one();
    const uint32_t tm = uniform(tmem), ring = uniform(smem_u32(kring)), qaddr = uniform(smem_u32(qs));
    int st = 0, tt = 0;
    uint32_t ph = 0;
#pragma unroll 1
    for (int u = 0; unit_wait(u); ++u) {
      const int slot = u % C::kUnits;
      const int tiles = (int)uniform((uint32_t)sm.unit[slot].tiles);
      // (waited for in units without tiles too: a phase left out would make the next wait pass early)
      bool good = wait(sm.q_full[u % C::kUnits], (uint32_t)(u / C::kUnits) & 1u);
      if (tiles > 0 && *abort_flag == 0) {
#pragma unroll 1
        for (int t = 0; good && t < tiles; ++t, ++tt) {
          good = wait(sm.k_full[st], ph) && (tt < 2 || wait(sm.s_free[tt & 1], (uint32_t)((tt >> 1) - 1) & 1u));
          if (!good) break;
          if (lead) {
            tc_fence_after();
            const uint32_t kt = ring + st * C::kTile, qt = qaddr;
#pragma unroll
            for (int term = 0; term < 2; ++term)
#pragma unroll
              for (int k = 0; k < D / 32; ++k)
                mma_ss_f8(tm + (uint32_t)(tt & 1) * NCOL, smem_desc(kt + k * 32, 16, 8 * D, C::kKSwz),
                          smem_desc(qt + term * NCOL * D + k * 32, 16, 8 * D, C::kKSwz), id, term + k > 0 ? 1u : 0u);
            mma_commit(smem_u32(&sm.k_empty[st]));
            mma_commit(smem_u32(&sm.s_full[tt & 1]));
          }
          __syncwarp();
          if (++st == kKStages) st = 0, ph ^= 1;
        }
        if (!good) fail();
      }
      if (lead) mma_commit(smem_u32(&sm.q_free));             // (once per unit: its parity goes by them)
      unit_done(u);
    }
    if (lead) mma_commit(smem_u32(&sm.drain[0]));
    __syncwarp();
    if (!wait_at(smem_u32(&sm.drain[0]), 0, false, 1)) fail();
  } else if (warp == 2) {
    // ---------------- PV issuer: O^T += V16^T(t) P^T(t) ----------------
    constexpr uint32_t id = idesc_fp16_mn(NCOL);
    const bool lead = elect_one();
    const uint32_t tm = uniform(tmem), paddr = uniform(smem_u32(ps));
    int tt = 0, o_units = 0;
#pragma unroll 1
    for (int u = 0; unit_wait(u); ++u) {
      const int tiles = (int)uniform((uint32_t)sm.unit[u % C::kUnits].tiles);
      if (tiles > 0 && *abort_flag == 0) {
        bool good = o_units < 2 || wait(sm.o_free[o_units & 1], (uint32_t)((o_units >> 1) - 1) & 1u);
        const uint32_t dO = tm + 2 * NCOL + (uint32_t)(o_units & 1) * NCOL;
#pragma unroll 1
        for (int t = 0; good && t < tiles; ++t, ++tt) {
          const uint32_t buf = tt % kBufs;
          good = wait(sm.w_full[tt % C::kWBufs], (uint32_t)(tt / C::kWBufs) & 1u) && wait(sm.p_full[buf], (uint32_t)(tt / kBufs) & 1u);
          if (!good) break;
          if (lead) {
            tc_fence_after();
            const uint32_t vt = tm + 4 * NCOL + (uint32_t)(tt % C::kWBufs) * kWCols, pt = paddr + buf * C::kPBytes;
#pragma unroll
            for (int k = 0; k < kNt / 16; ++k)
              mma_ts(dO, vt + k * 8,
                     smem_desc(pt + k * 16 * C::kPitch, C::kPBytes, 8 * C::kPitch, C::kPSwz), id, t + k > 0 ? 1u : 0u);
            mma_commit(smem_u32(&sm.w_empty[tt % C::kWBufs]));
            mma_commit(smem_u32(&sm.p_free[buf]));
          }
          __syncwarp();
        }
        if (!good) fail();
        ++o_units;
      }
      unit_done(u);
    }
    if (lead) mma_commit(smem_u32(&sm.drain[1]));
    __syncwarp();
    if (!wait_at(smem_u32(&sm.drain[1]), 0, false, 1)) fail();
  }
  } else if (warp < kSoftWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" :: "n"(C::kConvRegs));
    // ---------------- query split, then value tiles to fp16 ----------------
    const int ct = tid - 32 * kConvWarp, dim0 = 32 * (warp - kConvWarp);
    int st = 0, tt = 0;
    uint32_t ph = 0;
#pragma unroll 1
    for (int u = 0; unit_wait(u); ++u) {
      const int slot = u % C::kUnits;
      Unit<NCOL>& w = sm.unit[slot];
      const int tiles = w.tiles, t0 = w.t0, ke = w.ke, lim_min = w.lim_min;
      // the last unit's scores are done with the query's buffer
      if (u > 0 && !wait(sm.q_free, (uint32_t)(u - 1) & 1u)) fail();
      {
        // query rows: D / 8 lanes a row; the row's largest magnitude goes to [128, 256), hi = e4m3(q),
        // lo = e4m3(q - hi); a value that is not finite makes its row NaN
        constexpr int kLanes = D / 8, kRowsAt = 128 / kLanes;
        const int c8 = ct % kLanes;
        uint8_t* qd = qs;
#pragma unroll 1
        for (int h = ct / kLanes; h < NCOL; h += kRowsAt) {
          uint4 raw = make_uint4(0, 0, 0, 0);
          const int i = (w.row0 + h) / p.gsize, head = w.g * p.gsize + (w.row0 + h) - i * p.gsize;
          const bool there = h < w.rows && i < w.n;
          const long long row = ((long long)w.b * p.Lq + i) * p.Hq + head;
          if (there) raw = __ldg(reinterpret_cast<const uint4*>(p.q + row * D) + c8);
          if (c8 == 0) {
            w.lim[h] = there && tiles > 0 ? min(w.keys, held_below(w.first + i + 1, w.r, p.I, p.N)) : 0;
            w.at[h] = w.slot >= 0 ? (long long)w.slot * NCOL + h : (long long)w.r * p.B * p.Lq * p.Hq + row;
          }
            const uint32_t words[4] = {raw.x, raw.y, raw.z, raw.w};
            float x[8], most = 0.f;
#pragma unroll
            for (int k = 0; k < 4; ++k) x[2 * k] = bf16_lo(words[k]), x[2 * k + 1] = bf16_hi(words[k]);
#pragma unroll
            for (int k = 0; k < 8; ++k) most = fmaxf(most, fabsf(x[k]));
#pragma unroll
            for (int o = kLanes / 2; o > 0; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
            // 2^e <= most < 2^(e + 1): the row times 2^(7 - e), in two steps (either may leave fp32's exponents)
            const int e = max((int)(__float_as_uint(most) >> 23) - 127, -126);
            const int by = 7 - e, by1 = by / 2, by2 = by - by1;
            const float f1 = __uint_as_float((uint32_t)(127 + by1) << 23), f2 = __uint_as_float((uint32_t)(127 + by2) << 23);
            uint32_t hi[2], lo2[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              uint32_t h16[2], l16[2];
#pragma unroll
              for (int m2 = 0; m2 < 2; ++m2) {
                float v[2], rest[2];
#pragma unroll
                for (int z = 0; z < 2; ++z) {
                  v[z] = x[4 * k + 2 * m2 + z] * f1 * f2;
                  if (!(fabsf(v[z]) <= 448.f)) v[z] = NAN;
                }
                h16[m2] = codes_of(v[0], v[1]);
                const uint32_t back = f16x2_of_codes(h16[m2]);
                const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&back));
                rest[0] = v[0] - f.x, rest[1] = v[1] - f.y;
                l16[m2] = codes_of(rest[0], rest[1]);
              }
              hi[k] = h16[0] | h16[1] << 16;
              lo2[k] = l16[0] | l16[1] << 16;
            }
            const uint32_t off = h * D + (C::kchunk((uint32_t)(c8 >> 1), (uint32_t)h) << 4) + (c8 & 1) * 8;
            *reinterpret_cast<uint2*>(qd + off) = make_uint2(hi[0], hi[1]);
            *reinterpret_cast<uint2*>(qd + NCOL * D + off) = make_uint2(lo2[0], lo2[1]);
            if (c8 == 0) w.qf[h] = __uint_as_float((uint32_t)max(127 - by, 1) << 23);
        }
        fence_proxy_async_smem();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&sm.q_full[slot]));   // (once per unit: its parity goes by them)
      if (tiles > 0 && *abort_flag == 0) {
        bool good = true;
#pragma unroll 1
        for (int t = 0; t < tiles; ++t, ++tt) {
          const int j0 = (t0 + t) * kNt;
          const bool edge = j0 > lim_min - kNt;               // keys that some row does not see
          good = wait(sm.v_full[st], ph) && (tt < C::kWBufs || wait(sm.w_empty[tt % C::kWBufs], (uint32_t)(tt / C::kWBufs - 1) & 1u));
          if (!good) break;
          if (edge && dim0 < D) {
            // This warp's dims of a key past the range become 0; of a key that some row does not see, NaN becomes 0
            // here and the epilogue puts it into the rows that see it.  (The warps do not meet here: one that gives up
            // would leave the others waiting.)
#pragma unroll 1
            for (int key = lane; key < kNt; key += 32) {
              const int j = j0 + key;
              if (j < lim_min) continue;
#pragma unroll
              for (int half = 0; half < 2; ++half) {
                uint4* at = reinterpret_cast<uint4*>(vring + st * C::kTile + key * D +
                                                     (C::kchunk((uint32_t)(dim0 / 16 + half), (uint32_t)key) << 4));
                uint4 v = *at;
                uint32_t* words = &v.x;
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                  const uint32_t nan = (((words[m] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) >> 7;
                  if (nan != 0 && j < ke) w.nan_values = 1;
                  words[m] = j < ke ? words[m] & ~(nan * 0xffu) : 0u;
                }
                *at = v;
              }
            }
            fence_proxy_async_smem();                         // (the stage's next tile comes by a copy)
            __syncwarp();
          }
          // this warp's 32 dims: the tile's bytes transposed on the way out of shared memory (16 keys x 16
          // dims a matrix: a lane gets 4 keys of dim lane / 4), fp16, to TMEM lane = dim, column = key / 2
          if (dim0 < D) {
            tc_fence_after();
            const uint32_t src = smem_u32(vring + st * C::kTile) + lane * D;
            const uint32_t dst = tmem + ((uint32_t)dim0 << 16) + 4 * NCOL + (uint32_t)(tt % C::kWBufs) * kWCols;
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              uint32_t r[4][4];
#pragma unroll
              for (int m = 0; m < 4; ++m)                     // 32 keys each
                ldmatrix_t_b8(src + m * 32 * D + (C::kchunk((uint32_t)(dim0 / 16 + half), (uint32_t)lane) << 4), r[m]);
#pragma unroll
              for (int m = 0; m < 4; m += 2) {
                uint32_t o[16];
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                  o[2 * q] = f16x2_of_codes(r[m + (q >> 2)][q & 3]);
                  o[2 * q + 1] = f16x2_of_codes(r[m + (q >> 2)][q & 3] >> 16);
                }
                tmem_st_16x256b_x4(dst + ((uint32_t)(half * 16) << 16) + m * 16, o);
              }
            }
            tmem_wait_st();
            tc_fence_before();
          }
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(smem_u32(&sm.v_empty[st]));
            mbar_arrive(smem_u32(&sm.w_full[tt % C::kWBufs]));
          }
          if (++st == kVStages) st = 0, ph ^= 1;
        }
        if (!good) fail();
      }
      unit_done(u);
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" :: "n"(C::kSoftRegs));
    // ---------------- softmax and epilogue ----------------
    constexpr int HC = 16;                                    // columns (query rows) of a thread
    const int qd = warp & 3;                                  // TMEM lane quadrant
    const int h0 = ((warp - kSoftWarp) >> 2) * HC;
    const int lrow = qd * 32 + lane;                          // key of the tile; value dim of O^T
    const uint32_t lane_base = tmem + ((uint32_t)(qd * 32) << 16);
    const int st = tid - 32 * kSoftWarp;                      // thread st looks after row st where one has to
    int tt = 0, o_units = 0;
    bool dead = false;                                        // a wait ran out: the same in every softmax thread
    // (they meet at barriers, so none may give up alone on a unit that comes late: the scheduler has
    // given up on its own wait long before this limit)
#pragma unroll 1
    for (int u = 0; unit_wait(u, 16); ++u) {
      const Unit<NCOL>& w = sm.unit[u % C::kUnits];
      const int tiles = w.tiles, t0 = w.t0, lim_min = w.lim_min;
      float nm[HC], l[HC];                                    // -R and the sum of a row
      const uint32_t tO = lane_base + 2 * NCOL + (uint32_t)(o_units & 1) * NCOL + h0;
      // The split warps write where the unit's rows go, in a CTA that has given up too: this wait does not heed that,
      // and without what it waits for nothing is written.
      const bool placed = wait_at(smem_u32(&sm.q_full[u % C::kUnits]), (uint32_t)(u / C::kUnits) & 1u, false, 16);
      bool bad = !placed, broke = dead || tiles == 0;
      if (st < NCOL) sm.nref[st] = kNoRef;
#pragma unroll
      for (int h = 0; h < HC; ++h) nm[h] = kNoRef, l[h] = 0.f;
#pragma unroll 1
      for (int t = 0; !broke && t < tiles; ++t, ++tt) {
        const uint32_t buf = tt & 1;
        bad |= !wait(sm.s_full[buf], (uint32_t)(tt >> 1) & 1u);           // (whatever is read then is not used)
        uint32_t v[HC];
        tc_fence_after();
        tmem_ld16(lane_base + buf * NCOL + h0, v);
        tmem_wait_ld();
        const uint32_t meta = sm.meta[tt & (kMeta - 1)][lrow >> p.box_shift];
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sm.s_free[buf]));
        const float kf = scale_factor(meta & 255u) * p.scale_log2;
        const int sv = (int)(meta >> 8);
        const float ev = sv == 255 ? NAN : (float)(sv - 127), inv = scale_factor((uint32_t)max(254 - sv, 0));

        // y = x + ev of this key's rows; hidden keys -inf.  (The query's factor times the product first: it is a power
        // of two, and no product of two factors leaves fp32's range on the way to a score that does not.)
        const int j = (t0 + t) * kNt + lrow;
        const bool full = (t0 + t) * kNt <= lim_min - kNt;
        float y[HC], most = -INFINITY;
#pragma unroll
        for (int h = 0; h < HC; h += 4) {
          const float4 qf = *reinterpret_cast<const float4*>(&w.qf[h0 + h]);
          y[h] = fmaf(__uint_as_float(v[h]) * qf.x, kf, ev);
          y[h + 1] = fmaf(__uint_as_float(v[h + 1]) * qf.y, kf, ev);
          y[h + 2] = fmaf(__uint_as_float(v[h + 2]) * qf.z, kf, ev);
          y[h + 3] = fmaf(__uint_as_float(v[h + 3]) * qf.w, kf, ev);
        }
        if (!full)
#pragma unroll
          for (int h = 0; h < HC; ++h) y[h] = j < w.lim[h0 + h] ? y[h] : -INFINITY;
#pragma unroll
        for (int h = 0; h < HC; ++h) most = fmaxf(most, y[h] + nm[h]);
        // one barrier per tile: does any row's reference have to move?
        if (bar_red_or(kBarSoftmax, kSoftThreads, most > kTop || bad)) {
          sm.red[qd][h0 + (lane >> 1)] = across_lanes(y, lane, [](float a, float b) { return fmaxf(a, b); });
          // O^T is rescaled: the previous tile's product must have landed
          if (t > 0) bad |= !wait(sm.p_free[(tt - 1) % kBufs], (uint32_t)((tt - 1) / kBufs) & 1u);
          if (bar_red_or(kBarSoftmax, kSoftThreads, bad)) {
            broke = dead = true;
            break;
          }
          if (st < NCOL) {
            const float top = fmaxf(fmaxf(sm.red[0][st], sm.red[1][st]), fmaxf(sm.red[2][st], sm.red[3][st]));
            const float was = sm.nref[st], is = fminf(was, kStart - top);
            sm.nref[st] = is;
            sm.by[st] = was == kNoRef ? 0.f : ex2(is - was);
          }
          named_bar_sync(kBarSoftmax, kSoftThreads);
#pragma unroll
          for (int h = 0; h < HC; ++h) {
            nm[h] = sm.nref[h0 + h];
            l[h] *= sm.by[h0 + h];
          }
          if (t > 0) {
            tc_fence_after();
            uint32_t o[HC];
            tmem_ld16(tO, o);
            tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < HC; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * sm.by[h0 + k]);
            tmem_st16(tO, o);
            tmem_wait_st();
          }
        }
        // (a hidden key's y is -inf, its P 0)
        uint32_t pk[HC / 2];
#pragma unroll
        for (int h = 0; h < HC; h += 2) {
          const float p0 = ex2(y[h] + nm[h]), p1 = ex2(y[h + 1] + nm[h + 1]);
          l[h] = fmaf(p0, inv, l[h]);
          l[h + 1] = fmaf(p1, inv, l[h + 1]);
          pk[h / 2] = pack_f16x2(p0, p1);
        }
        if (tt >= kBufs) bad |= !wait(sm.p_free[tt % kBufs], (uint32_t)(tt / kBufs - 1) & 1u);
        uint8_t* prow = ps + (tt % kBufs) * C::kPBytes + lrow * C::kPitch;
#pragma unroll
        for (int c = 0; c < HC / 8; ++c)
          *reinterpret_cast<uint4*>(prow + (C::pchunk((uint32_t)(h0 / 8 + c), (uint32_t)lrow) << 4)) =
              make_uint4(pk[4 * c], pk[4 * c + 1], pk[4 * c + 2], pk[4 * c + 3]);
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sm.p_full[tt % kBufs]));
      }

      // the last product, row sums over the 128 key threads, outputs
      bool have = !broke;
      if (have) bad |= !wait(sm.p_free[(tt - 1) % kBufs], (uint32_t)((tt - 1) / kBufs) & 1u);
      sm.red[qd][h0 + (lane >> 1)] = across_lanes(l, lane, [](float a, float b) { return a + b; });
      if (bar_red_or(kBarSoftmax, kSoftThreads, bad)) have = false, dead = true;
      if (bad) fail();
      if (st < w.rows) {
        const float sum = (sm.red[0][st] + sm.red[1][st]) + (sm.red[2][st] + sm.red[3][st]);
        const bool live = have && w.lim[st] > 0 && !(sum == 0.f);         // (NaN sums make NaN rows)
        sm.by[st] = live ? 1.f / sum : -1.f;
        if (placed)
          (w.slot >= 0 ? p.ws_lse : p.lse)[w.at[st]] = live ? (log2f(sum) - sm.nref[st]) * 0.69314718055994531f : -INFINITY;
      }
      uint32_t o[HC];                                         // (without a product whatever is there: not used)
      tc_fence_after();
      tmem_ld16(tO, o);
      tmem_wait_ld();
      tc_fence_before();
      __syncwarp();
      if (tiles > 0) {
        if (lane == 0) mbar_arrive(smem_u32(&sm.o_free[o_units & 1]));
        ++o_units;
      }
      named_bar_sync(kBarSoftmax, kSoftThreads);
      if (have && *(volatile const int*)&w.nan_values && lrow < D) {
        // NaN values among the keys that some row does not see: into the rows that see them
        const int32_t* bt = p.block_tables + ((long long)w.r * p.B + w.b) * p.max_lb;
#pragma unroll 1
        for (int j = max(lim_min, t0 * kNt); (unsigned)j < min((unsigned)w.ke, (unsigned)(t0 + tiles) * kNt); ++j) {
          const long long row = (long long)bt[j / p.bs] * p.bs + j % p.bs;
          const bool nan = (p.codes_v[(row * p.Hkv + w.g) * D + lrow] & 0x7f) == 0x7f;
#pragma unroll
          for (int h = 0; h < HC; ++h)
            if (nan && j < w.lim[h0 + h]) o[h] = 0x7fc00000u;
        }
      }
      float* const dst = (w.slot >= 0 ? p.ws_o : p.out) + lrow;
#pragma unroll
      for (int h = 0; h < HC; ++h)
        if (placed && h0 + h < w.rows && lrow < D) {
          const float by = sm.by[h0 + h];
          dst[w.at[h0 + h] * D] = by < 0.f ? 0.f : __uint_as_float(o[h]) * by;
        }
      unit_done(u);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

// Joins the partial rows of the units that borders of the CTAs' shares cut: a unit's first part
// is a CTA's tail slot, the others are the head slots of the CTAs behind it.
//   LSE = log sum exp lse_k,  o = sum exp(lse_k - LSE) o_k
// A warp takes rows in turn: a lane holds the weight of one part (32 at a time), then the parts' rows
// are summed, kAhead of them in flight.  Started while the attention kernel still runs
// (griddepcontrol), it waits for that one's memory here.
template <int NCOL, int D>
__global__ void __launch_bounds__(128) kv8_join_kernel(const Params p, int grid) {
  constexpr int V = D / 32, kAhead = 4;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int c = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long unit = p.cut[2 * c + 1];
  if (unit < 0) return;
  int n = 1;                                                  // parts
  for (bool more = true; more;) {
    const int k = c + n + lane;
    const unsigned same = __ballot_sync(0xffffffffu, k < grid && p.cut[2 * min(k, grid - 1)] == unit);
    more = same == 0xffffffffu;
    n += more ? 32 : __ffs(~same) - 1;
  }
  const unsigned units_per = (unsigned)p.Hkv * (unsigned)p.m_tiles;
  const int e = (int)quotient(unit, units_per), k = (int)(unit - (long long)e * units_per);
  const int b = e / p.N, r = e - b * p.N, g = k / p.m_tiles, row0 = (k - g * p.m_tiles) * NCOL;
  const int rows = min(NCOL, p.Lq * p.gsize - row0);
  auto row_of = [&](int s, int h) { return (long long)(s == 0 ? 2 * c + 1 : 2 * (c + s)) * NCOL + h; };
#pragma unroll 1
  for (int h = warp; h < rows; h += 4) {
    float top = -INFINITY, sum = 0.f, o[V];
#pragma unroll
    for (int v = 0; v < V; ++v) o[v] = 0.f;
    bool nan = false;
#pragma unroll 1
    for (int s0 = 0; s0 < n; s0 += 32) {
      const float lse = s0 + lane < n ? p.ws_lse[row_of(s0 + lane, h)] : -INFINITY;
      nan |= __any_sync(0xffffffffu, lse != lse);
      float is = lse;
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) is = fmaxf(is, __shfl_xor_sync(0xffffffffu, is, off));
      is = fmaxf(is, top);
      if (is == -INFINITY) continue;
      const float by = top == -INFINITY ? 0.f : exp2f((top - is) * 1.4426950408889634f);
      const float weight = lse == -INFINITY ? 0.f : exp2f((lse - is) * 1.4426950408889634f);
      top = is;
      sum *= by;
#pragma unroll
      for (int v = 0; v < V; ++v) o[v] *= by;
#pragma unroll 1
      for (int s = 0; s < min(32, n - s0); s += kAhead) {
        float x[kAhead][V], w[kAhead];
#pragma unroll
        for (int m = 0; m < kAhead; ++m) {
          w[m] = __shfl_sync(0xffffffffu, weight, (s + m) & 31);
          if (s0 + s + m >= n) w[m] = 0.f;
          const float* src = p.ws_o + row_of(min(s0 + s + m, n - 1), h) * D + lane;
#pragma unroll
          for (int v = 0; v < V; ++v) x[m][v] = src[32 * v];
        }
#pragma unroll
        for (int m = 0; m < kAhead; ++m) {
          // (a part without keys holds zeros; what is not finite counts however light its part is, as it does within one)
          sum += w[m];
#pragma unroll
          for (int v = 0; v < V; ++v) {
            const bool light = w[m] == 0.f && !(fabsf(x[m][v]) < INFINITY);
            o[v] = light ? o[v] + x[m][v] : fmaf(w[m], x[m][v], o[v]);
          }
        }
      }
    }
    const int rr = row0 + h, i = rr / p.gsize, head = g * p.gsize + rr - i * p.gsize;
    const long long at = (((long long)r * p.B + b) * p.Lq + i) * p.Hq + head;
    const bool any = top != -INFINITY;
#pragma unroll
    for (int v = 0; v < V; ++v) p.out[at * D + v * 32 + lane] = nan ? NAN : any ? o[v] / sum : 0.f;
    if (lane == 0) p.lse[at] = nan ? NAN : any ? top + logf(sum) : -INFINITY;
  }
}

int ncol_of(const AttnArgs& a) {
  const long long rows = (long long)a.Lq * (a.Hq / a.Hkv);
  return rows <= 16 ? 16 : rows <= 32 ? 32 : kMaxCols;
}

int m_tiles_of(const AttnArgs& a) {
  const int n = ncol_of(a);
  return (int)(((long long)a.Lq * (a.Hq / a.Hkv) + n - 1) / n);
}

// One to three CTAs per SM, fewer where there are not that many tiles.
int grid_of(const AttnArgs& a, int sm_count) {
  const int n = ncol_of(a), ctas = sm_count * (n == 16 ? 3 : n == 32 ? 2 : 1);
  const long long tiles = ((long long)a.max_lb * a.bs + kNt - 1) / kNt;
  const long long units = (long long)a.N * a.B * a.Hkv * m_tiles_of(a);
  return (int)std::min<long long>(ctas, units * std::min<long long>(tiles, ctas));
}

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

template <int NCOL, int D>
cudaError_t launch(const CUtensorMap& tm_k, const CUtensorMap& tm_v, const Params& p, int grid, cudaStream_t stream) {
  constexpr size_t smem = smem_bytes<NCOL, D>();
  static_assert(smem <= Cfg<NCOL, D>::kSmemLimit && stages<NCOL, D>(true) >= 1, "shared memory");
  static_assert(stages<NCOL, D>(false) + 2 <= kMeta, "a tile's scale bytes are read before their slot is used again");
  // the register split assumes the launch count (setmaxnreg.inc would wait for registers that do not exist)
  cudaFuncAttributes fa;
  cudaError_t e = cudaFuncGetAttributes(&fa, kv8_gqa_kernel<NCOL, D>);
  if (e != cudaSuccess) return e;
  if (fa.numRegs != Cfg<NCOL, D>::kLaunchRegs) return cudaErrorInvalidConfiguration;
  e = cudaFuncSetAttribute(kv8_gqa_kernel<NCOL, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  kv8_gqa_kernel<NCOL, D><<<(unsigned)grid, Cfg<NCOL, D>::kThreads, smem, stream>>>(tm_k, tm_v, p);
  e = cudaGetLastError();
  if (e != cudaSuccess || grid == 1) return e;
  // (its start overlaps the attention kernel's end)
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(grid - 1));
  cfg.blockDim = dim3(128);
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kv8_join_kernel<NCOL, D>, p, grid);
}

}  // namespace

bool kv8_gqa_supported(const AttnArgs& a) {
  if (a.kind != DCP_ATTN_GQA || (a.Dqk != 64 && a.Dqk != 128) || a.Dv != a.Dqk) return false;
  if ((long long)a.Lq * (a.Hq / a.Hkv) > (1LL << 20)) return false;
  if (a.bs % 8) return false;
  if (a.bs >= kNt ? (a.bs % kNt) : (kNt % a.bs)) return false;
  return (long long)a.num_blocks * a.bs < (1LL << 31) && (long long)a.N * a.B * a.Hkv * m_tiles_of(a) < (1LL << 31);
}

SplitPlan plan_kv8_gqa(const AttnArgs& a, int sm_count) {
  const int grid = grid_of(a, sm_count);
  SplitPlan plan{};
  plan.n_split = grid > 1 ? 2 : 1;             // (says that a join follows)
  plan.split_tokens = kNt;
  const size_t rows = (size_t)2 * grid * ncol_of(a);
  plan.ws_bytes = align256(2 * (size_t)grid * sizeof(long long)) + align256(rows * a.Dv * sizeof(float)) + rows * sizeof(float);
  return plan;
}

cudaError_t launch_kv8_gqa(const AttnArgs& a) {
  CUtensorMap tm_k, tm_v;
  const uint64_t rows = (uint64_t)a.num_blocks * a.bs;
  const uint64_t dims[3] = {(uint64_t)a.Dqk, (uint64_t)a.Hkv, rows};
  const uint64_t strides[2] = {(uint64_t)a.Dqk, (uint64_t)a.Hkv * a.Dqk};
  const int box_rows = a.bs < kNt ? a.bs : kNt;
  const uint32_t box[3] = {(uint32_t)a.Dqk, 1, (uint32_t)box_rows};
  const uint8_t* k_pool = static_cast<const uint8_t*>(a.kv);
  const uint8_t* v_pool = k_pool + rows * a.Hkv * a.Dqk;
  const CUtensorMapSwizzle swizzle = a.Dqk == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B;
  // a KV head's row is what L2 fetches at a time: the next head's is another unit's
  const CUtensorMapL2promotion fetch = a.Dqk == 128 ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B : CU_TENSOR_MAP_L2_PROMOTION_L2_64B;
  if (!make_tensor_map(&tm_k, CU_TENSOR_MAP_DATA_TYPE_UINT8, k_pool, 3, dims, strides, box, swizzle, fetch) ||
      !make_tensor_map(&tm_v, CU_TENSOR_MAP_DATA_TYPE_UINT8, v_pool, 3, dims, strides, box, swizzle, fetch))
    return cudaErrorInvalidValue;
  const int grid = grid_of(a, device_sm_count()), ncol = ncol_of(a);
  Params p{};
  p.q = static_cast<const __nv_bfloat16*>(a.q);
  p.codes_v = v_pool;
  p.scales = a.kv_scales;
  p.block_tables = a.block_tables, p.seq_lens = a.seq_lens, p.q_lens = a.q_lens;
  p.out = a.partial_out, p.lse = a.lse;
  char* ws = static_cast<char*>(a.workspace);
  p.cut = reinterpret_cast<long long*>(ws);
  ws += align256(2 * (size_t)grid * sizeof(long long));
  p.ws_o = reinterpret_cast<float*>(ws);
  ws += align256((size_t)2 * grid * ncol * a.Dv * sizeof(float));
  p.ws_lse = reinterpret_cast<float*>(ws);
  p.status = a.status;
  p.B = a.B, p.Lq = a.Lq, p.Hq = a.Hq, p.Hkv = a.Hkv, p.N = a.N, p.I = a.I;
  p.max_lb = a.max_lb, p.bs = a.bs, p.num_blocks = a.num_blocks;
  p.m_tiles = m_tiles_of(a), p.gsize = a.Hq / a.Hkv;
  for (p.box_shift = 0; (1 << p.box_shift) < box_rows;) ++p.box_shift;
  p.scale_log2 = a.scale * 1.4426950408889634f;
  p.wait_ns = (uint32_t)std::min<unsigned long long>(test_hooks().wait_ns, 4000000000ull);
  p.skip_tile = test_hooks().skip_tile;
  if (a.Dqk == 64)
    return ncol == 16   ? launch<16, 64>(tm_k, tm_v, p, grid, a.stream)
           : ncol == 32 ? launch<32, 64>(tm_k, tm_v, p, grid, a.stream)
                        : launch<64, 64>(tm_k, tm_v, p, grid, a.stream);
  return ncol == 16   ? launch<16, 128>(tm_k, tm_v, p, grid, a.stream)
         : ncol == 32 ? launch<32, 128>(tm_k, tm_v, p, grid, a.stream)
                      : launch<64, 128>(tm_k, tm_v, p, grid, a.stream);
}

}  // namespace dcp
