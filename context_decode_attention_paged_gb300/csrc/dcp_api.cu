// C-ABI layer of libdcp: argument checks, split planning, kernel selection,
// the per-stream device status words, NVTX ranges.  Every public entry point
// is declared in include/dcp.h.
#include <cuda_runtime.h>
#include <nvtx3/nvToolsExt.h>
#include <stdint.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <map>
#include <mutex>
#include <utility>

#include "dcp_internal.h"

namespace dcp {

namespace {

// One status word per stream: the first device-side error since that
// stream's last read.  Streams get their own word in order of first use;
// once DCP_STATUS_STREAMS - 1 streams of a device have one, further streams
// share the last word.
__device__ int g_status[DCP_STATUS_STREAMS];

constexpr int kMaxDevices = 64;
std::mutex g_status_mu;
int* g_status_base[kMaxDevices] = {nullptr};
std::map<std::pair<int, cudaStream_t>, int> g_status_slot;
int g_status_used[kMaxDevices] = {0};

// Device address of the status word of `stream` on the current device (the
// first use on a device looks up the array's address).
int* status_ptr(cudaStream_t stream) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return nullptr;
  std::lock_guard<std::mutex> lock(g_status_mu);
  if (!g_status_base[dev]) {
    void* p = nullptr;
    if (cudaGetSymbolAddress(&p, g_status) != cudaSuccess || p == nullptr) return nullptr;
    g_status_base[dev] = static_cast<int*>(p);
  }
  const auto key = std::make_pair(dev, stream);
  auto it = g_status_slot.find(key);
  int slot;
  if (it != g_status_slot.end()) {
    slot = it->second;
  } else {
    slot = std::min(g_status_used[dev], DCP_STATUS_STREAMS - 1);
    if (g_status_used[dev] < DCP_STATUS_STREAMS - 1) ++g_status_used[dev];
    g_status_slot.emplace(key, slot);
  }
  return g_status_base[dev] + slot;
}

// NVTX range around a C-ABI call (no cost unless a profiler is attached)
struct NvtxRange {
  explicit NvtxRange(const char* name) { nvtxRangePushA(name); }
  ~NvtxRange() { nvtxRangePop(); }
};

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

dcp_status_t from_cuda(cudaError_t e) { return e == cudaSuccess ? DCP_OK : DCP_ERR_CUDA; }

// Fill AttnArgs from the public arguments; INVALID_ARG / UNSUPPORTED on bad input.
dcp_status_t make_args(const dcp_attn_desc_t* d, int32_t dcp_size, int32_t interleave,
                       float scale, int32_t causal_q_len, AttnArgs* a) {
  if (!d) return DCP_ERR_INVALID_ARG;
  if (d->kind != DCP_ATTN_GQA && d->kind != DCP_ATTN_MLA) return DCP_ERR_INVALID_ARG;
  if (d->batch < 1 || d->q_len < 1 || d->num_q_heads < 1 || d->num_kv_heads < 1 ||
      d->head_dim_qk < 1 || d->head_dim_v < 1 || d->block_size < 1 || d->num_blocks < 1 ||
      d->max_local_blocks < 1)
    return DCP_ERR_INVALID_ARG;
  if (dcp_size < 1 || dcp_size > 32 || interleave < 1) return DCP_ERR_INVALID_ARG;
  if (causal_q_len != d->q_len) return DCP_ERR_INVALID_ARG;
  if (d->num_q_heads % d->num_kv_heads) return DCP_ERR_INVALID_ARG;
  if (d->kind == DCP_ATTN_MLA && (d->num_kv_heads != 1 || d->head_dim_v > d->head_dim_qk))
    return DCP_ERR_INVALID_ARG;
  if (d->kind == DCP_ATTN_GQA && d->head_dim_v != d->head_dim_qk) return DCP_ERR_INVALID_ARG;
  if (d->head_dim_qk % 8 || d->head_dim_v % 4) return DCP_ERR_UNSUPPORTED;
  if (!(scale > 0.f) || scale != scale) return DCP_ERR_INVALID_ARG;
  // element counts must fit the kernels' 64-bit index math and int32 grids
  if ((long long)dcp_size * d->batch > (1LL << 30)) return DCP_ERR_UNSUPPORTED;
  a->kind = d->kind;
  a->B = d->batch;
  a->Lq = d->q_len;
  a->Hq = d->num_q_heads;
  a->Hkv = d->num_kv_heads;
  a->Dqk = d->head_dim_qk;
  a->Dv = d->head_dim_v;
  a->bs = d->block_size;
  a->num_blocks = d->num_blocks;
  a->max_lb = d->max_local_blocks;
  a->N = dcp_size;
  a->I = interleave;
  a->scale = scale;
  return DCP_OK;
}

// The kernel that will run for these arguments, and its split plan.
enum class Impl { kSimt, kMlaTc, kGqaTc, kTreeGqa };

Impl select_impl(const AttnArgs& a) {
  if (a.tree_words > 0 && tree_gqa_supported(a)) return Impl::kTreeGqa;
  if (mla_tc_supported(a)) return Impl::kMlaTc;
  if (a.tree_words == 0 && gqa_tc_supported(a)) return Impl::kGqaTc;
  return Impl::kSimt;
}

SplitPlan plan_for(const AttnArgs& a, Impl impl, int sm_count) {
  switch (impl) {
    case Impl::kMlaTc:
      return plan_attn_mla_tc(a, sm_count);
    case Impl::kGqaTc:
      return plan_attn_gqa_tc(a, sm_count);
    case Impl::kTreeGqa:
      return plan_tree_gqa(a, sm_count);
    case Impl::kSimt:
    default:
      return plan_attn_simt(a, sm_count);
  }
}

// Run the planned kernel of a call whose arguments have been checked.
dcp_status_t launch_impl(const AttnArgs& a, Impl impl, const SplitPlan& plan) {
  switch (impl) {
    case Impl::kMlaTc:
      return from_cuda(launch_attn_mla_tc(a, plan));
    case Impl::kGqaTc:
      return from_cuda(launch_attn_gqa_tc(a, plan));
    case Impl::kTreeGqa:
      return from_cuda(launch_tree_gqa(a, plan));
    case Impl::kSimt:
    default:
      return from_cuda(launch_attn_simt(a, plan));
  }
}

int32_t kind_of(Impl impl) {
  switch (impl) {
    case Impl::kMlaTc: return DCP_KERNEL_MLA_TC;
    case Impl::kGqaTc:
    case Impl::kTreeGqa: return DCP_KERNEL_GQA_TC;
    case Impl::kSimt:
    default: return DCP_KERNEL_SIMT;
  }
}

// Arguments of a drafted-tree call: those of dcp_decode_attn and the node limit.
dcp_status_t make_tree_args(const dcp_attn_desc_t* d, int32_t dcp_size, int32_t interleave, float scale, AttnArgs* a) {
  const dcp_status_t st = make_args(d, dcp_size, interleave, scale, d ? d->q_len : 1, a);
  if (st != DCP_OK) return st;
  if (d->q_len > DCP_TREE_MAX_NODES) return DCP_ERR_UNSUPPORTED;
  a->tree_words = (d->q_len + 31) / 32;
  return DCP_OK;
}

// The cache side of an append or commit call (the checks of dcp_kv_cache_write).
bool cache_desc_ok(const dcp_attn_desc_t* d, int32_t dcp_size, int32_t interleave) {
  if (d->kind != DCP_ATTN_GQA && d->kind != DCP_ATTN_MLA) return false;
  if (d->batch < 1 || d->q_len < 1 || d->num_kv_heads < 1 || d->head_dim_qk < 1 || d->block_size < 1 ||
      d->num_blocks < 1 || d->max_local_blocks < 1 || dcp_size < 1 || interleave < 1)
    return false;
  if (d->kind == DCP_ATTN_MLA && d->num_kv_heads != 1) return false;
  const long long row_bytes = 2LL * d->head_dim_qk * d->num_kv_heads;
  if (d->head_dim_qk % 8 || row_bytes > (1LL << 20)) return false;
  return (long long)d->batch * dcp_size <= (1LL << 31) &&
         (long long)d->batch * dcp_size * d->max_local_blocks <= (1LL << 31) &&
         (long long)d->num_blocks * d->block_size <= (1LL << 31);
}

bool rope_ok(const dcp_rope_desc_t* r) {
  return r && r->rot_dim >= 2 && r->rot_dim % 2 == 0 && r->rot_dim <= DCP_ROPE_MAX_DIM && r->rot_offset >= 0 &&
         (r->layout == DCP_ROPE_HALF || r->layout == DCP_ROPE_INTERLEAVED) && std::isfinite(r->mscale);
}

}  // namespace

namespace {
std::mutex g_hooks_mu;
TestHooks g_hooks = {2000000000ull, -1};
}  // namespace

TestHooks test_hooks() {
  std::lock_guard<std::mutex> lock(g_hooks_mu);
  return g_hooks;
}

int device_sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 148;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 1)
    return 148;
  return n;
}

SplitPlan plan_splits(const AttnArgs& a, int sm_count, int tile_tokens, int units_per_split, int start_tiles,
                      int join_tiles) {
  SplitPlan p;
  // (lengths are 32-bit, whatever the table could hold: a split's first token is too)
  const long long max_local = std::min<long long>((long long)a.max_lb * a.bs, INT32_MAX);
  const long long base_units = (long long)a.N * a.B * units_per_split;
  const long long target = 2LL * sm_count;
  long long n = 1;
  const bool small = base_units < target;
  if ((small || (start_tiles > 0 && base_units < 8 * target)) && max_local > 4LL * tile_tokens) {
    // Split count by a wave model: units run in waves of sm_count CTAs and a
    // unit costs its tiles plus about kUnitStartTiles of start-up and drain (the
    // tree form of the MLA kernel: start_tiles, 12.  At 4 one request of 200,000 tokens
    // and 16 nodes takes 785 us in 7 splits, at 12 729 in 4; of 50,000, 32 nodes of
    // 16 heads 89 and 74; three of 40,000, 5 nodes 188 and 164; ten other shapes
    // differ by less than 2.5%), so pick the count with the fewest
    // waves x (tiles per split + start-up).  (Drafted trees: the largest count
    // within 2% of that instead, to even out requests of unlike lengths, took 4%
    // longer over 90 shapes of 1 to 16 requests: 0.71 to 1.72 of the time.)
    constexpr long long kUnitStartTiles = 4;
    const long long tiles = (max_local + tile_tokens - 1) / tile_tokens;
    const long long n_hi = std::max<long long>(1, std::min<long long>(small ? 32 : 4, max_local / (4LL * tile_tokens)));
    auto cost = [&](long long c) {
      const long long waves = (base_units * c + sm_count - 1) / sm_count;
      const long long extra = small ? std::max<long long>(kUnitStartTiles, start_tiles) : start_tiles + (c > 1 ? join_tiles : 0);
      return waves * ((tiles + c - 1) / c + extra);
    };
    for (long long c = 2; c <= n_hi; ++c)
      if (cost(c) < cost(n)) n = c;
  }
  long long per = (max_local + n - 1) / n;
  per = (per + tile_tokens - 1) / tile_tokens * tile_tokens;
  if (per < tile_tokens) per = tile_tokens;
  n = (max_local + per - 1) / per;
  if (n < 1) n = 1;
  p.lpt_order = false;
  p.order_offset = 0;
  p.n_split = (int)n;
  p.split_tokens = (int)std::min<long long>(per, 1LL << 30);
  p.ws_bytes = 0;
  if (p.n_split > 1) {
    const size_t rows = (size_t)a.N * a.B * a.Lq * a.Hq;
    p.ws_bytes = align256(rows * p.n_split * a.Dv * sizeof(float)) + rows * p.n_split * sizeof(float);
  }
  return p;
}

}  // namespace dcp

using namespace dcp;

extern "C" {

const char* dcp_status_string(dcp_status_t s) {
  switch (s) {
    case DCP_OK: return "DCP_OK";
    case DCP_ERR_INVALID_ARG: return "DCP_ERR_INVALID_ARG";
    case DCP_ERR_UNSUPPORTED: return "DCP_ERR_UNSUPPORTED";
    case DCP_ERR_CUDA: return "DCP_ERR_CUDA";
    case DCP_ERR_TIMEOUT: return "DCP_ERR_TIMEOUT";
    case DCP_ERR_BOUNDS: return "DCP_ERR_BOUNDS";
  }
  return "DCP_ERR_UNKNOWN";
}

dcp_status_t dcp_build_slot_map(const int32_t* seq_lens, int32_t batch, int32_t block_size,
                                int32_t interleave, int32_t dcp_size, int32_t* local_seq_lens,
                                int32_t* local_num_blocks, int32_t* shard_of, int32_t* local_pos,
                                int32_t max_seq, void* stream) {
  NvtxRange range("dcp_build_slot_map");
  if (batch < 0 || block_size < 1 || interleave < 1 || dcp_size < 1) return DCP_ERR_INVALID_ARG;
  if (batch > 0 && (!seq_lens || !local_seq_lens || !local_num_blocks)) return DCP_ERR_INVALID_ARG;
  if ((shard_of == nullptr) != (local_pos == nullptr)) return DCP_ERR_INVALID_ARG;
  if (shard_of && max_seq < 1) return DCP_ERR_INVALID_ARG;
  if ((long long)batch * dcp_size > (1LL << 30)) return DCP_ERR_INVALID_ARG;
  // one thread per (request, token) of the optional maps: the grid must fit
  if (shard_of && (long long)batch * max_seq > (long long)INT_MAX * 256) return DCP_ERR_INVALID_ARG;
  if (batch == 0) return DCP_OK;
  int* st = status_ptr(static_cast<cudaStream_t>(stream));
  if (!st) return DCP_ERR_CUDA;
  return from_cuda(launch_slot_map(seq_lens, batch, block_size, interleave, dcp_size,
                                   local_seq_lens, local_num_blocks, shard_of, local_pos, max_seq,
                                   st, static_cast<cudaStream_t>(stream)));
}

size_t dcp_decode_attn_workspace_size(const dcp_attn_desc_t* d, int32_t dcp_size) {
  AttnArgs a{};
  if (make_args(d, dcp_size, 1, 1.0f, d ? d->q_len : 1, &a) != DCP_OK) return 0;
  return plan_for(a, select_impl(a), device_sm_count()).ws_bytes;
}

dcp_status_t dcp_decode_attn(const dcp_attn_desc_t* d, const void* q, const void* kv_cache,
                             const int32_t* block_tables, const int32_t* seq_lens,
                             int32_t dcp_size, int32_t interleave, float scale,
                             int32_t causal_q_len, float* partial_out, float* lse,
                             void* workspace, size_t workspace_bytes, void* stream) {
  NvtxRange range("dcp_decode_attn");
  AttnArgs a{};
  dcp_status_t st = make_args(d, dcp_size, interleave, scale, causal_q_len, &a);
  if (st != DCP_OK) return st;
  if (!q || !kv_cache || !block_tables || !seq_lens || !partial_out || !lse)
    return DCP_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(kv_cache, 16) || !aligned(partial_out, 16) || !aligned(lse, 4))
    return DCP_ERR_INVALID_ARG;
  const Impl impl = select_impl(a);
  const SplitPlan plan = plan_for(a, impl, device_sm_count());
  if (plan.ws_bytes > 0 &&
      (!workspace || workspace_bytes < plan.ws_bytes || !aligned(workspace, 256)))
    return DCP_ERR_INVALID_ARG;
  a.q = q;
  a.kv = kv_cache;
  a.block_tables = block_tables;
  a.seq_lens = seq_lens;
  a.partial_out = partial_out;
  a.lse = lse;
  a.workspace = workspace;
  a.workspace_bytes = workspace_bytes;
  a.status = status_ptr(static_cast<cudaStream_t>(stream));
  if (!a.status) return DCP_ERR_CUDA;
  a.stream = static_cast<cudaStream_t>(stream);
  return launch_impl(a, impl, plan);
}

dcp_status_t dcp_kv_cache_write(const dcp_attn_desc_t* d, const void* new_k, const void* new_v,
                                void* kv_cache, const int32_t* block_tables, const int32_t* seq_lens,
                                int32_t dcp_size, int32_t interleave, int32_t n_new, void* stream) {
  NvtxRange range("dcp_kv_cache_write");
  if (!d || !new_k || !kv_cache || !block_tables || !seq_lens) return DCP_ERR_INVALID_ARG;
  if (d->kind != DCP_ATTN_GQA && d->kind != DCP_ATTN_MLA) return DCP_ERR_INVALID_ARG;
  const bool gqa = d->kind == DCP_ATTN_GQA;
  if (gqa != (new_v != nullptr)) return DCP_ERR_INVALID_ARG;
  if (d->batch < 1 || d->num_kv_heads < 1 || d->head_dim_qk < 1 || d->block_size < 1 || d->num_blocks < 1 ||
      d->max_local_blocks < 1 || dcp_size < 1 || interleave < 1 || n_new < 1)
    return DCP_ERR_INVALID_ARG;
  if (!gqa && d->num_kv_heads != 1) return DCP_ERR_INVALID_ARG;
  const long long row_bytes = 2LL * d->head_dim_qk * (gqa ? d->num_kv_heads : 1);
  if (row_bytes % 16 || row_bytes > (1LL << 20)) return DCP_ERR_INVALID_ARG;
  if ((long long)d->batch * dcp_size * d->max_local_blocks > (1LL << 31) ||
      (long long)d->num_blocks * d->block_size > (1LL << 31))
    return DCP_ERR_INVALID_ARG;
  if (!aligned(new_k, 16) || !aligned(kv_cache, 16) || (new_v && !aligned(new_v, 16)))
    return DCP_ERR_INVALID_ARG;
  int* st = status_ptr(static_cast<cudaStream_t>(stream));
  if (!st) return DCP_ERR_CUDA;
  return from_cuda(launch_kv_write(new_k, new_v, kv_cache, block_tables, seq_lens, d->batch, n_new, dcp_size,
                                   interleave, d->block_size, d->max_local_blocks, d->num_blocks,
                                   (int)row_bytes, st, static_cast<cudaStream_t>(stream)));
}

dcp_status_t dcp_merge(const float* partial_out, const float* lse, int32_t dcp_size,
                       int32_t batch, int32_t q_len, int32_t num_q_heads, int32_t head_dim_v,
                       void* out, float* out_lse, void* stream) {
  NvtxRange range("dcp_merge");
  if (!partial_out || !lse || !out) return DCP_ERR_INVALID_ARG;
  if (dcp_size < 1 || dcp_size > 32 || batch < 1 || q_len < 1 || num_q_heads < 1 ||
      head_dim_v < 4)
    return DCP_ERR_INVALID_ARG;
  if (num_q_heads % dcp_size || head_dim_v % 4) return DCP_ERR_INVALID_ARG;
  if (!aligned(partial_out, 16) || !aligned(out, 8) || !aligned(lse, 4) ||
      (out_lse && !aligned(out_lse, 4)))
    return DCP_ERR_INVALID_ARG;
  return from_cuda(launch_merge(partial_out, lse, dcp_size, batch, q_len, num_q_heads,
                                head_dim_v, out, out_lse, static_cast<cudaStream_t>(stream)));
}

// Test-only (see TestHooks in dcp_internal.h); not declared in include/dcp.h.
DCP_API void dcp_testing_set_hooks(unsigned long long wait_ns, int32_t skip_tile) {
  std::lock_guard<std::mutex> lock(g_hooks_mu);
  g_hooks.wait_ns = wait_ns > 0 ? wait_ns : 2000000000ull;
  g_hooks.skip_tile = skip_tile;
}

dcp_status_t dcp_get_last_device_status(void* stream) {
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  int* p = status_ptr(s);
  if (!p) return DCP_ERR_CUDA;
  // read and clear the word on the stream itself: later work on the stream
  // sees it cleared; no other stream is waited for
  int v = 0;
  if (cudaMemcpyAsync(&v, p, sizeof(int), cudaMemcpyDeviceToHost, s) != cudaSuccess) return DCP_ERR_CUDA;
  if (cudaMemsetAsync(p, 0, sizeof(int), s) != cudaSuccess) return DCP_ERR_CUDA;
  if (cudaStreamSynchronize(s) != cudaSuccess) return DCP_ERR_CUDA;
  return static_cast<dcp_status_t>(v);
}

int32_t dcp_decode_attn_launches(const dcp_attn_desc_t* d, int32_t dcp_size) {
  AttnArgs a{};
  if (make_args(d, dcp_size, 1, 1.0f, d ? d->q_len : 1, &a) != DCP_OK) return 0;
  const SplitPlan plan = plan_for(a, select_impl(a), device_sm_count());
  return 1 + (plan.n_split > 1 ? 1 : 0) + (plan.lpt_order ? 1 : 0);
}

int32_t dcp_decode_attn_kernel_kind(const dcp_attn_desc_t* d, int32_t dcp_size) {
  AttnArgs a{};
  if (make_args(d, dcp_size, 1, 1.0f, d ? d->q_len : 1, &a) != DCP_OK) return DCP_KERNEL_NONE;
  return kind_of(select_impl(a));
}

size_t dcp_tree_attn_workspace_size(const dcp_attn_desc_t* d, int32_t dcp_size) {
  AttnArgs a{};
  if (make_tree_args(d, dcp_size, 1, 1.0f, &a) != DCP_OK) return 0;
  return plan_for(a, select_impl(a), device_sm_count()).ws_bytes;
}

int32_t dcp_tree_attn_launches(const dcp_attn_desc_t* d, int32_t dcp_size) {
  AttnArgs a{};
  if (make_tree_args(d, dcp_size, 1, 1.0f, &a) != DCP_OK) return 0;
  const SplitPlan plan = plan_for(a, select_impl(a), device_sm_count());
  return 1 + (plan.n_split > 1 ? 1 : 0) + (plan.lpt_order ? 1 : 0);
}

int32_t dcp_tree_attn_kernel_kind(const dcp_attn_desc_t* d, int32_t dcp_size) {
  AttnArgs a{};
  if (make_tree_args(d, dcp_size, 1, 1.0f, &a) != DCP_OK) return DCP_KERNEL_NONE;
  return kind_of(select_impl(a));
}

dcp_status_t dcp_tree_attn(const dcp_attn_desc_t* d, const void* q, const void* kv_cache,
                           const int32_t* block_tables, const int32_t* seq_lens,
                           const int32_t* q_lens, const uint32_t* tree_mask, int64_t tree_mask_stride,
                           int32_t dcp_size, int32_t interleave, float scale, float* partial_out,
                           float* lse, void* workspace, size_t workspace_bytes, void* stream) {
  NvtxRange range("dcp_tree_attn");
  AttnArgs a{};
  const dcp_status_t st = make_tree_args(d, dcp_size, interleave, scale, &a);
  if (st != DCP_OK) return st;
  if (!q || !kv_cache || !block_tables || !seq_lens || !tree_mask || !partial_out || !lse)
    return DCP_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(kv_cache, 16) || !aligned(partial_out, 16) || !aligned(lse, 4) ||
      !aligned(tree_mask, 4))
    return DCP_ERR_INVALID_ARG;
  if (tree_mask_stride != 0 && tree_mask_stride < (int64_t)a.Lq * a.tree_words) return DCP_ERR_INVALID_ARG;
  const Impl impl = select_impl(a);
  const SplitPlan plan = plan_for(a, impl, device_sm_count());
  if (plan.ws_bytes > 0 && (!workspace || workspace_bytes < plan.ws_bytes || !aligned(workspace, 256)))
    return DCP_ERR_INVALID_ARG;
  a.q = q;
  a.kv = kv_cache;
  a.block_tables = block_tables;
  a.seq_lens = seq_lens;
  a.q_lens = q_lens;
  a.tree_mask = tree_mask;
  a.tree_mask_stride = tree_mask_stride;
  a.partial_out = partial_out;
  a.lse = lse;
  a.workspace = workspace;
  a.workspace_bytes = workspace_bytes;
  a.stream = static_cast<cudaStream_t>(stream);
  a.status = status_ptr(a.stream);
  if (!a.status) return DCP_ERR_CUDA;
  return launch_impl(a, impl, plan);
}

dcp_status_t dcp_rope_steps(const dcp_rope_desc_t* r, const double* inv_freq, uint64_t* steps) {
  if (!rope_ok(r) || !steps) return DCP_ERR_INVALID_ARG;
  const int pairs = r->rot_dim / 2;
  const double two_pi = 6.283185307179586;
  double base = r->base, lo = 0, hi = 0;
  if (!inv_freq) {
    if (!std::isfinite(base) || !(base > 1.0)) return DCP_ERR_INVALID_ARG;
    if (r->scaling < DCP_ROPE_SCALE_NONE || r->scaling > DCP_ROPE_SCALE_YARN) return DCP_ERR_INVALID_ARG;
    if (r->scaling != DCP_ROPE_SCALE_NONE && !(std::isfinite(r->factor) && r->factor > 0.0)) return DCP_ERR_INVALID_ARG;
    if (r->scaling == DCP_ROPE_SCALE_NTK) {
      if (r->rot_dim < 4) return DCP_ERR_INVALID_ARG;
      base *= std::pow(r->factor, (double)r->rot_dim / (r->rot_dim - 2));
    }
    if (r->scaling == DCP_ROPE_SCALE_YARN) {
      if (r->original_max_position < 1 || !(r->beta_slow > 0.0) || !(r->beta_fast > r->beta_slow) ||
          !std::isfinite(r->beta_fast))
        return DCP_ERR_INVALID_ARG;
      auto pair_of = [&](double turns) {
        return r->rot_dim * std::log(r->original_max_position / (turns * two_pi)) / (2.0 * std::log(base));
      };
      lo = std::max(std::floor(pair_of(r->beta_fast)), 0.0);
      hi = std::min(std::ceil(pair_of(r->beta_slow)), (double)(r->rot_dim - 1));
    }
  }
  for (int k = 0; k < pairs; ++k) {
    double f;
    if (inv_freq) {
      f = inv_freq[k];
    } else {
      f = std::pow(base, -2.0 * k / r->rot_dim);
      if (r->scaling == DCP_ROPE_SCALE_LINEAR) f /= r->factor;
      if (r->scaling == DCP_ROPE_SCALE_YARN) {
        const double ramp = std::min(std::max((k - lo) / std::max(hi - lo, 1e-3), 0.0), 1.0);
        f = f / r->factor * ramp + f * (1.0 - ramp);
      }
    }
    if (!std::isfinite(f)) return DCP_ERR_INVALID_ARG;      // (a factor that takes the base or f past a double's range)
    const double turns = f / two_pi;
    const double frac = turns - std::floor(turns);          // [0, 1); 1 after rounding is a whole turn
    steps[k] = frac < 1.0 ? (uint64_t)std::ldexp(frac, 64) : 0;
  }
  return DCP_OK;
}

dcp_status_t dcp_kv_cache_append(const dcp_attn_desc_t* d, const dcp_rope_desc_t* rope, const uint64_t* rope_steps,
                                 const void* new_k, const void* new_v, const void* q,
                                 const dcp_append_strides_t* strides, void* q_out, const int32_t* pos_offsets,
                                 int64_t pos_offsets_stride, const int32_t* q_lens, void* kv_cache,
                                 const int32_t* block_tables, const int32_t* seq_lens, int32_t dcp_size,
                                 int32_t interleave, void* stream) {
  NvtxRange range("dcp_kv_cache_append");
  if (!d || !rope_steps || !new_k || !kv_cache || !block_tables || !seq_lens) return DCP_ERR_INVALID_ARG;
  if (!cache_desc_ok(d, dcp_size, interleave) || !rope_ok(rope)) return DCP_ERR_INVALID_ARG;
  const bool gqa = d->kind == DCP_ATTN_GQA;
  if (gqa != (new_v != nullptr) || (q != nullptr) != (q_out != nullptr)) return DCP_ERR_INVALID_ARG;
  if (rope->rot_offset > d->head_dim_qk - rope->rot_dim) return DCP_ERR_INVALID_ARG;
  if (q && (d->num_q_heads < 1 || (long long)d->num_q_heads * d->head_dim_qk > (1LL << 24))) return DCP_ERR_INVALID_ARG;
  if (!aligned(new_k, 16) || !aligned(kv_cache, 16) || !aligned(rope_steps, 8) || (new_v && !aligned(new_v, 16)) ||
      (q && (!aligned(q, 16) || !aligned(q_out, 16))) || (pos_offsets && !aligned(pos_offsets, 4)))
    return DCP_ERR_INVALID_ARG;
  if (pos_offsets && pos_offsets_stride != 0 && pos_offsets_stride < d->q_len) return DCP_ERR_INVALID_ARG;
  if ((long long)d->batch * d->q_len > INT_MAX) return DCP_ERR_INVALID_ARG;
  const long long k_row = (long long)d->num_kv_heads * d->head_dim_qk;
  const long long q_row = q ? (long long)d->num_q_heads * d->head_dim_qk : 0;
  AppendArgs a{};
  a.k_batch = k_row * d->q_len, a.k_token = k_row;
  a.v_batch = k_row * d->q_len, a.v_token = k_row;
  a.q_batch = q_row * d->q_len, a.q_token = q_row;
  if (strides) {
    auto stride_ok = [](int64_t batch, int64_t token, long long row) {
      return batch % 8 == 0 && token % 8 == 0 && batch >= 0 && (token == 0 || token >= row);
    };
    if (!stride_ok(strides->k_batch, strides->k_token, k_row) ||
        (gqa && !stride_ok(strides->v_batch, strides->v_token, k_row)) ||
        (q && !stride_ok(strides->q_batch, strides->q_token, q_row)))
      return DCP_ERR_INVALID_ARG;
    if (q && q == q_out && (strides->q_token != a.q_token || strides->q_batch != a.q_batch)) return DCP_ERR_INVALID_ARG;
    a.k_batch = strides->k_batch, a.k_token = strides->k_token;
    a.v_batch = strides->v_batch, a.v_token = strides->v_token;
    a.q_batch = strides->q_batch, a.q_token = strides->q_token;
  }
  a.k = new_k, a.v = new_v, a.q = q, a.q_out = q_out;
  a.steps = reinterpret_cast<const unsigned long long*>(rope_steps);
  a.pos_offsets = pos_offsets, a.pos_stride = pos_offsets_stride, a.q_lens = q_lens;
  a.cache = kv_cache, a.block_tables = block_tables, a.seq_lens = seq_lens;
  a.B = d->batch, a.L = d->q_len, a.Hq = q ? d->num_q_heads : 0, a.Hkv = d->num_kv_heads, a.D = d->head_dim_qk;
  a.bs = d->block_size, a.num_blocks = d->num_blocks, a.max_lb = d->max_local_blocks, a.N = dcp_size, a.I = interleave;
  a.rot_dim = rope->rot_dim, a.rot_offset = rope->rot_offset;
  a.interleaved = rope->layout == DCP_ROPE_INTERLEAVED, a.mscale = rope->mscale;
  a.stream = static_cast<cudaStream_t>(stream);
  a.status = status_ptr(a.stream);
  if (!a.status) return DCP_ERR_CUDA;
  return from_cuda(launch_kv_append(a));
}

dcp_status_t dcp_kv_cache_commit(const dcp_attn_desc_t* d, void* kv_cache, const int32_t* block_tables,
                                 const int32_t* seq_lens, const int32_t* q_lens, const int32_t* accepted,
                                 const int32_t* num_accepted, int32_t max_accept, int32_t* new_seq_lens,
                                 int32_t dcp_size, int32_t interleave, void* stream) {
  NvtxRange range("dcp_kv_cache_commit");
  if (!d || !kv_cache || !block_tables || !seq_lens || !accepted || !num_accepted || !new_seq_lens)
    return DCP_ERR_INVALID_ARG;
  if (!cache_desc_ok(d, dcp_size, interleave) || max_accept < 1) return DCP_ERR_INVALID_ARG;
  if (max_accept > DCP_COMMIT_MAX_ACCEPT) return DCP_ERR_UNSUPPORTED;
  if (!aligned(kv_cache, 16)) return DCP_ERR_INVALID_ARG;
  CommitArgs a{};
  a.cache = kv_cache;
  a.gqa = d->kind == DCP_ATTN_GQA;
  a.block_tables = block_tables, a.seq_lens = seq_lens, a.q_lens = q_lens;
  a.accepted = accepted, a.num_accepted = num_accepted, a.new_seq_lens = new_seq_lens;
  a.B = d->batch, a.L = d->q_len, a.max_accept = max_accept;
  a.row16 = d->num_kv_heads * d->head_dim_qk / 8;
  a.bs = d->block_size, a.num_blocks = d->num_blocks, a.max_lb = d->max_local_blocks, a.N = dcp_size, a.I = interleave;
  a.stream = static_cast<cudaStream_t>(stream);
  a.status = status_ptr(a.stream);
  if (!a.status) return DCP_ERR_CUDA;
  return from_cuda(launch_kv_commit(a));
}

}  // extern "C"
