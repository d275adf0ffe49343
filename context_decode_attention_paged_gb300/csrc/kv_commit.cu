// Keeping the accepted path of a verified tree: the cache rows of its nodes
// move to the positions right behind the context.
//
// Node a_k goes from position base + a_k to base + k.  The path increases, so
// a_k >= k and a_k < a_(k+1): writing position k overwrites no row that a later
// step still has to read.  A thread owns a 16-byte column of the row and walks
// the path in order, so the moves of a request need no barrier between them;
// four rows are loaded before four are stored, which only moves reads ahead of
// writes.  Columns are independent, requests own their cells.
//
// A request moves a few KB, so the launch and the chain of dependent loads
// (lengths, path, table, row) bound it: one block of 256 threads per request,
// thread k < num_accepted finding and checking the cells of step k.  Measured
// (GB300, one of five in a graph): 64 requests of up to 8 accepted nodes (1 MB) 4.6
// us; 512 of up to 16, rows of 1,152 bytes (8.4 MB), 5.8 us.
#include "dcp_device.cuh"
#include "dcp_internal.h"

namespace dcp {
namespace {

constexpr int kThreads = 256;
constexpr int kAhead = 4;          // rows loaded before the first is stored

__global__ void __launch_bounds__(kThreads) kv_commit_kernel(const CommitArgs a) {
  __shared__ long long from[DCP_COMMIT_MAX_ACCEPT], to[DCP_COMMIT_MAX_ACCEPT];   // 16-byte units; -1: stays
  static_assert(DCP_COMMIT_MAX_ACCEPT <= kThreads, "one thread per accepted node");
  const int b = blockIdx.x, tid = threadIdx.x;
  const int S = a.seq_lens[b];
  const int n = a.q_lens ? a.q_lens[b] : a.L;
  const int m = a.num_accepted[b];
  bool bad = n < 0 || n > a.L || S < n || m < 0 || m > a.max_accept || m > n;
  const long long base = (long long)S - n;
  auto cell = [&](long long t) -> long long {
    const int r = (int)((t / a.I) % a.N);
    const long long j = (t / ((long long)a.I * a.N)) * a.I + t % a.I;
    const long long jb = j / a.bs;
    const int blk = jb < a.max_lb ? a.block_tables[((long long)r * a.B + b) * a.max_lb + jb] : -1;
    if ((unsigned)blk >= (unsigned)a.num_blocks) return -1;
    return ((long long)blk * a.bs + j % a.bs) * a.row16;
  };
  if (!bad && tid < m) {
    const int node = a.accepted[(long long)b * a.max_accept + tid];
    const int before = tid > 0 ? a.accepted[(long long)b * a.max_accept + tid - 1] : -1;
    bad = node <= before || node >= n || before < -1;
    if (!bad && node != tid) {
      from[tid] = cell(base + node);
      to[tid] = cell(base + tid);
      bad = from[tid] < 0 || to[tid] < 0;
    } else {
      to[tid] = -1;
    }
  }
  if (__syncthreads_or(bad)) {
    if (tid == 0) {
      set_status(a.status, DCP_ERR_BOUNDS);
      a.new_seq_lens[b] = S;
    }
    return;
  }
  uint4* pool = static_cast<uint4*>(a.cache);
  const long long pool16 = (long long)a.num_blocks * a.bs * a.row16;
  const int cols = a.gqa ? 2 * a.row16 : a.row16;
  for (int c = tid; c < cols; c += kThreads) {
    uint4* col = c < a.row16 ? pool + c : pool + pool16 + (c - a.row16);
    for (int k0 = 0; k0 < m; k0 += kAhead) {
      uint4 v[kAhead];
#pragma unroll
      for (int k = 0; k < kAhead; ++k)
        if (k0 + k < m && to[k0 + k] >= 0) v[k] = col[from[k0 + k]];
#pragma unroll
      for (int k = 0; k < kAhead; ++k)
        if (k0 + k < m && to[k0 + k] >= 0) col[to[k0 + k]] = v[k];
    }
  }
  if (tid == 0) a.new_seq_lens[b] = (int)(base + m);
}

}  // namespace

cudaError_t launch_kv_commit(const CommitArgs& a) {
  kv_commit_kernel<<<(unsigned)a.B, kThreads, 0, a.stream>>>(a);
  return cudaGetLastError();
}

}  // namespace dcp
