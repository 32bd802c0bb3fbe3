// Compaction of an accepted path: of a request's drafted rows, the accepted ones move together
// behind its committed tokens, in both pools and every KV head.
//
// Node path[i] (i < path_lens[b]) sits at position base + path[i] and moves to base + i, base =
// context_lens[b] - tree_lens[b]. The path increases strictly, so path[i] >= i: in path order no
// row is written before it has been read. A thread owns 16 bytes of every row of one head of one
// request and reads kAhead of its rows before it writes the first of them (a row written, i, is
// below every node still to be read, path[k] >= k > i), so threads never wait for one another and
// the moves' latency overlaps. Bound by latency: a step moves a few rows per request (64 requests of
// up to 5 accepted nodes, bf16: 3.0 us a call in a graph, 256 of up to 12, FP8: 3.8).
#include <algorithm>

#include "pkv_device.cuh"
#include "pkv_internal.h"

namespace pkv {

namespace {

constexpr int kThreads = 128;
constexpr int kAhead = 4;

__global__ void __launch_bounds__(kThreads) tree_commit_kernel(const CommitArgs a) {
  const int b = blockIdx.x;
  const int ctx = a.context_lens[b], nodes = a.tree_lens[b], n = a.path_lens[b];
  const int32_t* path = a.path + (size_t)b * a.max_path;
  int bad = nodes < 0 || nodes > ctx || n < 0 || n > nodes || n > a.max_path;
  if (!bad)
    for (int i = threadIdx.x; i < n; i += kThreads)
      bad |= path[i] < 0 || path[i] >= nodes || (i > 0 && path[i] <= path[i - 1]);
  bad = __syncthreads_or(bad);
  const int base = ctx - nodes;
  if (threadIdx.x == 0 && blockIdx.y == 0) {
    if (bad) atomicOr(a.err, PKV_DEVERR_BAD_TREE);
    if (a.new_lens) a.new_lens[b] = bad ? ctx : base + n;
  }
  if (bad) return;
  const int vecs = a.row_bytes / 16;
  const int e = blockIdx.y * kThreads + threadIdx.x;
  if (e >= a.h_kv * vecs) return;
  const int h = e / vecs;
  const int64_t col = (int64_t)(e % vecs) * 16;
  const int32_t* table = a.block_tables + (size_t)b * a.max_pages;
  // byte offset of this thread's part of position p, or -1 (a position the table does not hold,
  // a bad page id)
  auto at = [&](int p) -> int64_t {
    const int id = p / kPageSize < a.max_pages ? table[p / kPageSize] : -1;
    if (id < 0 || id >= a.num_pages) return -1;
    return (((int64_t)id * a.h_kv + h) * kPageSize + p % kPageSize) * a.row_bytes + col;
  };
  uint8_t* kp = static_cast<uint8_t*>(a.k_cache);
  uint8_t* vp = static_cast<uint8_t*>(a.v_cache);
  for (int i0 = 0; i0 < n; i0 += kAhead) {
    uint4 kx[kAhead], vx[kAhead];
    int64_t to[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      to[u] = -1;
      const int i = i0 + u;
      const int from = i < n ? path[i] : i;
      if (from == i) continue;  // stays in its place
      const int64_t src = at(base + from), dst = at(base + i);
      if (src < 0 || dst < 0) {
        atomicOr(a.err, PKV_DEVERR_BAD_PAGE);
        continue;
      }
      to[u] = dst;
      kx[u] = *reinterpret_cast<const uint4*>(kp + src);
      vx[u] = *reinterpret_cast<const uint4*>(vp + src);
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      if (to[u] < 0) continue;
      *reinterpret_cast<uint4*>(kp + to[u]) = kx[u];
      *reinterpret_cast<uint4*>(vp + to[u]) = vx[u];
    }
  }
}

}  // namespace

cudaError_t launch_tree_commit(const CommitArgs& a, cudaStream_t s) {
  const int work = a.h_kv * (a.row_bytes / 16);
  tree_commit_kernel<<<dim3(a.batch, (work + kThreads - 1) / kThreads), kThreads, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace pkv
