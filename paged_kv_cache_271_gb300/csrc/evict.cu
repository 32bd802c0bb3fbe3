// Eviction from the paged cache by accumulated attention weight: the choice of the positions to keep,
// and their copy onto new pages.
//
// Choice. Request b keeps n = min(context, budget) positions for each KV head: its first `sink`, its last
// `recent`, and of those between the n - sink - recent with the largest sums, equal ones in the order of
// their positions. A float's bits, with the sign's order mended, order like the float (NaN above all):
// the smallest kept sum is found by its digits of 11, 11 and 10 bits, the highest first, from counts of
// the candidates that agree with it so far (radix selection), then kept positions are written in rising
// order. A row of sums belongs to a cluster of up to 8 blocks, each with a contiguous slice that it reads
// from memory once and keeps in shared memory as integers (slices too long for that are read again);
// the blocks' counts are added up, and their places found, through distributed shared memory. (One
// block a row that read it five times: 168 us with the copy for 8 rows of 65536, now 33, of which the
// choice is 20.)
#include <cooperative_groups.h>

#include <atomic>

#include "pkv_device.cuh"
#include "pkv_internal.h"

namespace pkv {

namespace {

constexpr int kSelectThreads = 512;
constexpr int kSelectWarps = kSelectThreads / 32;
constexpr int kDigitBits = 11, kDigits = 1 << kDigitBits;
constexpr int kMostParts = 8;    // blocks of a row
constexpr int kSliceKeys = 8192;  // of a block's slice, kept in shared memory

// Integers that order like the sums: -0 and +0 alike, NaN above everything.
__device__ __forceinline__ uint32_t order_key(float x) {
  if (x != x) return 0xffffffffu;
  const uint32_t u = __float_as_uint(x + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__global__ void __launch_bounds__(kSelectThreads) evict_select_kernel(const EvictSelectArgs a) {
  namespace cg = cooperative_groups;
  cg::cluster_group cluster = cg::this_cluster();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int parts = cluster.num_blocks(), part = cluster.block_rank();
  auto sync_all = [&] {  // (a cluster of one needs no more than a block's barrier)
    if (parts > 1)
      cluster.sync();
    else
      __syncthreads();
  };
  const int j = blockIdx.y, b = blockIdx.z, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  __shared__ __align__(16) int count[kDigits];   // this block's candidates by digit
  __shared__ int above[kSelectWarps], same[kSelectWarps];
  __shared__ int block_above, block_same, found_digit, found_above, found_count;
  __shared__ uint32_t keys[kSliceKeys];
  int ctx = a.context_lens[b];
  if (ctx < 0 || ctx > a.width) {  // left out: nothing is kept
    if (threadIdx.x == 0 && part == 0) atomicOr(a.err, PKV_DEVERR_BAD_CHUNK);
    ctx = 0;
  }
  const int n = min(ctx, a.budget);
  if (j == 0 && part == 0 && threadIdx.x == 0) a.kept_lens[b] = n;
  const float* w = a.weights + ((int64_t)b * a.h_kv + j) * a.width;
  int32_t* kept = a.kept + ((int64_t)b * a.h_kv + j) * a.budget;
  // candidates: positions lo .. hi - 1, of which `need` are kept; this block's are p0 .. p1 - 1
  const int lo = min(a.sink, n), hi = max(lo, ctx - min(a.recent, n - lo));
  int need = n - lo - (ctx - hi);
  const int per = ((hi - lo + parts - 1) / parts + 31) & ~31;
  const int p0 = min(hi, lo + part * per), p1 = min(hi, p0 + per);
  const bool every = need == hi - lo, cached = p1 - p0 <= kSliceKeys;
  auto key_of = [&](int p) { return cached ? keys[p - p0] : order_key(w[p]); };
  uint32_t prefix = 0;  // digits of the smallest kept key so far
  bool exact = false;   // every key from `prefix` on is kept
  if (need > 0 && !every) {
    int shift = 32 - kDigitBits, bits = kDigitBits;
    for (int pass = 0; pass < 3; ++pass) {
      for (int i = threadIdx.x; i < kDigits; i += kSelectThreads) count[i] = 0;
      __syncthreads();
#pragma unroll 4
      for (int p = p0 + threadIdx.x; p < p1; p += kSelectThreads) {
        uint32_t key;
        if (pass == 0) {
          key = order_key(w[p]);
          if (cached) keys[p - p0] = key;
        } else {
          key = key_of(p);
        }
        if (pass == 0 || (key >> (shift + bits)) == prefix)
          atomicAdd(&count[(key >> shift) & ((1u << bits) - 1)], 1);
      }
      sync_all();
      // the digit with `need` candidates at or above it: a thread adds up four digits, highest first
      const int digits = 1 << bits, top = digits - 1 - 4 * (int)threadIdx.x;
      int c[4] = {0, 0, 0, 0}, mine = 0;
      if (top >= 0) {
#pragma unroll
        for (int r = 0; r < kMostParts; ++r) {  // (unrolled: the reads are under way together)
          if (r >= parts) break;
          const int4 v = *reinterpret_cast<const int4*>(cluster.map_shared_rank(count, r) + top - 3);
          c[0] += v.w; c[1] += v.z; c[2] += v.y; c[3] += v.x;
        }
        mine = c[0] + c[1] + c[2] + c[3];
      }
      int x = mine;
#pragma unroll
      for (int o = 1; o < 32; o *= 2) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      if (lane == 31) above[warp] = x;
      __syncthreads();
      for (int v = 0; v < warp; ++v) x += above[v];
      if (x >= need && x - mine < need) {
        int before = x - mine, d = 0;
        while (before + c[d] < need) before += c[d++];
        found_digit = top - d;
        found_above = before;
        found_count = c[d];
      }
      sync_all();  // (the counts have been read: they are cleared next)
      prefix = (prefix << bits) | (uint32_t)found_digit;
      need -= found_above;
      if (need == found_count) {  // all of them are kept: the border lies below the digit
        prefix <<= shift;
        exact = true;
        break;
      }
      bits = pass == 0 ? 11 : 10;
      shift -= bits;
    }
  }
  // positions in rising order; of those equal to the border the first `need`. A warp has a contiguous
  // piece of the slice: it counts, learns what comes before it, and writes.
  const int piece = (((p1 - p0 + kSelectWarps - 1) / kSelectWarps) + 31) & ~31;
  const int w0 = min(p1, p0 + warp * piece), w1 = min(p1, w0 + piece);
  const bool some = need > 0 || every;  // (need has not changed where every candidate or none is kept)
  auto judge = [&](int p, bool& is_above, bool& is_same) {
    const uint32_t key = p < w1 && !every ? key_of(p) : 0u;
    is_above = p < w1 && (every || key > prefix || (exact && key == prefix));
    is_same = p < w1 && !every && !exact && key == prefix;
  };
  if (some) {
    int n_above = 0, n_same = 0;
    for (int q = w0; q < w1; q += 32) {
      bool is_above, is_same;
      judge(q + lane, is_above, is_same);
      n_above += __popc(__ballot_sync(0xffffffffu, is_above));
      n_same += __popc(__ballot_sync(0xffffffffu, is_same));
    }
    __syncthreads();  // (`above` has been read)
    if (lane == 0) {
      above[warp] = n_above;
      same[warp] = n_same;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
      int x = 0, y = 0;
      for (int v = 0; v < kSelectWarps; ++v) {
        x += above[v];
        y += same[v];
      }
      block_above = x;
      block_same = y;
    }
  }
  sync_all();
  if (some) {
    int a0 = 0, s0 = 0;
#pragma unroll
    for (int r = 0; r < kMostParts; ++r) {
      if (r >= part) break;
      a0 += *cluster.map_shared_rank(&block_above, r);
      s0 += *cluster.map_shared_rank(&block_same, r);
    }
    for (int v = 0; v < warp; ++v) {
      a0 += above[v];
      s0 += same[v];
    }
    const uint32_t below = (1u << lane) - 1;
    for (int q = w0; q < w1; q += 32) {
      bool is_above, is_same;
      judge(q + lane, is_above, is_same);
      const uint32_t ma = __ballot_sync(0xffffffffu, is_above), ms = __ballot_sync(0xffffffffu, is_same);
      const int equal = s0 + __popc(ms & below);
      if (is_above || (is_same && equal < need))
        kept[lo + a0 + __popc(ma & below) + min(equal, need)] = q + lane;
      a0 += __popc(ma);
      s0 += __popc(ms);
    }
  }
  const int all = parts * kSelectThreads, me = part * kSelectThreads + threadIdx.x;
  for (int i = me; i < lo; i += all) kept[i] = i;
  for (int i = me; i < ctx - hi; i += all) kept[n - (ctx - hi) + i] = hi + i;
  for (int i = n + me; i < a.budget; i += all) kept[i] = 0;
  if (parts > 1) cluster.sync();  // (no block leaves while another reads its counts)
}

// Copy. A block takes 16 kept positions (a new page) of one KV head; a row is moved by 16-byte lanes.
constexpr int kMoveThreads = 128;

__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const EvictMoveArgs a) {
  const int j = blockIdx.y, b = blockIdx.z, page = blockIdx.x;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // (the choice, where it is just before)
  const int n = a.kept_lens[b];
  const bool wrong = n < 0 || n > a.budget || n > (long long)a.new_pages * kPageSize ||
                     (a.weights && n > a.new_width);
  if (wrong && page == 0 && j == 0 && threadIdx.x == 0) atomicOr(a.err, PKV_DEVERR_BAD_CHUNK);
  if (wrong) return;
  const int i0 = page * kPageSize;
  const int64_t head = (int64_t)b * a.h_kv + j;
  if (i0 < n) {
    const int to = a.new_tables[(int64_t)b * a.new_pages + page];
    const bool to_there = to >= 0 && to < a.num_pages;
    const int per = a.row_bytes / 16;
    bool bad = !to_there;
    if (to_there) {
      uint8_t* const k_to = static_cast<uint8_t*>(a.k_cache) +
                            ((int64_t)to * a.h_kv + j) * kPageSize * a.row_bytes;
      uint8_t* const v_to = static_cast<uint8_t*>(a.v_cache) +
                            ((int64_t)to * a.h_kv + j) * kPageSize * a.row_bytes;
      const int rows = min(kPageSize, n - i0);
      // a thread's pieces, two of K and two of V under way together
      for (int e0 = threadIdx.x; e0 < rows * per; e0 += 2 * kMoveThreads) {
        uint4 k[2], v[2];
        bool there[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int e = e0 + u * kMoveThreads;
          there[u] = false;
          if (e >= rows * per) continue;
          const int r = e / per, c = e - r * per;
          const int p = a.kept[head * a.budget + i0 + r];
          const int from = p >= 0 && p < (long long)a.max_pages * kPageSize
                               ? a.block_tables[(int64_t)b * a.max_pages + p / kPageSize]
                               : -1;
          there[u] = from >= 0 && from < a.num_pages;
          bad |= !there[u];
          if (!there[u]) continue;
          const int64_t at =
              (((int64_t)from * a.h_kv + j) * kPageSize + p % kPageSize) * a.row_bytes + 16 * c;
          k[u] = *reinterpret_cast<const uint4*>(static_cast<uint8_t*>(a.k_cache) + at);
          v[u] = *reinterpret_cast<const uint4*>(static_cast<uint8_t*>(a.v_cache) + at);
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          if (!there[u]) continue;
          const int e = e0 + u * kMoveThreads;
          *reinterpret_cast<uint4*>(k_to + 16 * e) = k[u];
          *reinterpret_cast<uint4*>(v_to + 16 * e) = v[u];
        }
      }
    }
    if (bad) atomicOr(a.err, PKV_DEVERR_BAD_PAGE);
  }
  if (a.weights) {
    for (int64_t i = i0 + threadIdx.x; i < a.new_width; i += kMoveThreads) {
      if (i >= i0 + kPageSize && page + 1 < (int)gridDim.x) break;  // (the last block: the rest)
      float x = 0.f;
      if (i < n) {
        const int p = a.kept[head * a.budget + i];
        if (p >= 0 && p < a.width) x = a.weights[head * a.width + p];
      }
      a.new_weights[head * a.new_width + i] = x;
    }
  }
}

}  // namespace

cudaError_t launch_evict_select(const EvictSelectArgs& a, cudaStream_t s) {
  // blocks a row: none smaller than a slice of 2048, and no more than about two for every SM in all
  int parts = 1;
  while (parts < kMostParts && a.width >= 4096ll * parts && (long long)a.h_kv * a.batch * parts * 2 <= 2 * 152)
    parts *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(parts, a.h_kv, a.batch);
  cfg.blockDim = dim3(kSelectThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = parts;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, evict_select_kernel, a);
}

cudaError_t launch_evict_move(const EvictMoveArgs& a, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((a.budget + kPageSize - 1) / kPageSize, a.h_kv, a.batch);
  cfg.blockDim = dim3(kMoveThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, evict_move_kernel, a);
}

}  // namespace pkv
