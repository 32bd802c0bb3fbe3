// Eviction from the paged cache by accumulated attention weight: the choice of the positions to keep,
// and their copy onto new pages.
//
// Choice. Request b keeps n = min(context, budget) positions for each KV head: its first `sink`, its last
// `recent`, and of those between the n - sink - recent with the largest sums, equal ones in the order of
// their positions. A float's bits, with the sign's order mended, order like the float (NaN above all):
// the smallest kept sum is found by its digits, the highest first, from counts of the candidates that
// agree with it so far (radix selection), then kept positions are written in rising order.
#include <atomic>

#include "pkv_device.cuh"
#include "pkv_internal.h"

namespace pkv {

namespace {

constexpr int kSelectThreads = 512;
constexpr int kDigitBits = 8, kDigits = 1 << kDigitBits;

// Integers that order like the sums: -0 and +0 alike, NaN above everything.
__device__ __forceinline__ uint32_t order_key(float x) {
  if (x != x) return 0xffffffffu;
  const uint32_t u = __float_as_uint(x + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// Sums of v over the threads before this one; *total: over all. Two barriers.
__device__ __forceinline__ int scan_before(int v, int* scratch, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o *= 2) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();
  if (lane == 31) scratch[warp] = x;
  __syncthreads();
  int below = x - v, all = 0;
#pragma unroll
  for (int w = 0; w < kSelectThreads / 32; ++w) {
    if (w < warp) below += scratch[w];
    all += scratch[w];
  }
  *total = all;
  return below;
}

__global__ void __launch_bounds__(kSelectThreads) evict_select_kernel(const EvictSelectArgs a) {
  const int j = blockIdx.x, b = blockIdx.y;
  __shared__ int count[kDigits], scratch[kSelectThreads / 32], found[2];
  int ctx = a.context_lens[b];
  if (ctx < 0 || ctx > a.width) {  // left out: nothing is kept
    if (threadIdx.x == 0) atomicOr(a.err, PKV_DEVERR_BAD_CHUNK);
    ctx = 0;
  }
  const int n = min(ctx, a.budget);
  if (j == 0 && threadIdx.x == 0) a.kept_lens[b] = n;
  const float* w = a.weights + ((int64_t)b * a.h_kv + j) * a.width;
  int32_t* kept = a.kept + ((int64_t)b * a.h_kv + j) * a.budget;
  // candidates: positions lo .. hi - 1, of which `need` are kept
  const int lo = min(a.sink, n), hi = max(lo, ctx - min(a.recent, n - lo));
  int need = n - lo - (ctx - hi);
  const int all = need;
  uint32_t prefix = 0;  // digits of the smallest kept key so far
  if (need > 0 && need < hi - lo) {
    for (int shift = 32 - kDigitBits; shift >= 0; shift -= kDigitBits) {
      for (int i = threadIdx.x; i < kDigits; i += kSelectThreads) count[i] = 0;
      __syncthreads();
      for (int p = lo + threadIdx.x; p < hi; p += kSelectThreads) {
        const uint32_t key = order_key(w[p]);
        if (shift + kDigitBits == 32 || (key >> (shift + kDigitBits)) == prefix)
          atomicAdd(&count[(key >> shift) & (kDigits - 1)], 1);
      }
      __syncthreads();
      if (threadIdx.x < 32) {  // the digit with `need` candidates at or above it
        int mine = 0;  // lane L: digits 8 (31 - L) .. + 7, the highest first
        const int d0 = (31 - (int)threadIdx.x) * (kDigits / 32);
        for (int d = 0; d < kDigits / 32; ++d) mine += count[d0 + d];
        int x = mine;
#pragma unroll
        for (int o = 1; o < 32; o *= 2) {
          const int y = __shfl_up_sync(0xffffffffu, x, o);
          if ((int)threadIdx.x >= o) x += y;
        }
        if (x >= need && x - mine < need) {
          int above = x - mine, d = d0 + kDigits / 32 - 1;
          while (above + count[d] < need) above += count[d--];
          found[0] = d;
          found[1] = above;
        }
      }
      __syncthreads();
      prefix = (prefix << kDigitBits) | (uint32_t)found[0];
      need -= found[1];
    }
  } else if (need > 0) {
    need = 0;  // every candidate is kept (keys are at least 0, so none equals the border alone)
  }
  // positions in rising order: `need` of those equal to the border, the first ones
  int done = lo, equal = 0;
  for (int i = threadIdx.x; i < lo; i += kSelectThreads) kept[i] = i;
  const bool every = all == hi - lo;
  if (all > 0) {
    for (int p0 = lo; p0 < hi; p0 += kSelectThreads) {
      const int p = p0 + threadIdx.x;
      bool above = false, same = false;
      if (p < hi) {
        const uint32_t key = every ? 0u : order_key(w[p]);
        above = every || key > prefix;
        same = !every && key == prefix;
      }
      int sames, takes;
      const int before = scan_before(same, scratch, &sames);
      const bool take = above || (same && equal + before < need);
      const int at = scan_before(take, scratch, &takes);
      if (take) kept[done + at] = p;
      done += takes;
      equal += sames;
    }
  }
  for (int i = threadIdx.x; i < ctx - hi; i += kSelectThreads) kept[n - (ctx - hi) + i] = hi + i;
  for (int i = n + threadIdx.x; i < a.budget; i += kSelectThreads) kept[i] = 0;
}

// Copy. A block takes 16 kept positions (a new page) of one KV head; a row is moved by 16-byte lanes.
constexpr int kMoveThreads = 128;

__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const EvictMoveArgs a) {
  const int j = blockIdx.y, b = blockIdx.z, page = blockIdx.x;
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
      for (int e = threadIdx.x; e < rows * per; e += kMoveThreads) {
        const int r = e / per, c = e - r * per;
        const int p = a.kept[head * a.budget + i0 + r];
        const int from = p >= 0 && p < (long long)a.max_pages * kPageSize
                             ? a.block_tables[(int64_t)b * a.max_pages + p / kPageSize]
                             : -1;
        if (from < 0 || from >= a.num_pages) {
          bad = true;
          continue;
        }
        const int64_t at =
            (((int64_t)from * a.h_kv + j) * kPageSize + p % kPageSize) * a.row_bytes + 16 * c;
        const uint4 k = *reinterpret_cast<const uint4*>(static_cast<uint8_t*>(a.k_cache) + at);
        const uint4 v = *reinterpret_cast<const uint4*>(static_cast<uint8_t*>(a.v_cache) + at);
        *reinterpret_cast<uint4*>(k_to + 16 * e) = k;
        *reinterpret_cast<uint4*>(v_to + 16 * e) = v;
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
  evict_select_kernel<<<dim3(a.h_kv, a.batch), kSelectThreads, 0, s>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_evict_move(const EvictMoveArgs& a, cudaStream_t s) {
  evict_move_kernel<<<dim3((a.budget + kPageSize - 1) / kPageSize, a.h_kv, a.batch), kMoveThreads, 0,
                      s>>>(a);
  return cudaGetLastError();
}

}  // namespace pkv
