// How a tree-attention call is split over its CTAs, shared by the attention kernels and their
// combine.
//
// Request b reads its cached positions in tiles of tile_tokens; its (node, query head) rows of one
// KV head are cut into units of unit_rows. A (KV head, unit) of b is one pass over b's tiles, and
// the tiles of all passes of all requests, in order, form one stream. Each CTA takes an equal
// contiguous share of it, whatever the lengths: no CTA idles beside a long request, and few rows
// over a long context still fill the GPU. A pass that lies in one share is finished by its CTA; one
// that crosses shares leaves a partial (running maximum, sum, weighted values) in each, at most
// two per CTA (slot 0: the pass began in an earlier share; slot 1: it began here and goes on),
// which the combine merges in share order. The split depends on the lengths and the grid alone, so
// equal inputs give equal results.
#pragma once

#include <stdint.h>

#include "pkv_device.cuh"
#include "pkv_internal.h"

namespace pkv {

struct TreeReq {
  int nodes;  // query positions (0: the request has no work)
  int base;   // position of node 0: the cached positions before it are seen by every node
  int read;   // positions the page table holds, <= base + nodes
  int err;    // device error bits of the request's arguments
};

__device__ __forceinline__ TreeReq tree_request(const TreeArgs& a, int b) {
  const int ctx = a.context_lens[b];
  const int n = a.tree_lens ? a.tree_lens[b] : (ctx > 0 ? a.nodes : 0);
  TreeReq r{0, 0, 0, 0};
  if (n < 0 || n > a.nodes || ctx < n) {
    r.err = PKV_DEVERR_BAD_TREE;
    return r;
  }
  const long long cap = (long long)a.max_pages * kPageSize;
  r.nodes = n;
  r.base = ctx - n;
  r.read = ctx;
  if (ctx > cap) {
    r.err = PKV_DEVERR_BAD_PAGE;
    r.read = (int)cap;
  }
  return r;
}

struct TreeSize {
  int tiles;  // of one pass
  int units;  // row units of one KV head
};

__device__ __forceinline__ TreeSize tree_size(const TreeArgs& a, const TreeReq& r) {
  if (r.nodes == 0) return TreeSize{0, 0};
  return TreeSize{(r.read + a.tile_tokens - 1) / a.tile_tokens,
                  (r.nodes * a.group + a.unit_rows - 1) / a.unit_rows};
}

// (The host refuses a call whose table could hold 2^31 tiles: the stream's positions are ints.)
__device__ __forceinline__ int tree_tiles(const TreeArgs& a, const TreeSize& z) {
  return z.tiles * z.units * a.h_kv;
}

// Sums over a block: `below` of the values of threads before this one, `total` of all. Shared
// scratch of 32 words; every thread of the block calls it.
template <int THREADS>
__device__ __forceinline__ void block_scan(int v, int* scratch, int& below, int& total) {
  constexpr int W = (THREADS + 31) / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o *= 2) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) scratch[warp] = x;
  __syncthreads();
  below = x - v;
  total = 0;
#pragma unroll
  for (int w = 0; w < W; ++w) {
    if (w < warp) below += scratch[w];
    total += scratch[w];
  }
}

// Where a CTA's share begins: in request b at tile `off` of that request's part of the stream,
// `count` tiles long (0: nothing to do).
struct TreeShare {
  int b, off, count;
};

__device__ __forceinline__ int tree_share_size(const TreeArgs& a, int total) {
  return max(a.min_tiles, (int)(((unsigned)total + a.ctas - 1) / (unsigned)a.ctas));
}

// Every thread of a block of THREADS takes part; `out` and `scratch` are shared memory. Argument
// errors are reported by block 0. Ends with a block barrier.
template <int THREADS>
__device__ __forceinline__ void tree_share(const TreeArgs& a, int* scratch, TreeShare* out) {
  const int per = (a.batch + THREADS - 1) / THREADS;
  const int b0 = min(a.batch, (int)threadIdx.x * per), b1 = min(a.batch, b0 + per);
  int mine = 0, err = 0;
  for (int b = b0; b < b1; ++b) {
    const TreeReq r = tree_request(a, b);
    err |= r.err;
    mine += tree_tiles(a, tree_size(a, r));
  }
  if (err && blockIdx.x == 0) atomicOr(a.err, err);
  if (threadIdx.x == 0) out->count = 0;
  int below, total;
  block_scan<THREADS>(mine, scratch, below, total);
  const int share = tree_share_size(a, total);
  const long long start = (long long)blockIdx.x * share;
  if (start >= below && start < below + mine) {
    int at = below, b = b0;
    for (; b < b1 - 1; ++b) {  // (one request per thread up to THREADS requests)
      const int t = tree_tiles(a, tree_size(a, tree_request(a, b)));
      if (start < at + t) break;
      at += t;
    }
    out->b = b;
    out->off = (int)start - at;
    out->count = min(share, total - (int)start);
  }
  __syncthreads();
}

// A run of tiles of one pass.
struct TreeRun {
  TreeReq req;
  int b, j;        // request, KV head
  int row0, rows;  // first row of the unit and its rows: row r is node r / group, head r % group
  int tile0, n;    // tiles tile0 .. tile0 + n - 1
  bool whole;      // the pass lies in this share
  int slot;        // partial slot otherwise
};

// Walks a share run by run. Uniform over its callers (it reads the lengths itself).
struct TreeWalk {
  int b, off, left;
  __device__ __forceinline__ bool next(const TreeArgs& a, TreeRun& r) {
    while (left > 0 && b < a.batch) {
      const TreeReq q = tree_request(a, b);
      const TreeSize z = tree_size(a, q);
      const int t = tree_tiles(a, z);
      if (off >= t) {
        off -= t;
        ++b;
        continue;
      }
      const int pass = (int)((unsigned)off / (unsigned)z.tiles);
      const int unit = (int)((unsigned)pass % (unsigned)z.units);
      r.req = q;
      r.b = b;
      r.j = (int)((unsigned)pass / (unsigned)z.units);
      r.row0 = unit * a.unit_rows;
      r.rows = min(a.unit_rows, q.nodes * a.group - r.row0);
      r.tile0 = off - pass * z.tiles;
      r.n = min(z.tiles - r.tile0, left);
      r.whole = r.n == z.tiles;
      r.slot = r.tile0 > 0 ? 0 : 1;
      off += r.n;
      left -= r.n;
      return true;
    }
    return false;
  }
};

// Which of the 64 positions p0 .. p0 + 63 node t of a request sees, as bits.
__device__ __forceinline__ uint64_t low_bits(int n) {  // the lowest n bits, n clamped to 0 .. 64
  return n <= 0 ? 0ull : n >= 64 ? ~0ull : (1ull << n) - 1;
}

__device__ __forceinline__ uint64_t tree_seen(const TreeArgs& a, const TreeReq& r, int b, int t,
                                              int p0) {
  uint64_t seen = low_bits(r.base - p0);
  const int n0 = p0 - r.base;  // node of bit 0 (negative: a cached position)
  if (n0 > -64) {
    uint64_t w;
    if (a.mask == nullptr) {
      w = low_bits(t + 1 - max(n0, 0));
      if (n0 < 0) w <<= -n0;
    } else {
      const uint64_t* row = a.mask + (size_t)b * a.mask_stride + (size_t)t * a.mask_words;
      if (n0 < 0) {
        w = row[0] << -n0;
      } else {
        const int i = n0 >> 6, s = n0 & 63;
        w = i < a.mask_words ? row[i] >> s : 0ull;
        if (s && i + 1 < a.mask_words) w |= row[i + 1] << (64 - s);
      }
    }
    seen |= w & ~low_bits(r.base - p0);
  }
  return seen & low_bits(r.read - p0);
}

}  // namespace pkv
