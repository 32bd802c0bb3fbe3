// How a tree-attention call is split over its CTAs, shared by the attention kernels and their
// combine.
//
// Request b reads its cached positions in tiles of tile_tokens; its (node, query head) rows of one
// KV head are cut into units of unit_rows. A (KV head, unit) of b is one pass over b's tiles, and
// the passes of all requests, in order, form one stream. Each CTA takes an equal contiguous share of
// it, whatever the lengths: no CTA idles beside a long request, and few rows over a long context
// still fill the GPU. The stream is measured in half tiles of work: a tile of a pass of up to
// narrow_rows rows counts 2, of a wider one wide_tile; and beginning a pass (its queries, its
// output) costs a CTA as much as pass_cost, so in calls of many tiles per CTA every pass is that
// much longer, at its beginning: shares with many short passes get fewer tiles. A tile belongs to
// the share that holds its end. A pass whose tiles lie in one share is finished by its CTA; one that
// crosses shares leaves a partial (running maximum, sum, weighted values) in each, at most two per
// CTA (slot 0: the pass began in an earlier share; slot 1: it began here and goes on), which the
// combine merges in share order. The split depends on the lengths and the grid alone, so equal
// inputs give equal results.
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
  int tiles;      // of one pass
  int units;      // row units of one KV head
  int last_tile;  // half tiles a tile of the last unit counts (of the others: wide_tile)
};

__device__ __forceinline__ TreeSize tree_size(const TreeArgs& a, const TreeReq& r) {
  if (r.nodes == 0) return TreeSize{0, 0, 2};
  const int rows = r.nodes * a.group, units = (rows + a.unit_rows - 1) / a.unit_rows;
  return TreeSize{(r.read + a.tile_tokens - 1) / a.tile_tokens, units,
                  rows - (units - 1) * a.unit_rows > a.narrow_rows ? a.wide_tile : 2};
}

// Half tiles of one KV head's passes, without what the passes cost besides.
__device__ __forceinline__ int tree_work(const TreeArgs& a, const TreeSize& z) {
  return z.units == 0 ? 0 : z.tiles * ((z.units - 1) * a.wide_tile + z.last_tile);
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

// The stream of a call: its length, what a pass costs beyond its tiles, and a share's length, in
// half tiles. (The host refuses a call whose table could hold 2^30 of them: positions are ints.)
struct TreeStream {
  int total, pass_cost, share;
};

__device__ __forceinline__ TreeStream tree_stream(const TreeArgs& a, int work, int passes) {
  TreeStream s;
  s.pass_cost = work >= 32 * a.ctas ? 2 * a.pass_cost : 0;
  s.total = work + s.pass_cost * passes;
  s.share = max(2 * a.min_tiles, (int)(((unsigned)s.total + a.ctas - 1) / (unsigned)a.ctas));
  return s;
}

// A request's part of the stream.
__device__ __forceinline__ int tree_length(const TreeArgs& a, const TreeSize& z, int pass_cost) {
  return (tree_work(a, z) + z.units * pass_cost) * a.h_kv;
}

// A CTA's share: from request b on, `off` into that request's part of the stream, `count` long.
struct TreeShare {
  int b, off, count, pass_cost;
};

// Every thread of a block of THREADS takes part; `out` and `scratch` (64 words) are shared memory.
// Argument errors are reported by block 0. Ends with a block barrier.
template <int THREADS>
__device__ __forceinline__ void tree_share(const TreeArgs& a, int* scratch, TreeShare* out) {
  const int per = (a.batch + THREADS - 1) / THREADS;
  const int b0 = min(a.batch, (int)threadIdx.x * per), b1 = min(a.batch, b0 + per);
  int work = 0, passes = 0, err = 0;
  for (int b = b0; b < b1; ++b) {
    const TreeReq r = tree_request(a, b);
    const TreeSize z = tree_size(a, r);
    err |= r.err;
    work += tree_work(a, z) * a.h_kv;
    passes += z.units * a.h_kv;
  }
  if (err && blockIdx.x == 0) atomicOr(a.err, err);
  if (threadIdx.x == 0) out->count = 0;
  int work_below, work_all, passes_below, passes_all;
  block_scan<THREADS>(work, scratch, work_below, work_all);
  block_scan<THREADS>(passes, scratch + 32, passes_below, passes_all);
  const TreeStream s = tree_stream(a, work_all, passes_all);
  const int mine = work + s.pass_cost * passes, below = work_below + s.pass_cost * passes_below;
  const long long start = (long long)blockIdx.x * s.share;
  if (start >= below && start < (long long)below + mine) {
    int at = below, b = b0;
    for (; b < b1 - 1; ++b) {  // (one request per thread up to THREADS requests)
      const int t = tree_length(a, tree_size(a, tree_request(a, b)), s.pass_cost);
      if (start < at + t) break;
      at += t;
    }
    out->b = b;
    out->off = (int)start - at;
    out->count = min(s.share, s.total - (int)start);
    out->pass_cost = s.pass_cost;
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

// Walks a share run by run. Uniform over its callers (it reads the lengths itself, a request's when
// the walk comes to it).
struct TreeWalk {
  int b, left, pass_cost;
  TreeReq req;  // of request b
  TreeSize z;
  int j, unit, x;  // KV head, unit and offset in its pass of the next run
  int wide_tile;
  __device__ __forceinline__ TreeWalk(const TreeArgs& a, const TreeShare& s)
      : b(s.b), left(s.count), pass_cost(s.pass_cost) {
    if (left <= 0) return;
    load(a);
    const int head = tree_work(a, z) + z.units * pass_cost;  // of one KV head
    j = (int)((unsigned)s.off / (unsigned)head);
    x = s.off - j * head;
    while (unit < z.units - 1 && x >= length()) {
      x -= length();
      ++unit;
    }
  }
  __device__ __forceinline__ void load(const TreeArgs& a) {
    req = tree_request(a, b);
    z = tree_size(a, req);
    wide_tile = a.wide_tile;
    j = unit = x = 0;
  }
  __device__ __forceinline__ int tile() const {
    return unit == z.units - 1 ? z.last_tile : wide_tile;
  }
  __device__ __forceinline__ int length() const { return z.tiles * tile() + pass_cost; }
  __device__ __forceinline__ bool next(const TreeArgs& a, TreeRun& r) {
    while (left > 0) {
      if (j >= a.h_kv || z.units == 0) {
        if (++b >= a.batch) return false;
        load(a);
        continue;
      }
      const int len = length(), per = tile();
      const int x0 = x, x1 = min(len, x0 + left);
      const int tile0 = (int)((unsigned)max(0, x0 - pass_cost) / (unsigned)per);
      const int tile1 = (int)((unsigned)max(0, x1 - pass_cost) / (unsigned)per);
      r.req = req;
      r.b = b;
      r.j = j;
      r.row0 = unit * a.unit_rows;
      r.rows = min(a.unit_rows, req.nodes * a.group - r.row0);
      r.tile0 = tile0;
      r.n = tile1 - tile0;
      r.whole = r.n == z.tiles;
      r.slot = tile0 > 0 ? 0 : 1;
      left -= x1 - x0;
      x = x1;
      if (x == len) {
        x = 0;
        if (++unit == z.units) {
          unit = 0;
          ++j;
        }
      }
      if (tile1 > tile0) return true;
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
