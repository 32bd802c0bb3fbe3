// How a chunk-attention call is split over its CTAs.
//
// The new tokens of request b are cut into blocks of unit_tokens whole tokens, so that the block's
// (token, query head) rows of one KV head are at most unit_rows (a token with more query heads than
// that is cut into `subs` parts). A (KV head, block, part) is a unit: one pass over the tiles of
// tile_tokens cached positions that any of its rows sees, from the first to the block's last token
// (causal), without the tiles between the sinks and the window. The units of all requests, in order,
// form one stream of tiles, and each CTA takes an equal contiguous share of it, whatever the lengths:
// a long prompt's late units, a short chunk over a long context and single tokens are cut alike. As
// in the tree attention the stream is measured in half tiles: a tile counts wide_tile, of a last
// block of up to narrow_rows rows 2, and in calls of many tiles a unit is pass_cost tiles longer at
// its beginning. A tile belongs to the share that holds its end. A unit whose tiles lie in one share is
// finished by its CTA; one that crosses shares leaves a partial (running maximum, sum, weighted
// values) in each, at most two per CTA (slot 0: the unit began in an earlier share; slot 1: it began
// here and goes on). The CTA of slot 1 also leaves a record of the unit, from which the combine
// merges the partials in share order. The split depends on lengths and grid alone, so equal inputs
// give equal results.
//
// The tiles of a request's first k units are an arithmetic progression rounded up to tiles: their
// sum is counted in closed form (tiles_below), so that a share's place is found without walking
// thousands of units.
#pragma once

#include <stdint.h>

#include "pkv_device.cuh"
#include "pkv_internal.h"
#include "tree_plan.cuh"

namespace pkv {

struct ChunkReq {
  int n;     // new tokens (0: the request has no work)
  int q0;    // the first one's row in q and out
  int base;  // its position
  int err;   // device error bits of the request's arguments
};

__device__ __forceinline__ ChunkReq chunk_request(const ChunkArgs& a, int b) {
  const int q0 = a.query_starts[b], q1 = a.query_starts[b + 1], ctx = a.context_lens[b];
  ChunkReq r{0, 0, 0, 0};
  if (q0 < 0 || q1 < q0 || q1 > a.num_rows || ctx < q1 - q0) {
    r.err = PKV_DEVERR_BAD_CHUNK;
  } else if (q1 > q0 && ctx > (long long)a.max_pages * kPageSize) {
    r.err = PKV_DEVERR_BAD_PAGE;
  } else {
    r = ChunkReq{q1 - q0, q0, ctx - (q1 - q0), 0};
  }
  return r;
}

// Whether the accepted requests have more rows in all than the call: starts that fall somewhere can give a
// row to several of them. The plan's sums are bounded (by the host) for num_rows rows, so such a call's
// requests are all left out. Every thread of the block calls it, `falls` if a start that it looked at may
// fall (that request is flagged); a barrier.
__device__ __forceinline__ bool chunk_rows_overlap(const ChunkArgs& a, bool falls) {
  if (!__syncthreads_or(falls)) return false;
  long long rows = 0;
#pragma unroll 1
  for (int b = 0; b < a.batch; ++b) rows += chunk_request(a, b).n;
  return rows > a.num_rows;
}

// Tiles that hold the first n positions (their size is a power of two).
__device__ __forceinline__ int tiles_for(const ChunkArgs& a, int n) {
  return (int)((unsigned)n + a.tile_tokens - 1 >> a.tile_shift);
}

// The tiles of a unit: `sinks` from position 0 on, then those from tile `first` on, `n` in all.
struct ChunkTiles {
  int n, sinks, first;
  __device__ __forceinline__ int operator[](int i) const { return i < sinks ? i : first + i - sinks; }
};

__device__ __forceinline__ ChunkTiles chunk_tiles(const ChunkArgs& a, const ChunkReq& r, int block) {
  const int t0 = block * a.unit_tokens, t1 = min(r.n, t0 + a.unit_tokens);
  const int end = tiles_for(a, r.base + t1);
  ChunkTiles x{end, 0, 0};
  if (a.window > 0) {
    const int first = max(0, r.base + t0 + 1 - a.window) >> a.tile_shift, sinks = tiles_for(a, a.sink);
    if (first > sinks) x = ChunkTiles{sinks + end - first, sinks, first};
  }
  return x;
}

// sum over 0 <= i < n of floor((a i + b) / m): whole multiples of m are taken out of a and b, the rest
// counts lattice points below a line, which the same sum with the axes exchanged counts too. (Less than
// m n + m must fit 32 bits: a tile's tokens by a request's blocks, at most 64 2^26 or 128 2^23 here.)
__device__ __forceinline__ long long floor_sum(unsigned n, unsigned m, unsigned a, unsigned b) {
  unsigned long long sum = 0;
  while (n > 0) {
    if (a >= m) {
      const unsigned q = a / m;
      sum += (unsigned long long)n * (n - 1) / 2 * q;
      a -= q * m;
    }
    if (b >= m) {
      const unsigned q = b / m;
      sum += (unsigned long long)q * n;
      b -= q * m;
    }
    const unsigned top = a * n + b;
    if (top < m) break;
    n = top / m;
    b = top - n * m;
    const unsigned t = m;
    m = a;
    a = t;
  }
  return (long long)sum;
}

// Tiles of the first k blocks' units (all of them full blocks).
__device__ __forceinline__ long long tiles_below(const ChunkArgs& a, const ChunkReq& r, int k) {
  if (k <= 0) return 0;
  const int T = a.tile_tokens, U = a.unit_tokens;
  long long n = floor_sum(k, T, U, r.base + U + T - 1);
  if (a.window > 0) {  // from block i1 on, the tiles between the sinks and the window are left out
    const int sinks = tiles_for(a, a.sink);
    const long long from = (long long)(sinks + 1) * T + a.window - 1 - r.base;
    const long long i1 = from <= 0 ? 0 : (from + U - 1) / U;
    if (i1 < k)
      n -= floor_sum(k - (int)i1, T, U, (unsigned)(r.base + i1 * U + 1 - a.window)) -
           (long long)(k - i1) * sinks;
  }
  return n;
}

struct ChunkSize {
  int blocks;
  int last_tile;  // half tiles a tile of the last block's units counts (of the others: wide_tile)
};

__device__ __forceinline__ ChunkSize chunk_size(const ChunkArgs& a, const ChunkReq& r) {
  const int blocks = (r.n + a.unit_tokens - 1) / a.unit_tokens;
  const int rows = (r.n - (blocks - 1) * a.unit_tokens) * a.group;
  return ChunkSize{blocks, rows > a.narrow_rows ? a.wide_tile : 2};
}

// Half tiles of the units of the first k blocks of one KV head (one part each), without pass costs.
__device__ __forceinline__ int chunk_work(const ChunkArgs& a, const ChunkReq& r, const ChunkSize& z,
                                          int k) {
  if (k <= 0) return 0;
  if (k < z.blocks) return (int)tiles_below(a, r, k) * a.wide_tile;
  return (int)tiles_below(a, r, k - 1) * a.wide_tile + chunk_tiles(a, r, k - 1).n * z.last_tile;
}

// block_scan of two values at once (scratch of 64 words).
template <int THREADS>
__device__ __forceinline__ void block_scan2(int v, int w, int* scratch, int& v_below, int& v_total,
                                            int& w_below, int& w_total) {
  constexpr int W = (THREADS + 31) / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v, y = w;
#pragma unroll
  for (int o = 1; o < 32; o *= 2) {
    const int a = __shfl_up_sync(0xffffffffu, x, o), b = __shfl_up_sync(0xffffffffu, y, o);
    if (lane >= o) {
      x += a;
      y += b;
    }
  }
  if (lane == 31) {
    scratch[warp] = x;
    scratch[32 + warp] = y;
  }
  __syncthreads();
  // (every warp adds up the warps' sums for itself)
  int a = lane < W ? scratch[lane] : 0, b = lane < W ? scratch[32 + lane] : 0;
  const int a0 = a, b0 = b;
#pragma unroll
  for (int o = 1; o < 32; o *= 2) {
    const int c = __shfl_up_sync(0xffffffffu, a, o), d = __shfl_up_sync(0xffffffffu, b, o);
    if (lane >= o) {
      a += c;
      b += d;
    }
  }
  v_total = __shfl_sync(0xffffffffu, a, 31);
  w_total = __shfl_sync(0xffffffffu, b, 31);
  v_below = __shfl_sync(0xffffffffu, a - a0, warp) + x - v;
  w_below = __shfl_sync(0xffffffffu, b - b0, warp) + y - w;
}

// A CTA's share: from (request, KV head, block, part) on, x half tiles into that unit, `count` long.
struct ChunkShare {
  int b, j, block, sub, x, count, pass_cost, share;
};

// Every thread of a block of THREADS takes part (the first warp whole); `out` and `scratch` (64
// words) are shared memory. Argument errors are reported by block 0. Ends with a block barrier.
template <int THREADS>
__device__ __forceinline__ void chunk_share(const ChunkArgs& a, int* scratch, ChunkShare* out) {
  const int per = (a.batch + THREADS - 1) / THREADS;
  const int b0 = min(a.batch, (int)threadIdx.x * per), b1 = min(a.batch, b0 + per);
  int work = 0, passes = 0, err = 0;
  for (int b = b0; b < b1; ++b) {
    const ChunkReq r = chunk_request(a, b);
    err |= r.err;
    if (r.n == 0) continue;
    const ChunkSize z = chunk_size(a, r);
    work += chunk_work(a, r, z, z.blocks) * a.subs * a.h_kv;
    passes += z.blocks * a.subs * a.h_kv;
  }
  if (err && blockIdx.x == 0) atomicOr(a.err, err);
  if (threadIdx.x == 0) out->count = 0;
  const bool overlap = chunk_rows_overlap(a, err & PKV_DEVERR_BAD_CHUNK);
  int work_below, work_all, passes_below, passes_all;
  block_scan2<THREADS>(work, passes, scratch, work_below, work_all, passes_below, passes_all);
  const int cost = work_all >= 32 * a.ctas ? 2 * a.pass_cost : 0;
  const int total = work_all + cost * passes_all;
  const int share =
      max(2 * a.min_tiles, (int)(((unsigned)total + a.ctas - 1) / (unsigned)a.ctas));
  const int mine = work + cost * passes, below = work_below + cost * passes_below;
  const long long start = (long long)blockIdx.x * share;
  if (!overlap && start >= below && start < (long long)below + mine) {
    int at = below, b = b0;
    for (; b < b1 - 1; ++b) {
      const ChunkReq r = chunk_request(a, b);
      if (r.n == 0) continue;
      const ChunkSize z = chunk_size(a, r);
      const int t = (chunk_work(a, r, z, z.blocks) + cost * z.blocks) * a.subs * a.h_kv;
      if (start < at + t) break;
      at += t;
    }
    out->b = b;
    out->x = (int)start - at;  // (into the request, for the first warp)
    out->count = min(share, total - (int)start);
    out->pass_cost = cost;
    out->share = share;
  }
  __syncthreads();
  if (threadIdx.x < 32 && out->count > 0) {
    const ChunkReq r = chunk_request(a, out->b);
    const ChunkSize z = chunk_size(a, r);
    const int head = (chunk_work(a, r, z, z.blocks) + cost * z.blocks) * a.subs;
    const int j = (int)((unsigned)out->x / (unsigned)head);
    int x = out->x - j * head;
    // the last block that begins at or before x: 32 candidates at a time
    int lo = 0, hi = z.blocks;  // it is in [lo, hi)
    while (hi - lo > 1) {
      const int step = (hi - lo + 31) / 32, k = lo + (int)threadIdx.x * step;
      const bool before = k < hi && (chunk_work(a, r, z, k) + cost * k) * a.subs <= x;
      const int last = 31 - __clz(__ballot_sync(0xffffffffu, before));  // (lane 0 always is)
      lo += last * step;
      hi = min(hi, lo + step);
    }
    x -= (chunk_work(a, r, z, lo) + cost * lo) * a.subs;
    const int unit = chunk_tiles(a, r, lo).n * (lo == z.blocks - 1 ? z.last_tile : a.wide_tile) + cost;
    __syncwarp();
    if (threadIdx.x == 0) {
      out->j = j;
      out->block = lo;
      out->sub = x / unit;
      out->x = x - out->sub * unit;
    }
  }
  __syncthreads();
}

// A run of tiles of one unit.
struct ChunkRun {
  ChunkReq req;
  int b, j;        // request, KV head
  int t0, tokens;  // first token of the block, its tokens
  int g0, rows;    // first query head of the part; rows: row r is token t0 + r / heads, head
  int heads;       // g0 + r % heads of the KV head's group
  ChunkTiles tiles;
  int i0, n;   // tiles[i0 .. i0 + n - 1]
  bool whole;  // the unit lies in this share
  int slot;    // partial slot otherwise
  int shares;  // slot 1: later shares that the unit reaches into
};

// Walks a share run by run. Uniform over its callers.
struct ChunkWalk {
  int b, left, pass_cost, share;
  ChunkReq req;  // of request b
  ChunkSize z;
  int j, block, sub, x;  // KV head, block, part and offset in its unit of the next run
  __device__ __forceinline__ ChunkWalk(const ChunkArgs& a, const ChunkShare& s)
      : b(s.b), left(s.count), pass_cost(s.pass_cost), share(s.share) {
    if (left <= 0) return;
    load(a);
    j = s.j;
    block = s.block;
    sub = s.sub;
    x = s.x;
  }
  __device__ __forceinline__ void load(const ChunkArgs& a) {
    req = chunk_request(a, b);
    z = chunk_size(a, req);
    j = block = sub = x = 0;
  }
  __device__ __forceinline__ bool next(const ChunkArgs& a, ChunkRun& r) {
    while (left > 0) {
      if (j >= a.h_kv || req.n == 0) {
        if (++b >= a.batch) return false;
        load(a);
        continue;
      }
      const int per = block == z.blocks - 1 ? z.last_tile : a.wide_tile;
      const ChunkTiles tiles = chunk_tiles(a, req, block);
      const int len = tiles.n * per + pass_cost;
      const int x0 = x, x1 = min(len, x0 + left);
      const int i0 = (int)((unsigned)max(0, x0 - pass_cost) / (unsigned)per);
      const int i1 = (int)((unsigned)max(0, x1 - pass_cost) / (unsigned)per);
      r.req = req;
      r.b = b;
      r.j = j;
      r.t0 = block * a.unit_tokens;
      r.tokens = min(a.unit_tokens, req.n - r.t0);
      r.g0 = sub * a.unit_rows;
      r.heads = a.subs > 1 ? min(a.unit_rows, a.group - r.g0) : a.group;
      r.rows = r.tokens * r.heads;
      r.tiles = tiles;
      r.i0 = i0;
      r.n = i1 - i0;
      r.whole = r.n == tiles.n;
      r.slot = i0 > 0 ? 0 : 1;
      // the unit's end lies len - x1 behind this share's, its last tile in the share that holds that
      r.shares = (len - x1 + share - 1) / share;
      left -= x1 - x0;
      x = x1;
      if (x == len) {
        x = 0;
        if (++sub == a.subs) {
          sub = 0;
          if (++block == z.blocks) {
            block = 0;
            ++j;
          }
        }
      }
      if (i1 > i0) return true;
    }
    return false;
  }
};

// Offset of row r of a run in q and out, in rows of head_dim; in lse the same.
__device__ __forceinline__ size_t chunk_row(const ChunkArgs& a, const ChunkRun& run, int r) {
  const int t = (int)((unsigned)r / (unsigned)run.heads);
  return (size_t)(run.req.q0 + run.t0 + t) * a.h_q + run.j * a.group + run.g0 + (r - t * run.heads);
}

// Which of the 64 positions p0 .. p0 + 63 a query at position pq sees, as bits.
__device__ __forceinline__ uint64_t chunk_seen(const ChunkArgs& a, int pq, int p0) {
  uint64_t seen = low_bits(pq + 1 - p0);
  if (a.window > 0) seen &= ~low_bits(pq + 1 - a.window - p0) | low_bits(a.sink - p0);
  return seen;
}

// Whether some of the positions p0 .. p0 + n - 1 are not seen by some of a run's rows.
__device__ __forceinline__ bool chunk_edge(const ChunkArgs& a, const ChunkRun& run, int p0, int n) {
  const int q_first = run.req.base + run.t0, q_last = q_first + run.tokens - 1;
  return p0 + n - 1 > q_first || (a.window > 0 && p0 < q_last + 1 - a.window && p0 + n > a.sink);
}

// What the combine reads of the unit that begins in a share and goes on (rows = 0: there is none).
struct ChunkRecord {
  int row0;   // first row of q and out: (request's first token + block's) * h_q + first head
  int heads;  // row r: r / heads tokens on, head r % heads on
  int rows;
  int shares;
};

}  // namespace pkv
