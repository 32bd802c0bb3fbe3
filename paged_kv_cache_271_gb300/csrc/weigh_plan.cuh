// How a call that sums attention weights is split over its CTAs.
//
// Request b's counted rows are its last last_rows new tokens (0: all) by the query heads of a KV head. An
// item is a tile of tile_tokens cached positions of one KV head; it takes a step for each unit_rows
// rows that may see some of the tile (one step where there are none: its sums are still written), and one
// more for its beginning. The items of all requests, in order, form one stream of steps, and each CTA
// takes an equal contiguous share of it: early positions of a prompt are seen by all rows, late ones by
// few, and a decode step has one step an item. An item whose steps lie in one share is finished by its
// CTA; one that crosses shares leaves partial sums in each, at most two per CTA (slot 0: the item began
// in an earlier share; slot 1: it began here and goes on), with a record by which the combine adds them in
// share order. The split depends on lengths and grid alone, so equal inputs give equal results.
//
// From tile to tile the steps of an item change by 0 or by step = tile_tokens group / unit_rows, a whole
// number, up or down, between at most three places where that changes: their sum has a closed form.
#pragma once

#include <stdint.h>

#include "chunk_plan.cuh"
#include "pkv_device.cuh"
#include "pkv_internal.h"

namespace pkv {

struct WeighReq {
  ChunkReq r;
  int from;   // first counted token
  int items;  // tiles of its positions
};

__device__ __forceinline__ WeighReq weigh_request(const ChunkArgs& a, int b) {
  WeighReq w{chunk_request(a, b), 0, 0};
  const int ctx = w.r.base + w.r.n;
  if (w.r.err == 0 && ctx > a.width) w.r = ChunkReq{0, 0, 0, PKV_DEVERR_BAD_CHUNK};
  if (w.r.err != 0) return w;
  w.from = a.last_rows > 0 ? max(0, w.r.n - a.last_rows) : 0;
  w.items = tiles_for(a, ctx);
  return w;
}

// Counted tokens t0 .. t1 - 1 may see some positions of item i.
struct WeighTokens {
  int t0, t1;
};

__device__ __forceinline__ WeighTokens weigh_tokens(const ChunkArgs& a, const WeighReq& w, int i) {
  const int p0 = i << a.tile_shift;
  WeighTokens x{max(w.from, p0 - w.r.base), w.r.n};
  if (a.window > 0 && p0 >= a.sink)
    x.t1 = (int)min((long long)x.t1, (long long)p0 + a.tile_tokens - 1 + a.window - w.r.base);
  return x;
}

// Steps of item i, where there are none 0 or less.
__device__ __forceinline__ long long weigh_steps(const ChunkArgs& a, const WeighReq& w, int i) {
  const WeighTokens x = weigh_tokens(a, w, i);
  const long long rows = ((long long)x.t1 - x.t0) * a.group;
  return (rows + a.unit_rows - 1) >> a.rows_shift;  // (towards minus infinity: ceil(rows / unit_rows))
}

// Steps of the first k items, each at least one.
__device__ __forceinline__ long long weigh_below(const ChunkArgs& a, const WeighReq& w, int k) {
  const int step = a.tile_tokens * a.group >> a.rows_shift;
  // the places: from here the first row is the tile's own; the sinks end; the window's end is the chunk's
  const int own = (w.from + w.r.base >> a.tile_shift) + 1;
  int sinks = 0, last = 0;
  if (a.window > 0) {
    const long long x = (long long)w.r.base + w.r.n - a.window - a.tile_tokens + 1;
    sinks = tiles_for(a, a.sink);
    last = max(sinks, x > 0 ? (int)(x + a.tile_tokens - 1 >> a.tile_shift) : 0);
  }
  long long sum = 0;
  for (int i = 0; i < k;) {
    int end = k;
    if (i < own) end = min(end, own);
    if (i < sinks) end = min(end, sinks);
    if (i < last) end = min(end, last);
    const long long n = end - i;
    const long long v = weigh_steps(a, w, i), d = n > 1 ? weigh_steps(a, w, i + 1) - v : 0;
    if (d == 0) {
      sum += n * max(1ll, v);
    } else if (d < 0) {  // m items down to the last with a step of its own
      const long long m = v >= 1 ? min(n, (v - 1) / step + 1) : 0;
      sum += m * v - step * (m * (m - 1) / 2) + (n - m);
    } else {
      const long long m = v >= 1 ? 0 : min(n, (step - v) / step);
      const long long q = n - m;
      sum += m + q * (v + step * m) + step * (q * (q - 1) / 2);
    }
    i = end;
  }
  return sum;
}

// A CTA's share: from item `item` of KV head j of request b on, x into it, `count` long.
struct WeighShare {
  int b, j, item, x, count, share;
};

// Every thread of a block of THREADS takes part (the first warp whole); `out` and `scratch` (32
// words) are shared memory. Argument errors are reported by block 0. Ends with a block barrier.
template <int THREADS>
__device__ __forceinline__ void weigh_share(const ChunkArgs& a, int* scratch, WeighShare* out) {
  const int per = (a.batch + THREADS - 1) / THREADS;
  const int b0 = min(a.batch, (int)threadIdx.x * per), b1 = min(a.batch, b0 + per);
  int mine = 0, err = 0;
  auto length = [&](const WeighReq& w, int k) { return (int)weigh_below(a, w, k) + k; };
  for (int b = b0; b < b1; ++b) {
    const WeighReq w = weigh_request(a, b);
    err |= w.r.err;
    mine += length(w, w.items) * a.h_kv;
  }
  if (err && blockIdx.x == 0) atomicOr(a.err, err);
  if (threadIdx.x == 0) out->count = 0;
  const bool overlap = chunk_rows_overlap(a, err & PKV_DEVERR_BAD_CHUNK);
  int below, total;
  block_scan<THREADS>(mine, scratch, below, total);
  const int share = max(2, (int)(((unsigned)total + a.ctas - 1) / (unsigned)a.ctas));
  const long long start = (long long)blockIdx.x * share;
  if (!overlap && start >= below && start < (long long)below + mine) {
    int at = below, b = b0;
    for (; b < b1 - 1; ++b) {
      const WeighReq w = weigh_request(a, b);
      const int t = length(w, w.items) * a.h_kv;
      if (start < at + t) break;
      at += t;
    }
    out->b = b;
    out->x = (int)start - at;  // (into the request, for the first warp)
    out->count = min(share, total - (int)start);
    out->share = share;
  }
  __syncthreads();
  if (threadIdx.x < 32 && out->count > 0) {
    const WeighReq w = weigh_request(a, out->b);
    const int head = length(w, w.items);
    const int j = (int)((unsigned)out->x / (unsigned)head);
    const int x = out->x - j * head;
    int lo = 0, hi = w.items;  // the last item that begins at or before x is in [lo, hi)
    while (hi - lo > 1) {
      const int step = (hi - lo + 31) / 32, k = lo + (int)threadIdx.x * step;
      const bool before = k < hi && length(w, k) <= x;
      const int last = 31 - __clz(__ballot_sync(0xffffffffu, before));  // (lane 0 always is)
      lo += last * step;
      hi = min(hi, lo + step);
    }
    __syncwarp();
    if (threadIdx.x == 0) {
      out->j = j;
      out->item = lo;
      out->x = x - length(w, lo);
    }
  }
  __syncthreads();
}

// A run of steps of one item.
struct WeighRun {
  ChunkReq req;
  int b, j, item;
  int t0, rows;  // first token of the item's rows, the rows: row r is token t0 + r / group, head
                 // r % group of the KV head's
  int s0, n;     // steps s0 .. s0 + n - 1 (rows = 0: one step without rows)
  bool whole;    // the item lies in this share
  int slot;      // partial slot otherwise
  int shares;    // slot 1: later shares that the item reaches into
};

// Walks a share run by run. Uniform over its callers.
struct WeighWalk {
  int b, left, share;
  WeighReq w;  // of request b
  int j, item, x;
  __device__ __forceinline__ WeighWalk(const ChunkArgs& a, const WeighShare& s)
      : b(s.b), left(s.count), share(s.share) {
    if (left <= 0) return;
    w = weigh_request(a, b);
    j = s.j;
    item = s.item;
    x = s.x;
  }
  __device__ __forceinline__ bool next(const ChunkArgs& a, WeighRun& r) {
    while (left > 0) {
      if (j >= a.h_kv || w.items == 0) {
        if (++b >= a.batch) return false;
        w = weigh_request(a, b);
        j = item = x = 0;
        continue;
      }
      const int steps = (int)max(1ll, weigh_steps(a, w, item)), len = steps + 1;
      const int x0 = x, x1 = min(len, x0 + left);
      const int s0 = max(0, x0 - 1), s1 = max(0, x1 - 1);
      const WeighTokens t = weigh_tokens(a, w, item);
      r.req = w.r;
      r.b = b;
      r.j = j;
      r.item = item;
      r.t0 = t.t0;
      r.rows = max(0, t.t1 - t.t0) * a.group;
      r.s0 = s0;
      r.n = s1 - s0;
      r.whole = r.n == steps;
      r.slot = s0 > 0 ? 0 : 1;
      r.shares = (len - x1 + share - 1) / share;
      left -= x1 - x0;
      x = x1;
      if (x == len) {
        x = 0;
        if (++item == w.items) {
          item = 0;
          ++j;
        }
      }
      if (s1 > s0) return true;
    }
    return false;
  }
};

// What the combine reads of the item that begins in a share and goes on (shares = 0: there is none).
struct WeighRecord {
  int row;  // b * h_kv + j
  int p0;   // its first position
  int n;    // its positions
  int shares;
};

}  // namespace pkv
