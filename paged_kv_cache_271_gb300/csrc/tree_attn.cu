// Tree attention on CUDA cores, for fp32 queries over an fp32, FP8 or INT8 cache, and the combine of
// a split call of any type.
//
// For node t of request b and query head h over KV head j:
//   s_p = scale <q, K_p> for the positions p that node t sees, out = sum_p softmax(s)_p V_p,
// the cached positions before the draft all seen, drafted node i seen when bit i of the mask row
// is set; a row that sees nothing gives 0.
//
// A block takes units of 32 rows over tiles of 64 tokens (tree_plan.cuh). K and V of a tile are fp32
// in shared memory and used by all 32 rows; a thread computes 4 rows x 4 tokens of scores and 4 rows
// x D / 16 dims of the weighted values, so that a 16-byte shared-memory load feeds eight to eleven
// FMAs, issued as pairs. The next tile is on its way meanwhile, into the same buffers: its K comes
// while this tile's softmax and values are worked on, its V during the next scores. The softmax is
// online: the running maximum and sum stay in the registers of the 16 threads that share a row; sums
// are fp32 throughout, as the fp32 types need, and a tile's weighted values are summed before they
// join the whole's.
//
// Bound by FMAs and by the latency of the loads that feed them (two blocks of four warps on an SM):
// 16 requests of 500 .. 4000 tokens, 96 rows a KV head, 128 dims, F32: 15.0 GFLOP in 462 us, 33
// TFLOP/s, two fifths of the fp32 rate (on other lengths 423 us against 503 with 2 rows x 4 tokens a
// thread and 32-token tiles); 32 rows, FP8: 182 us (171 against 278). One request, 2000 tokens, 8 nodes:
// 25 us with its combine (single calls after a flush of the L2 32, 64 threads and 32-token tiles 46).
#include <math.h>

#include <atomic>

#include "pkv_device.cuh"
#include "pkv_internal.h"
#include "tcgen05.cuh"
#include "tree_plan.cuh"

namespace pkv {

namespace {

constexpr int kThreads = 128;
constexpr int kRows = kTreeSimtRows, kTok = kTreeSimtTokens;
constexpr int kPages = kTok / kPageSize;
static_assert(kRows == 32 && kTok == 64, "a thread has 4 rows and 4 tokens of a tile");

template <int D>
struct SimtShape {
  static constexpr int LD = D + 4;   // row pitch (floats): keeps float4 alignment, spreads banks
  static constexpr int LP = kTok + 8;
  static constexpr int SMEM = 4 * ((kRows + 2 * kTok) * LD + kRows * LP);
  static constexpr int CTAS = tree_simt_wave(D) / 152;  // resident on an SM
};

// 16 bytes from global to shared memory, asynchronously; zeros when the source is not there.
__device__ __forceinline__ void copy16(float* dst, const void* src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src),
               "r"(there ? 16 : 0)
               : "memory");
}

template <bool B>
struct Flag {
  static constexpr bool value = B;
};

// Four fp32 values of shared memory as two pairs.
__device__ __forceinline__ ulonglong2 pairs(const float* p) {
  return *reinterpret_cast<const ulonglong2*>(p);
}

template <typename KV, int D>
__global__ void __launch_bounds__(kThreads, SimtShape<D>::CTAS) tree_simt_kernel(const TreeArgs a) {
  using S = SimtShape<D>;
  constexpr bool WIDEN = KV::bytes == 1;
  constexpr int NQ = D / 64;  // float4 groups of dims a thread accumulates, 64 dims apart
  constexpr int LD = S::LD, LP = S::LP;
  extern __shared__ float4 smem4[];
  float* qs = reinterpret_cast<float*>(smem4);
  float* ks = qs + kRows * LD;
  float* vs = ks + kTok * LD;
  float* ps = vs + kTok * LD;
  __shared__ int scratch[64];
  __shared__ TreeShare share;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  tree_share<kThreads>(a, scratch, &share);
  TreeWalk walk(a, share);
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;  // tokens tx + 16 m / dims, rows ty + 8 i
  TreeRun run;
  while (walk.next(a, run)) {
    const int b = run.b, j = run.j;
    const int32_t* table = a.block_tables + (size_t)b * a.max_pages;
    // the pages of a tile: their first rows in the pools, in elements, or -1
    struct Pages {
      int64_t row[kPages];
      bool bad;  // one that should be there is not in the pool
    };
    auto pages_of = [&](int tile) {
      Pages p;
      p.bad = false;
#pragma unroll
      for (int h = 0; h < kPages; ++h) {
        const int lp = kPages * tile + h;
        const bool wanted = lp * kPageSize < run.req.read;
        const int id = wanted ? table[lp] : -1;
        const bool there = id >= 0 && id < a.num_pages;
        p.row[h] = there ? ((int64_t)id * a.h_kv + j) * kPageSize * D : -1;
        p.bad |= wanted && !there;
      }
      return p;
    };
    auto first_row = [](const Pages& p, int h) {  // (no indexing: the rows stay in registers)
      return h < 2 ? (h == 0 ? p.row[0] : p.row[1]) : (h == 2 ? p.row[2] : p.row[3]);
    };
    // A tile of K or V comes into shared memory as fp32, zeros for a page that is not there: from an
    // fp32 pool by asynchronous copies, from an 8-bit one through registers (get, then put).
    auto copy = [&](float* dst, const void* pool, const Pages& p) {
#pragma unroll
      for (int i = 0; i < kTok * D / 4 / kThreads; ++i) {
        const int e = i * kThreads + threadIdx.x, r = e / (D / 4), c = e % (D / 4);
        const int64_t from = first_row(p, r / kPageSize);
        copy16(dst + r * LD + 4 * c,
               static_cast<const float*>(pool) + (from < 0 ? 0 : from + r % kPageSize * D + 4 * c),
               from >= 0);
      }
    };
    auto copied = [] { asm volatile("cp.async.commit_group;" ::: "memory"); };
    constexpr int RAW = WIDEN ? kTok * D / 16 / kThreads : 1;  // 16-code chunks of a thread
    auto get = [&](uint4 (&raw)[RAW], const void* pool, const Pages& p) {
#pragma unroll
      for (int i = 0; i < RAW; ++i) {
        const int e = i * kThreads + threadIdx.x, r = e / (D / 16), c = e % (D / 16);
        const int64_t from = first_row(p, r / kPageSize);
        raw[i] = from < 0 ? make_uint4(0, 0, 0, 0)
                          : *reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(pool) +
                                                            from + r % kPageSize * D + 16 * c);
      }
    };
    auto put = [&](float* dst, const uint4 (&raw)[RAW]) {
#pragma unroll
      for (int i = 0; i < RAW; ++i) {
        const int e = i * kThreads + threadIdx.x, r = e / (D / 16), c = e % (D / 16);
        const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          float o[4];
          RowLoad<KV, 4>::run(reinterpret_cast<const uint8_t*>(&w[k]), o);
          *reinterpret_cast<float4*>(dst + r * LD + 16 * c + 4 * k) =
              make_float4(o[0], o[1], o[2], o[3]);
        }
      }
    };
    uint4 kraw[RAW], vraw[RAW];
    __syncthreads();  // the previous run is done with the shared tiles
    Pages here = pages_of(run.tile0);
    if constexpr (WIDEN) {
      get(kraw, a.k_cache, here);
      get(vraw, a.v_cache, here);
    } else {
      copy(ks, a.k_cache, here);
      copied();
      copy(vs, a.v_cache, here);
      copied();
    }
    for (int e = threadIdx.x; e < kRows * (D / 4); e += kThreads) {
      const int r = e / (D / 4), c = e % (D / 4);
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      if (r < run.rows) {
        const int R = run.row0 + r, t = R / a.group, g = R % a.group;
        v = *reinterpret_cast<const float4*>(
            static_cast<const float*>(a.q) +
            (((int64_t)b * a.nodes + t) * a.h_q + j * a.group + g) * D + 4 * c);
      }
      *reinterpret_cast<float4*>(qs + r * LD + 4 * c) = v;
    }
    if constexpr (WIDEN) {
      put(ks, kraw);
      put(vs, vraw);
    }
    float m[4], l[4];
    uint64_t acc[4][2 * NQ];  // pairs of dims
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      m[i] = -INFINITY;
      l[i] = 0.f;
#pragma unroll
      for (int k = 0; k < 2 * NQ; ++k) acc[i][k] = 0;
    }
    const float sc = a.scale_log2 * (WIDEN ? a.k_scales[j] : 1.f);
    for (int i0 = 0; i0 < run.n; ++i0) {
      const int tile = run.tile0 + i0, p0 = tile * kTok;
      const bool more = i0 + 1 < run.n;
      const bool tail = p0 + kTok > min(run.req.base, run.req.read);  // not all positions seen
      uint64_t page_ok = 0;  // one bit per token
#pragma unroll
      for (int h = 0; h < kPages; ++h)
        if (here.row[h] >= 0) page_ok |= 0xffffull << (16 * h);
      if (here.bad && threadIdx.x == 0) atomicOr(a.err, PKV_DEVERR_BAD_PAGE);
      if (more) here = pages_of(tile + 1);
      if constexpr (WIDEN) {
        if (more) {
          get(kraw, a.k_cache, here);
          get(vraw, a.v_cache, here);
        }
      } else {
        asm volatile("cp.async.wait_group 1;" ::: "memory");  // K (V may still be on its way)
      }
      __syncthreads();
      // ---- scores of rows ty + 8 i, tokens tx + 16 m: sums of even and of odd dims ----
      uint64_t s2[4][4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) s2[i][k] = 0;
#pragma unroll 4
      for (int d = 0; d < D; d += 4) {
        ulonglong2 k[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) k[t] = pairs(ks + (tx + 16 * t) * LD + d);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const ulonglong2 q = pairs(qs + (ty + 8 * i) * LD + d);
#pragma unroll
          for (int t = 0; t < 4; ++t) s2[i][t] = fma2(q.y, k[t].y, fma2(q.x, k[t].x, s2[i][t]));
        }
      }
      __syncthreads();  // K is used up: the next tile's comes in its place
      if constexpr (WIDEN) {
        if (more) put(ks, kraw);
      } else {
        if (more) copy(ks, a.k_cache, here);
        copied();
      }
      // ---- online softmax; a row's 16 threads hold the same m and l ----
      uint64_t seen[4];
      float scale[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int R = ty + 8 * i;
        seen[i] = page_ok;
        if (tail)
          seen[i] &= R < run.rows
                         ? tree_seen(a, run.req, b, (run.row0 + R) / a.group, p0)
                         : 0ull;
        float s[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          float even, odd;
          unpack2(s2[i][t], even, odd);
          s[t] = (seen[i] >> (tx + 16 * t)) & 1 ? (even + odd) * sc : -INFINITY;
        }
        float mx = fmaxf(fmaxf(s[0], s[1]), fmaxf(s[2], s[3]));
#pragma unroll
        for (int o = 8; o >= 1; o /= 2) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        const float mn = fmaxf(m[i], mx);
        const float mu = mn == -INFINITY ? 0.f : mn;
        const float alpha = exp2f(m[i] - mu);
        float sum = 0.f;
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const float e = exp2f(s[t] - mu);
          ps[R * LP + tx + 16 * t] = e;
          sum += e;
        }
#pragma unroll
        for (int o = 8; o >= 1; o /= 2) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        l[i] = fmaf(l[i], alpha, sum);
        m[i] = mn;
        scale[i] = alpha;
      }
      if constexpr (WIDEN) {
        __syncwarp();  // a row's P is written and read by the same half warp
      } else {
        asm volatile("cp.async.wait_group 1;" ::: "memory");  // V
        __syncthreads();
      }
      // ---- weighted values of rows ty + 8 i, dims 4 tx + 64 k ..: the tile's own sums first, so that
      // a long context's sums do not round once per token against the whole ----
      uint64_t own[4][2 * NQ];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int k = 0; k < 2 * NQ; ++k) own[i][k] = 0;
      // an unseen value may be infinite or NaN, which a weight of 0 does not remove: where some
      // positions are not seen, a token whose values are not all finite takes part row by row
      auto weigh = [&](auto careful_) {
      constexpr bool careful = decltype(careful_)::value;
#pragma unroll 2
      for (int t = 0; t < kTok; t += 4) {
        float4 p[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          p[i] = *reinterpret_cast<const float4*>(ps + (ty + 8 * i) * LP + t);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          ulonglong2 v[NQ];
#pragma unroll
          for (int k = 0; k < NQ; ++k) v[k] = pairs(vs + (t + u) * LD + 4 * tx + 64 * k);
          bool hot = false;
          if constexpr (careful) {
            uint64_t z = 0;  // sums of 0 v
#pragma unroll
            for (int k = 0; k < NQ; ++k) z = fma2(v[k].y, 0, fma2(v[k].x, 0, z));
            float z0, z1;
            unpack2(z, z0, z1);
            hot = z0 + z1 != 0.f;
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (careful && hot && !((seen[i] >> (t + u)) & 1)) continue;
            const float w = u == 0 ? p[i].x : u == 1 ? p[i].y : u == 2 ? p[i].z : p[i].w;
            const uint64_t ww = pack2(w, w);
#pragma unroll
            for (int k = 0; k < NQ; ++k) {
              own[i][2 * k] = fma2(ww, v[k].x, own[i][2 * k]);
              own[i][2 * k + 1] = fma2(ww, v[k].y, own[i][2 * k + 1]);
            }
          }
        }
      }
      };
      if (tail || page_ok != ~0ull)
        weigh(Flag<true>{});
      else
        weigh(Flag<false>{});
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint64_t c = pack2(scale[i], scale[i]);
#pragma unroll
        for (int k = 0; k < 2 * NQ; ++k) acc[i][k] = fma2(acc[i][k], c, own[i][k]);
      }
      __syncthreads();  // V is used up
      if constexpr (WIDEN) {
        if (more) put(vs, vraw);
      } else {
        if (more) copy(vs, a.v_cache, here);
        copied();
      }
    }
    // ---- the run's rows: finished, or a partial ----
    const float vsc = WIDEN ? a.v_scales[j] : 1.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = ty + 8 * i;
      if (r >= run.rows) continue;
      float* o;
      if (run.whole) {
        const int R = run.row0 + r, t = R / a.group, g = R % a.group;
        o = static_cast<float*>(a.out) +
            (((int64_t)b * a.nodes + t) * a.h_q + j * a.group + g) * D + 4 * tx;
      } else {
        const size_t part = ((size_t)blockIdx.x * 2 + run.slot) * kRows + r;
        o = a.ws_acc + part * D + 4 * tx;
        if (tx == 0) *reinterpret_cast<float2*>(a.ws_ml + 2 * part) = make_float2(m[i], l[i]);
      }
#pragma unroll
      for (int k = 0; k < NQ; ++k) {
        float4 v;
        unpack2(acc[i][2 * k], v.x, v.y);
        unpack2(acc[i][2 * k + 1], v.z, v.w);
        if (!run.whole)
          v = make_float4(v.x * vsc, v.y * vsc, v.z * vsc, v.w * vsc);
        else if (l[i] != 0.f)  // (a NaN sum stays NaN)
          v = make_float4(v.x / l[i] * vsc, v.y / l[i] * vsc, v.z / l[i] * vsc, v.w / l[i] * vsc);
        else
          v = make_float4(0.f, 0.f, 0.f, 0.f);
        *reinterpret_cast<float4*>(o + 64 * k) = v;
      }
    }
  }
}

// ---- combine ---------------------------------------------------------------------------------

// Rows of the passes that crossed shares: with partials c = 0 .. n-1 of a row in share order,
// M = max m_c, out = sum 2^(m_c - M) acc_c / sum 2^(m_c - M) l_c. A warp merges RW rows, reading
// the (m, l) pairs of up to 32 partials of each at once and the values of CB partials of each
// together: a row is two reads that wait on one another, so what counts is how many are under way.
// Few rows in all: one row per warp (with the attention, one request of 8 nodes: 20 us against 24 with
// four rows a warp, over 8000 tokens 30 against 36); many: four, in fewer blocks, each of which has to
// find its place in the split first (64 ragged drafts of up to 256 rows: 141 us against 162 with one;
// 128 requests of 192 rows a head, FP8: 366 against 401). Launched as a programmatic dependent: blocks that start early find it while
// the attention still runs.
constexpr int kCombineThreads = 128;
constexpr int kCombineWarps = kCombineThreads / 32;

template <typename TQ, int D, int RW, int CB>
__global__ void __launch_bounds__(kCombineThreads) tree_combine_kernel(const TreeArgs a) {
  constexpr int DL = D / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int j = blockIdx.y, b = blockIdx.z;
  const int row_block = blockIdx.x * (kCombineWarps * RW);
  __shared__ int scratch[4][32];
  const TreeReq req = tree_request(a, b);
  const TreeSize z = tree_size(a, req);
  const int rows = req.nodes * a.group;
  // this grid must not complete before the attention does, also when nothing is left to merge
  const bool first_block = blockIdx.x == 0 && j == 0 && b == 0;
  if (row_block >= rows) {
    if (first_block) asm volatile("griddepcontrol.wait;" ::: "memory");
    return;
  }
  int work = 0, passes = 0, work_before = 0, passes_before = 0;
  for (int i = threadIdx.x; i < a.batch; i += kCombineThreads) {
    const TreeSize y = tree_size(a, tree_request(a, i));
    const int w = tree_work(a, y) * a.h_kv, p = y.units * a.h_kv;
    work += w;
    passes += p;
    if (i < b) {
      work_before += w;
      passes_before += p;
    }
  }
  int below, work_all, passes_all, work_pre, passes_pre;
  block_scan<kCombineThreads>(work, scratch[0], below, work_all);
  block_scan<kCombineThreads>(passes, scratch[1], below, passes_all);
  block_scan<kCombineThreads>(work_before, scratch[2], below, work_pre);
  block_scan<kCombineThreads>(passes_before, scratch[3], below, passes_pre);
  const TreeStream st = tree_stream(a, work_all, passes_all);
  const int unit = row_block / a.unit_rows;  // (a block's rows lie in one unit)
  // the pass's tiles in the stream, and the shares that hold the ends of its first and last
  const int tile = unit == z.units - 1 ? z.last_tile : a.wide_tile;
  const int start = work_pre + st.pass_cost * passes_pre +
                    j * (tree_work(a, z) + z.units * st.pass_cost) +
                    unit * (z.tiles * a.wide_tile + st.pass_cost) + st.pass_cost;
  const int c0 = (start + tile - 1) / st.share, c1 = (start + z.tiles * tile - 1) / st.share;
  if (c0 == c1) {
    if (first_block) asm volatile("griddepcontrol.wait;" ::: "memory");
    return;
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int n = c1 - c0 + 1;
  const int first = row_block + warp * RW;  // this warp's rows
  const int live = min(RW, rows - first);
  if (live <= 0) return;
  auto part = [&](int i, int c) {  // partial c of row first + i (the pass begins in share c0)
    return ((size_t)(c0 + c) * 2 + (c == 0 ? 1 : 0)) * a.unit_rows + first + min(i, live - 1) -
           unit * a.unit_rows;
  };
  float M[RW], L[RW], A[RW][DL];
#pragma unroll
  for (int i = 0; i < RW; ++i) {
    M[i] = -INFINITY;
    L[i] = 0.f;
#pragma unroll
    for (int k = 0; k < DL; ++k) A[i][k] = 0.f;
  }
  for (int q0 = 0; q0 < n; q0 += 32) {
    const int nc = min(32, n - q0);
    float2 ml[RW];
#pragma unroll
    for (int i = 0; i < RW; ++i) {
      ml[i] = make_float2(-INFINITY, 0.f);
      if (lane < nc) ml[i] = *reinterpret_cast<const float2*>(a.ws_ml + 2 * part(i, q0 + lane));
    }
    float w[RW];
#pragma unroll
    for (int i = 0; i < RW; ++i) {
      float mr = ml[i].x;
#pragma unroll
      for (int o = 16; o >= 1; o /= 2) mr = fmaxf(mr, __shfl_xor_sync(0xffffffffu, mr, o));
      const float Mn = fmaxf(M[i], mr);
      const float Mu = Mn == -INFINITY ? 0.f : Mn;
      const float rescale = exp2f(M[i] - Mu);
      // a partial that saw nothing weighs 0; a NaN sum stays one whatever its weight
      w[i] = ml[i].x == -INFINITY ? 0.f : exp2f(ml[i].x - Mu);
      float lw = w[i] != 0.f || ml[i].y != ml[i].y ? w[i] * ml[i].y : 0.f;
#pragma unroll
      for (int o = 16; o >= 1; o /= 2) lw += __shfl_xor_sync(0xffffffffu, lw, o);
      L[i] = fmaf(L[i], rescale, lw);
#pragma unroll
      for (int k = 0; k < DL; ++k) A[i][k] *= rescale;
      M[i] = Mn;
    }
    for (int q = 0; q < nc; q += CB) {
      float v[RW][CB][DL];
#pragma unroll
      for (int i = 0; i < RW; ++i)
#pragma unroll
        for (int u = 0; u < CB; ++u) {
          const float* src = a.ws_acc + part(i, q0 + min(q + u, nc - 1)) * D + lane * DL;
          if constexpr (DL == 4) {
            const float4 x = *reinterpret_cast<const float4*>(src);
            v[i][u][0] = x.x; v[i][u][1] = x.y; v[i][u][2] = x.z; v[i][u][3] = x.w;
          } else {
            const float2 x = *reinterpret_cast<const float2*>(src);
            v[i][u][0] = x.x; v[i][u][1] = x.y;
          }
        }
#pragma unroll
      for (int i = 0; i < RW; ++i)
#pragma unroll
        for (int u = 0; u < CB; ++u) {
          const float wu = __shfl_sync(0xffffffffu, w[i], (q + u) & 31);
          if (q + u < nc && wu != 0.f) {
#pragma unroll
            for (int k = 0; k < DL; ++k) A[i][k] = fmaf(wu, v[i][u][k], A[i][k]);
          }
        }
    }
  }
#pragma unroll
  for (int i = 0; i < RW; ++i) {
    if (i >= live) break;
    const int R = first + i, t = R / a.group, g = R % a.group;
    TQ* o = static_cast<TQ*>(a.out) + (((int64_t)b * a.nodes + t) * a.h_q + j * a.group + g) * D +
            lane * DL;
#pragma unroll
    for (int k = 0; k < DL; ++k) store_from_float(o, k, L[i] != 0.f ? A[i][k] / L[i] : 0.f);
  }
}

template <typename KV, int D>
cudaError_t simt_go(const TreeArgs& a, cudaStream_t s) {
  static std::atomic<unsigned long long> attr_done{0};  // one bit per device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !((attr_done.load() >> dev) & 1ull)) {
    e = cudaFuncSetAttribute(tree_simt_kernel<KV, D>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, SimtShape<D>::SMEM);
    if (e != cudaSuccess) return e;
    if (dev < 64) attr_done.fetch_or(1ull << dev);
  }
  tree_simt_kernel<KV, D><<<a.ctas, kThreads, SimtShape<D>::SMEM, s>>>(a);
  return cudaGetLastError();
}

template <int D>
cudaError_t simt_types(const TreeArgs& a, int kv_dtype, cudaStream_t s) {
  if (kv_dtype == PKV_F32) return simt_go<F32, D>(a, s);
  if (kv_dtype == PKV_FP8_E4M3) return simt_go<FP8, D>(a, s);
  return simt_go<INT8, D>(a, s);
}

template <typename TQ, int D, int RW, int CB>
cudaError_t launch_combine_rows(const TreeArgs& a, cudaStream_t s) {
  constexpr int R = kCombineWarps * RW;
  static_assert(kTreeSimtRows % R == 0 && kTreeTcRows % R == 0, "a block's rows lie in one unit");
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((a.nodes * a.group + R - 1) / R, a.h_kv, a.batch);
  cfg.blockDim = dim3(kCombineThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, tree_combine_kernel<TQ, D, RW, CB>, a);
}

template <typename TQ, int D>
cudaError_t launch_combine(const TreeArgs& a, cudaStream_t s) {
  // one row per warp while its blocks are resident at once
  const long long rows = (long long)a.nodes * a.group * a.h_kv * a.batch;
  return rows <= 152 * 7 * kCombineWarps ? launch_combine_rows<TQ, D, 1, 16>(a, s)
                                         : launch_combine_rows<TQ, D, 4, 4>(a, s);
}

}  // namespace

cudaError_t launch_tree_simt(const TreeArgs& a, int kv_dtype, int head_dim, cudaStream_t s) {
  return head_dim == 64 ? simt_types<64>(a, kv_dtype, s) : simt_types<128>(a, kv_dtype, s);
}

cudaError_t launch_tree_combine(const TreeArgs& a, int q_dtype, int head_dim, cudaStream_t s) {
  if (q_dtype == PKV_BF16)
    return head_dim == 64 ? launch_combine<__nv_bfloat16, 64>(a, s)
                          : launch_combine<__nv_bfloat16, 128>(a, s);
  return head_dim == 64 ? launch_combine<float, 64>(a, s) : launch_combine<float, 128>(a, s);
}

}  // namespace pkv
