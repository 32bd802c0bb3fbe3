// Tree attention on CUDA cores, for every cache and query type and both head dimensions, and the
// combine of a split call.
//
// For node t of request b and query head h over KV head j:
//   s_p = scale <q, K_p> for the positions p that node t sees, out = sum_p softmax(s)_p V_p,
// the cached positions before the draft all seen, drafted node i seen when bit i of the mask row
// is set; a row that sees nothing gives 0.
//
// A block takes units of 32 rows over tiles of 32 tokens (tree_plan.cuh): K and V of a tile are
// widened to fp32 in shared memory and used by all 32 rows; a thread computes 4 rows x 2 tokens of
// scores and 4 rows x D/16 dims of the weighted values, so each 16-byte shared-memory load feeds
// five to six FMAs. The softmax is online: the running maximum and sum stay in the registers of
// the 16 threads that share a row. It is bound by the FMA rate and by shared memory; the sums are
// fp32 throughout, which the fp32 types need.
#include <math.h>

#include <atomic>

#include "pkv_device.cuh"
#include "pkv_internal.h"
#include "tree_plan.cuh"

namespace pkv {

namespace {

constexpr int kThreads = 128;
constexpr int kRows = kTreeSimtRows, kTok = kTreeSimtTokens;

template <typename KV, int D>
struct SimtShape {
  static constexpr int LD = D + 4;   // row pitch (floats): keeps float4 alignment, spreads banks
  static constexpr int LP = kTok + 4;
  // an fp32 cache's next tile is copied (cp.async) while this one is worked on: two K and V tiles
  static constexpr bool AHEAD = KV::bytes == 4;
  static constexpr int TILES = AHEAD ? 2 : 1;
  static constexpr int SMEM = 4 * ((1 + 2 * TILES) * kRows * LD + kRows * LP);
};
static_assert(kRows == kTok, "Q, K and V tiles have the same shape");

// Four consecutive elements, widened.
template <typename T>
__device__ __forceinline__ float4 load4(const void* base, int64_t i) {
  float o[4];
  RowLoad<T, 4>::run(static_cast<const uint8_t*>(base) + i * T::bytes, o);
  return make_float4(o[0], o[1], o[2], o[3]);
}

__device__ __forceinline__ void fma4(float4& acc, float p, const float4& v) {
  acc.x = fmaf(p, v.x, acc.x);
  acc.y = fmaf(p, v.y, acc.y);
  acc.z = fmaf(p, v.z, acc.z);
  acc.w = fmaf(p, v.w, acc.w);
}

__device__ __forceinline__ void store4(float* p, const float4& v) {
  *reinterpret_cast<float4*>(p) = v;
}

// 16 bytes from global to shared memory, asynchronously; zeros when the source is not there.
__device__ __forceinline__ void copy16(float* dst, const void* src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src),
               "r"(there ? 16 : 0)
               : "memory");
}

template <typename KV, typename Q, int D>
__global__ void __launch_bounds__(kThreads) tree_simt_kernel(const TreeArgs a) {
  using S = SimtShape<KV, D>;
  using TQ = typename Q::storage;
  constexpr int NQ = D / 64;  // float4 groups of dims a thread accumulates, 64 dims apart
  constexpr int LD = S::LD, LP = S::LP;
  extern __shared__ float4 smem4[];
  float* qs = reinterpret_cast<float*>(smem4);
  float* tiles = qs + kRows * LD;  // K and V of a tile, of the next one behind them
  float* ps = tiles + 2 * S::TILES * kTok * LD;
  __shared__ int scratch[64];
  __shared__ TreeShare share;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  tree_share<kThreads>(a, scratch, &share);
  TreeWalk walk(a, share);
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;  // tokens / dims, group of 4 rows
  TreeRun run;
  while (walk.next(a, run)) {
    const int b = run.b, j = run.j;
    __syncthreads();  // the previous run is done with the shared tiles
    for (int e = threadIdx.x; e < kRows * (D / 4); e += kThreads) {
      const int r = e / (D / 4), c = e % (D / 4);
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      if (r < run.rows) {
        const int R = run.row0 + r, t = R / a.group, g = R % a.group;
        v = load4<Q>(a.q, (((int64_t)b * a.nodes + t) * a.h_q + j * a.group + g) * D + 4 * c);
      }
      *reinterpret_cast<float4*>(qs + r * LD + 4 * c) = v;
    }
    float m[4], l[4];
    float4 acc[4][NQ];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      m[i] = -INFINITY;
      l[i] = 0.f;
#pragma unroll
      for (int k = 0; k < NQ; ++k) acc[i][k] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    const float sc = a.scale_log2 * (KV::bytes == 1 ? a.k_scales[j] : 1.f);
    const int32_t* table = a.block_tables + (size_t)b * a.max_pages;
    // a tile's K and V, widened, into buffer `at`; rows past the context or on a bad page are zero
    auto fetch = [&](int tile, float* at) {
      for (int e = threadIdx.x; e < kTok * (D / 4); e += kThreads) {
        const int r = e / (D / 4), c = e % (D / 4), pos = tile * kTok + r;
        const int id = pos < run.req.read ? table[pos / kPageSize] : -1;
        const bool there = id >= 0 && id < a.num_pages;
        const int64_t from =
            there ? (((int64_t)id * a.h_kv + j) * kPageSize + pos % kPageSize) * D + 4 * c : 0;
        float* k = at + r * LD + 4 * c;
        float* v = k + kTok * LD;
        if constexpr (S::AHEAD) {
          copy16(k, static_cast<const float*>(a.k_cache) + from, there);
          copy16(v, static_cast<const float*>(a.v_cache) + from, there);
        } else {
          const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
          *reinterpret_cast<float4*>(k) = there ? load4<KV>(a.k_cache, from) : zero;
          *reinterpret_cast<float4*>(v) = there ? load4<KV>(a.v_cache, from) : zero;
        }
      }
      if constexpr (S::AHEAD) asm volatile("cp.async.commit_group;" ::: "memory");
    };
    if constexpr (S::AHEAD) fetch(run.tile0, tiles);
    for (int i0 = 0; i0 < run.n; ++i0) {
      const int tile = run.tile0 + i0, p0 = tile * kTok;
      const bool tail = p0 + kTok > min(run.req.base, run.req.read);  // not all positions seen
      uint32_t page_ok = 0;  // one bit per token
#pragma unroll
      for (int pg = 0; pg < kTok / kPageSize; ++pg) {
        const int lp = p0 / kPageSize + pg;
        const int id = lp * kPageSize < run.req.read ? table[lp] : -1;
        if (id >= 0 && id < a.num_pages)
          page_ok |= 0xffffu << (16 * pg);
        else if (lp * kPageSize < run.req.read && threadIdx.x == 0)
          atomicOr(a.err, PKV_DEVERR_BAD_PAGE);
      }
      float* ks = tiles;
      if constexpr (S::AHEAD) {
        ks = tiles + (i0 & 1) * 2 * kTok * LD;
        if (i0 + 1 < run.n) {
          fetch(tile + 1, tiles + (~i0 & 1) * 2 * kTok * LD);
          asm volatile("cp.async.wait_group 1;" ::: "memory");
        } else {
          asm volatile("cp.async.wait_group 0;" ::: "memory");
        }
      } else {
        __syncthreads();  // the previous tile is used up
        fetch(tile, tiles);
      }
      const float* vs = ks + kTok * LD;
      __syncthreads();
      // ---- scores of rows 4 ty + i, tokens tx and tx + 16 ----
      float s[4][2];
#pragma unroll
      for (int i = 0; i < 4; ++i) s[i][0] = s[i][1] = 0.f;
#pragma unroll 4
      for (int d = 0; d < D; d += 4) {
        const float4 k0 = *reinterpret_cast<const float4*>(ks + tx * LD + d);
        const float4 k1 = *reinterpret_cast<const float4*>(ks + (tx + 16) * LD + d);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float4 q = *reinterpret_cast<const float4*>(qs + (4 * ty + i) * LD + d);
          s[i][0] = fmaf(q.x, k0.x, fmaf(q.y, k0.y, fmaf(q.z, k0.z, fmaf(q.w, k0.w, s[i][0]))));
          s[i][1] = fmaf(q.x, k1.x, fmaf(q.y, k1.y, fmaf(q.z, k1.z, fmaf(q.w, k1.w, s[i][1]))));
        }
      }
      // ---- online softmax; a row's 16 threads hold the same m and l ----
      uint32_t seen[4];
      float scale[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int R = 4 * ty + i;
        seen[i] = page_ok;
        if (tail)
          seen[i] &= R < run.rows
                         ? (uint32_t)tree_seen(a, run.req, b, (run.row0 + R) / a.group, p0)
                         : 0u;
        s[i][0] = (seen[i] >> tx) & 1 ? s[i][0] * sc : -INFINITY;
        s[i][1] = (seen[i] >> (tx + 16)) & 1 ? s[i][1] * sc : -INFINITY;
        float mx = fmaxf(s[i][0], s[i][1]);
#pragma unroll
        for (int o = 8; o >= 1; o /= 2) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        const float mn = fmaxf(m[i], mx);
        const float mu = mn == -INFINITY ? 0.f : mn;
        const float alpha = exp2f(m[i] - mu);
        const float e0 = exp2f(s[i][0] - mu), e1 = exp2f(s[i][1] - mu);
        float sum = e0 + e1;
#pragma unroll
        for (int o = 8; o >= 1; o /= 2) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        l[i] = fmaf(l[i], alpha, sum);
        m[i] = mn;
        scale[i] = alpha;
        ps[R * LP + tx] = e0;
        ps[R * LP + tx + 16] = e1;
      }
      __syncwarp();  // a row's P is written and read by the same half warp
      // ---- weighted values of rows 4 ty + i, dims 4 tx + 64 k ..: the tile's own sums first, so that
      // a long context's sums do not round once per token against the whole ----
      float4 own[4][NQ];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int k = 0; k < NQ; ++k) own[i][k] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (!tail && page_ok == 0xffffffffu) {
#pragma unroll 4
        for (int t = 0; t < kTok; ++t) {
          float p[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) p[i] = ps[(4 * ty + i) * LP + t];
#pragma unroll
          for (int k = 0; k < NQ; ++k) {
            const float4 v = *reinterpret_cast<const float4*>(vs + t * LD + 4 * tx + 64 * k);
#pragma unroll
            for (int i = 0; i < 4; ++i) fma4(own[i][k], p[i], v);
          }
        }
      } else {  // an unseen value may be infinite or NaN: it takes no part at all
        for (int t = 0; t < kTok; ++t) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (!((seen[i] >> t) & 1)) continue;
            const float p = ps[(4 * ty + i) * LP + t];
#pragma unroll
            for (int k = 0; k < NQ; ++k)
              fma4(own[i][k], p, *reinterpret_cast<const float4*>(vs + t * LD + 4 * tx + 64 * k));
          }
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int k = 0; k < NQ; ++k) {
          acc[i][k].x = fmaf(acc[i][k].x, scale[i], own[i][k].x);
          acc[i][k].y = fmaf(acc[i][k].y, scale[i], own[i][k].y);
          acc[i][k].z = fmaf(acc[i][k].z, scale[i], own[i][k].z);
          acc[i][k].w = fmaf(acc[i][k].w, scale[i], own[i][k].w);
        }
      if constexpr (S::AHEAD) __syncthreads();  // the tile after the next may overwrite this one
    }
    // ---- the run's rows: finished, or a partial ----
    const float vsc = KV::bytes == 1 ? a.v_scales[j] : 1.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = 4 * ty + i;
      if (r >= run.rows) continue;
      if (run.whole) {
        const int R = run.row0 + r, t = R / a.group, g = R % a.group;
        TQ* o = static_cast<TQ*>(a.out) +
                (((int64_t)b * a.nodes + t) * a.h_q + j * a.group + g) * D + 4 * tx;
#pragma unroll
        for (int k = 0; k < NQ; ++k) {
          const float4 v = acc[i][k];
          const bool any = l[i] != 0.f;  // (a NaN sum stays NaN)
          store4(o + 64 * k, any ? make_float4(v.x / l[i] * vsc, v.y / l[i] * vsc,
                                               v.z / l[i] * vsc, v.w / l[i] * vsc)
                                 : make_float4(0.f, 0.f, 0.f, 0.f));
        }
      } else {
        const size_t part = ((size_t)blockIdx.x * 2 + run.slot) * kRows + r;
#pragma unroll
        for (int k = 0; k < NQ; ++k) {
          const float4 v = acc[i][k];
          store4(a.ws_acc + part * D + 4 * tx + 64 * k,
                 make_float4(v.x * vsc, v.y * vsc, v.z * vsc, v.w * vsc));
        }
        if (tx == 0) {
          a.ws_ml[2 * part] = m[i];
          a.ws_ml[2 * part + 1] = l[i];
        }
      }
    }
  }
}

// ---- combine ---------------------------------------------------------------------------------

// Rows of the passes that crossed shares: with partials c = 0 .. n-1 of a row in share order,
// M = max m_c, out = sum 2^(m_c - M) acc_c / sum 2^(m_c - M) l_c. A warp merges RW rows, reading
// the (m, l) pairs of up to 32 partials of each at once and the values of CB partials of each
// together: a row is two reads that wait on one another, so what counts is how many are under way.
// Few rows in all: one row per warp; many: four, in fewer blocks, each of which has to find its place
// in the split first. Launched as a programmatic dependent: blocks that start early find it while
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

template <typename KV, typename Q, int D>
cudaError_t simt_go(const TreeArgs& a, cudaStream_t s) {
  static std::atomic<unsigned long long> attr_done{0};  // one bit per device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !((attr_done.load() >> dev) & 1ull)) {
    e = cudaFuncSetAttribute(tree_simt_kernel<KV, Q, D>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, SimtShape<KV, D>::SMEM);
    if (e != cudaSuccess) return e;
    if (dev < 64) attr_done.fetch_or(1ull << dev);
  }
  tree_simt_kernel<KV, Q, D><<<a.ctas, kThreads, SimtShape<KV, D>::SMEM, s>>>(a);
  return cudaGetLastError();
}

template <int D>
cudaError_t simt_types(const TreeArgs& a, int kv_dtype, cudaStream_t s) {
  if (kv_dtype == PKV_F32) return simt_go<F32, F32, D>(a, s);
  if (kv_dtype == PKV_FP8_E4M3) return simt_go<FP8, F32, D>(a, s);
  return simt_go<INT8, F32, D>(a, s);
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
