// Attention of chunks of new tokens over the paged cache on CUDA cores, for fp32 queries, and the
// combine of a split call of any type.
//
// For the new token at position pq of a request and query head h over KV head j:
//   s_p = scale <q, K_p>, capped: s_p <- c tanh(s_p / c), with a bias: s_p <- s_p - slope_h (pq - p),
//   out = sum_p softmax(s)_p V_p, lse = ln sum_p e^{s_p}
// over the positions p <= pq (with a window W and S sinks those with p > pq - W or p < S).
//
// A block takes units of 32 rows over tiles of 64 tokens (chunk_plan.cuh), as the tree attention on CUDA
// cores does: K and V of a tile are fp32 in shared memory and used by all 32 rows; a thread computes 4
// rows x 4 tokens of scores and 4 rows x D / 16 dims of the weighted values, as paired FMAs. The next
// tile's K comes while this one's softmax and values are worked on, its V during the next scores.
// Sums are fp32 throughout, a tile's weighted values are summed before they join the whole's.
#include <math.h>

#include <atomic>

#include "chunk_plan.cuh"
#include "chunk_score.cuh"
#include "pkv_device.cuh"
#include "pkv_internal.h"
#include "tcgen05.cuh"

namespace pkv {

namespace {

constexpr int kThreads = 128;
constexpr int kRows = kChunkSimtRows, kTok = kChunkSimtTokens;
constexpr int kPages = kTok / kPageSize;
static_assert(kRows == 32 && kTok == 64, "a thread has 4 rows and 4 tokens of a tile");

template <int D>
struct SimtShape {
  static constexpr int LD = D + 4;   // row pitch (floats): keeps float4 alignment, spreads banks
  static constexpr int LP = kTok + 8;
  static constexpr int SMEM = 4 * ((kRows + 2 * kTok) * LD + kRows * LP);
  static constexpr int CTAS = chunk_simt_wave(D) / 152;  // resident on an SM
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

__device__ __forceinline__ void store4(float* p, float4 v) { *reinterpret_cast<float4*>(p) = v; }

template <typename KV, int D>
__global__ void __launch_bounds__(kThreads, SimtShape<D>::CTAS) chunk_simt_kernel(const ChunkArgs a) {
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
  __shared__ ChunkShare share;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  chunk_share<kThreads>(a, scratch, &share);
  ChunkWalk walk(a, share);
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;  // tokens tx + 16 m / dims, rows ty + 8 i
  ChunkRecord record{0, 1, 0, 0};
  ChunkRun run;
  while (walk.next(a, run)) {
    const int j = run.j;
    const int ctx = run.req.base + run.req.n;
    const int32_t* table = a.block_tables + (size_t)run.b * a.max_pages;
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
        // (a page outside every row's window may have been given back: it is not read)
        const int p0 = lp * kPageSize;
        const bool wanted = p0 < ctx && (a.window <= 0 || p0 < a.sink ||
                                         p0 + kPageSize > run.req.base + run.t0 + 1 - a.window);
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
    // fp32 pool by asynchronous copies, from a narrower one through registers (get, then put).
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
    constexpr int EL = WIDEN ? 16 / KV::bytes : 4;               // elements of a 16-byte chunk
    constexpr int RAW = WIDEN ? kTok * D / EL / kThreads : 1;    // chunks of a thread
    auto get = [&](uint4 (&raw)[RAW], const void* pool, const Pages& p) {
#pragma unroll
      for (int i = 0; i < RAW; ++i) {
        const int e = i * kThreads + threadIdx.x, r = e / (D / EL), c = e % (D / EL);
        const int64_t from = first_row(p, r / kPageSize);
        raw[i] = from < 0 ? make_uint4(0, 0, 0, 0)
                          : *reinterpret_cast<const uint4*>(
                                static_cast<const uint8_t*>(pool) +
                                (from + r % kPageSize * D) * KV::bytes + 16 * c);
      }
    };
    auto put = [&](float* dst, const uint4 (&raw)[RAW]) {
#pragma unroll
      for (int i = 0; i < RAW; ++i) {
        const int e = i * kThreads + threadIdx.x, r = e / (D / EL), c = e % (D / EL);
#pragma unroll
        for (int k = 0; k < EL / 4; ++k) {
          float o[4];
          RowLoad<KV, 4>::run(reinterpret_cast<const uint8_t*>(&raw[i]) + 4 * k * KV::bytes, o);
          *reinterpret_cast<float4*>(dst + r * LD + EL * c + 4 * k) =
              make_float4(o[0], o[1], o[2], o[3]);
        }
      }
    };
    uint4 kraw[RAW], vraw[RAW];
    __syncthreads();  // the previous run is done with the shared tiles
    Pages here = pages_of(run.tiles[run.i0]);
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
      if (r < run.rows) v = load4(static_cast<const float*>(a.q) + chunk_row(a, run, r) * D + 4 * c);
      *reinterpret_cast<float4*>(qs + r * LD + 4 * c) = v;
    }
    if constexpr (WIDEN) {
      put(ks, kraw);
      put(vs, vraw);
    }
    float m[4], l[4], slope[4];
    int pq[4];  // the rows' positions (no row: before every position)
    uint64_t acc[4][2 * NQ];  // pairs of dims
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int R = ty + 8 * i;
      m[i] = -INFINITY;
      l[i] = 0.f;
      pq[i] = R < run.rows ? run.req.base + run.t0 + R / run.heads : -1;
      slope[i] = a.slopes && R < run.rows
                     ? a.slopes[j * a.group + run.g0 + R % run.heads] * kLog2e
                     : 0.f;
#pragma unroll
      for (int k = 0; k < 2 * NQ; ++k) acc[i][k] = 0;
    }
    const ScoreForm form(a, KV::bytes == 1 ? a.k_scales[j] : 1.f);
    for (int i0 = 0; i0 < run.n; ++i0) {
      const int p0 = run.tiles[run.i0 + i0] * kTok;
      const bool more = i0 + 1 < run.n;
      const bool edge = chunk_edge(a, run, p0, kTok);  // not all positions seen
      uint64_t page_ok = 0;  // one bit per token
#pragma unroll
      for (int h = 0; h < kPages; ++h)
        if (here.row[h] >= 0) page_ok |= 0xffffull << (16 * h);
      if (here.bad && threadIdx.x == 0) atomicOr(a.err, PKV_DEVERR_BAD_PAGE);
      if (more) here = pages_of(run.tiles[run.i0 + i0 + 1]);
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
        if (edge || R >= run.rows) seen[i] &= chunk_seen(a, pq[i], p0);
        if (R >= run.rows) seen[i] = 0;
        float s[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          float even, odd;
          unpack2(s2[i][t], even, odd);
          s[t] = (seen[i] >> (tx + 16 * t)) & 1
                     ? form(even + odd, slope[i], pq[i] - p0 - tx - 16 * t)
                     : -INFINITY;
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
      if (edge || page_ok != ~0ull)
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
    const float vsc = KV::bytes == 1 ? a.v_scales[j] : 1.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = ty + 8 * i;
      if (r >= run.rows) continue;
      const size_t at = chunk_row(a, run, r);
      const size_t part = ((size_t)blockIdx.x * 2 + run.slot) * kRows + r;
      if (tx == 0) {
        if (!run.whole)
          *reinterpret_cast<float2*>(a.ws_ml + 2 * part) = make_float2(m[i], l[i]);
        else if (a.lse)
          a.lse[at] = l[i] != 0.f ? (m[i] + log2f(l[i])) * kLn2 : -INFINITY;
      }
#pragma unroll
      for (int k = 0; k < NQ; ++k) {
        float4 v;
        unpack2(acc[i][2 * k], v.x, v.y);
        unpack2(acc[i][2 * k + 1], v.z, v.w);
        if (!run.whole) {
          store4(a.ws_acc + part * D + 4 * tx + 64 * k,
                 make_float4(v.x * vsc, v.y * vsc, v.z * vsc, v.w * vsc));
          continue;
        }
        if (l[i] != 0.f)  // (a NaN sum stays NaN)
          v = make_float4(v.x / l[i] * vsc, v.y / l[i] * vsc, v.z / l[i] * vsc, v.w / l[i] * vsc);
        else
          v = make_float4(0.f, 0.f, 0.f, 0.f);
        store4(static_cast<float*>(a.out) + at * D + 4 * tx + 64 * k, v);
      }
    }
    if (!run.whole && run.slot == 1)
      record = ChunkRecord{(int)chunk_row(a, run, 0), run.heads, run.rows, run.shares};
  }
  if (threadIdx.x == 0) static_cast<ChunkRecord*>(a.ws_rec)[blockIdx.x] = record;
}

// ---- combine ---------------------------------------------------------------------------------

// Rows of the units that crossed shares: with partials c = 0 .. n-1 of a row in share order,
// M = max m_c, L = sum 2^(m_c - M) l_c, out = sum 2^(m_c - M) acc_c / L. A row of blocks for each share
// merges the unit that begins there and goes on, as its record says; a warp takes one row after the
// other, reading the (m, l) of up to 32 partials at once and the values of four together.
constexpr int kCombineThreads = 128;
constexpr int kCombineWarps = kCombineThreads / 32;

template <typename TQ, int D>
__global__ void __launch_bounds__(kCombineThreads) chunk_combine_kernel(const ChunkArgs a) {
  constexpr int DL = D / 32, CB = 4;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c0 = blockIdx.x;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const ChunkRecord rec = static_cast<const ChunkRecord*>(a.ws_rec)[c0];
  const int n = rec.shares + 1;
  for (int r = blockIdx.y * kCombineWarps + warp; r < rec.rows; r += gridDim.y * kCombineWarps) {
    auto part = [&](int c) {
      return ((size_t)(c0 + c) * 2 + (c == 0 ? 1 : 0)) * a.unit_rows + r;
    };
    float M = -INFINITY, L = 0.f, A[DL];
#pragma unroll
    for (int k = 0; k < DL; ++k) A[k] = 0.f;
    for (int q0 = 0; q0 < n; q0 += 32) {
      const int nc = min(32, n - q0);
      float2 ml = make_float2(-INFINITY, 0.f);
      if (lane < nc) ml = *reinterpret_cast<const float2*>(a.ws_ml + 2 * part(q0 + lane));
      float mr = ml.x;
#pragma unroll
      for (int o = 16; o >= 1; o /= 2) mr = fmaxf(mr, __shfl_xor_sync(0xffffffffu, mr, o));
      const float Mn = fmaxf(M, mr), Mu = Mn == -INFINITY ? 0.f : Mn;
      const float rescale = exp2f(M - Mu);
      // a partial that saw nothing weighs 0; a NaN sum stays one whatever its weight
      const float w = ml.x == -INFINITY ? 0.f : exp2f(ml.x - Mu);
      float lw = w != 0.f || ml.y != ml.y ? w * ml.y : 0.f;
#pragma unroll
      for (int o = 16; o >= 1; o /= 2) lw += __shfl_xor_sync(0xffffffffu, lw, o);
      L = fmaf(L, rescale, lw);
#pragma unroll
      for (int k = 0; k < DL; ++k) A[k] *= rescale;
      M = Mn;
      for (int q = 0; q < nc; q += CB) {
        float v[CB][DL];
#pragma unroll
        for (int u = 0; u < CB; ++u) {
          const float* src = a.ws_acc + part(q0 + min(q + u, nc - 1)) * D + lane * DL;
          if constexpr (DL == 4) {
            const float4 x = *reinterpret_cast<const float4*>(src);
            v[u][0] = x.x; v[u][1] = x.y; v[u][2] = x.z; v[u][3] = x.w;
          } else {
            const float2 x = *reinterpret_cast<const float2*>(src);
            v[u][0] = x.x; v[u][1] = x.y;
          }
        }
#pragma unroll
        for (int u = 0; u < CB; ++u) {
          const float wu = __shfl_sync(0xffffffffu, w, (q + u) & 31);
          if (q + u < nc && wu != 0.f) {
#pragma unroll
            for (int k = 0; k < DL; ++k) A[k] = fmaf(wu, v[u][k], A[k]);
          }
        }
      }
    }
    const int t = r / rec.heads;
    const size_t at = (size_t)rec.row0 + (size_t)t * a.h_q + (r - t * rec.heads);
    TQ* o = static_cast<TQ*>(a.out) + at * D + lane * DL;
#pragma unroll
    for (int k = 0; k < DL; ++k) store_from_float(o, k, L != 0.f ? A[k] / L : 0.f);
    if (a.lse && lane == 0) a.lse[at] = L != 0.f ? (M + log2f(L)) * kLn2 : -INFINITY;
  }
}

template <typename KV, int D>
cudaError_t simt_go(const ChunkArgs& a, cudaStream_t s) {
  static std::atomic<unsigned long long> attr_done{0};  // one bit per device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !((attr_done.load() >> dev) & 1ull)) {
    e = cudaFuncSetAttribute(chunk_simt_kernel<KV, D>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, SimtShape<D>::SMEM);
    if (e != cudaSuccess) return e;
    if (dev < 64) attr_done.fetch_or(1ull << dev);
  }
  chunk_simt_kernel<KV, D><<<a.ctas, kThreads, SimtShape<D>::SMEM, s>>>(a);
  return cudaGetLastError();
}

template <int D>
cudaError_t simt_types(const ChunkArgs& a, int kv_dtype, cudaStream_t s) {
  if (kv_dtype == PKV_F32) return simt_go<F32, D>(a, s);
  if (kv_dtype == PKV_FP8_E4M3) return simt_go<FP8, D>(a, s);
  return simt_go<INT8, D>(a, s);
}

template <typename TQ, int D>
cudaError_t launch_combine(const ChunkArgs& a, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  // rows of a unit over several blocks: up to four rows a warp
  cfg.gridDim = dim3(a.ctas, (a.unit_rows + 4 * kCombineWarps - 1) / (4 * kCombineWarps));
  cfg.blockDim = dim3(kCombineThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, chunk_combine_kernel<TQ, D>, a);
}

}  // namespace

cudaError_t launch_chunk_simt(const ChunkArgs& a, int kv_dtype, int head_dim, cudaStream_t s) {
  return head_dim == 64 ? simt_types<64>(a, kv_dtype, s) : simt_types<128>(a, kv_dtype, s);
}

cudaError_t launch_chunk_combine(const ChunkArgs& a, int q_dtype, int head_dim, cudaStream_t s) {
  if (q_dtype == PKV_BF16)
    return head_dim == 64 ? launch_combine<__nv_bfloat16, 64>(a, s)
                          : launch_combine<__nv_bfloat16, 128>(a, s);
  return head_dim == 64 ? launch_combine<float, 64>(a, s) : launch_combine<float, 128>(a, s);
}

}  // namespace pkv
