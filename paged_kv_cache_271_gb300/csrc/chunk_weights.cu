// Sums of the attention weights that the rows of a chunk give to each cached position, on CUDA cores:
//   out[b][j][p] = add_to[b][j][p] + sum over counted rows t and query heads h of group j that see p of
//                  e^{s_thp - lse_th},
// with the scores s of the chunk attention and the lse it left.
//
// For fp32 queries, on CUDA cores, and the combine of a split call of any type. A block takes tiles of 64
// positions of one KV head (weigh_plan.cuh): K of the tile stays in shared memory as fp32, the rows come
// by 32, a thread computes 4 rows x 4 positions of scores. Sums over thousands of rows are compensated
// (Kahan's summation), so that they are good to fp32.
#include <math.h>

#include <atomic>

#include "chunk_plan.cuh"
#include "chunk_score.cuh"
#include "pkv_device.cuh"
#include "pkv_internal.h"
#include "tcgen05.cuh"
#include "weigh_plan.cuh"

namespace pkv {

namespace {

constexpr int kThreads = 128;
constexpr int kRows = kChunkSimtRows, kTok = kChunkSimtTokens;

template <int D>
struct WeighShape {
  static constexpr int LD = D + 4;
  static constexpr int SMEM = 4 * ((kRows + kTok) * LD + 8 * kTok + kRows);
};

template <typename KV, int D>
__global__ void __launch_bounds__(kThreads) weights_simt_kernel(const ChunkArgs a) {
  constexpr int LD = WeighShape<D>::LD;
  extern __shared__ float4 smem4[];
  float* qs = reinterpret_cast<float*>(smem4);
  float* ks = qs + kRows * LD;
  float* sums = ks + kTok * LD;        // [8][64]
  float* lse2 = sums + 8 * kTok;       // [32] the rows' lse in the log2 domain
  __shared__ int scratch[32];
  __shared__ WeighShare share;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  weigh_share<kThreads>(a, scratch, &share);
  WeighWalk walk(a, share);
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;  // positions tx + 16 m, rows ty + 8 i
  WeighRecord record{0, 0, 0, 0};
  WeighRun it;
  while (walk.next(a, it)) {
    const ChunkReq& req = it.req;
    const int j = it.j, p0 = it.item * kTok, ctx = req.base + req.n, rows = it.rows;
    const int32_t* table = a.block_tables + (size_t)it.b * a.max_pages;
    uint64_t page_ok = 0;
    __syncthreads();  // the last item's tile and sums are used up
    if (rows > 0) {
      constexpr int EL = 16 / KV::bytes;
      bool bad = false;
#pragma unroll
      for (int h = 0; h < kTok / kPageSize; ++h) {
        const int q0 = p0 + h * kPageSize;  // (pages that no row sees are not read)
        const bool wanted = q0 < ctx && (a.window <= 0 || q0 < a.sink ||
                                         q0 + kPageSize > req.base + it.t0 + 1 - a.window);
        const int id = wanted ? table[q0 / kPageSize] : -1;
        const bool there = id >= 0 && id < a.num_pages;
        bad |= wanted && !there;
        if (there) page_ok |= 0xffffull << (16 * h);
        const uint8_t* src = static_cast<const uint8_t*>(a.k_cache) +
                             ((int64_t)(there ? id : 0) * a.h_kv + j) * kPageSize * D * KV::bytes;
        for (int e = threadIdx.x; e < kPageSize * D / EL; e += kThreads) {
          const int r = e / (D / EL), c = e % (D / EL);
          const uint4 raw = there ? *reinterpret_cast<const uint4*>(src + 16 * e)
                                  : make_uint4(0, 0, 0, 0);
#pragma unroll
          for (int k = 0; k < EL / 4; ++k) {
            float o[4];
            RowLoad<KV, 4>::run(reinterpret_cast<const uint8_t*>(&raw) + 4 * k * KV::bytes, o);
            *reinterpret_cast<float4*>(ks + (h * kPageSize + r) * LD + EL * c + 4 * k) =
                make_float4(o[0], o[1], o[2], o[3]);
          }
        }
      }
      if (bad && threadIdx.x == 0) atomicOr(a.err, PKV_DEVERR_BAD_PAGE);
    }
    // (a call without rows, which carries the sums over, may come without scales)
    const ScoreForm form(a, KV::bytes == 1 && rows > 0 ? a.k_scales[j] : 1.f);
    float total[4] = {0.f, 0.f, 0.f, 0.f}, lost[4] = {0.f, 0.f, 0.f, 0.f};
    for (int r0 = it.s0 * kRows; r0 < min(rows, (it.s0 + it.n) * kRows); r0 += kRows) {
      __syncthreads();  // the last rows are used up
      for (int e = threadIdx.x; e < kRows * (D / 4); e += kThreads) {
        const int r = e / (D / 4), c = e % (D / 4);
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (r0 + r < rows) {
          const int t = (r0 + r) / a.group, g = (r0 + r) - t * a.group;
          const size_t at = (size_t)(req.q0 + it.t0 + t) * a.h_q + j * a.group + g;
          v = load4(static_cast<const float*>(a.q) + at * D + 4 * c);
          if (c == 0) lse2[r] = a.lse[at] * kLog2e;
        }
        *reinterpret_cast<float4*>(qs + r * LD + 4 * c) = v;
      }
      __syncthreads();
      uint64_t s2[4][4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) s2[i][k] = 0;
#pragma unroll 4
      for (int d = 0; d < D; d += 4) {
        ulonglong2 k[4];
#pragma unroll
        for (int t = 0; t < 4; ++t)
          k[t] = *reinterpret_cast<const ulonglong2*>(ks + (tx + 16 * t) * LD + d);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const ulonglong2 q = *reinterpret_cast<const ulonglong2*>(qs + (ty + 8 * i) * LD + d);
#pragma unroll
          for (int t = 0; t < 4; ++t) s2[i][t] = fma2(q.y, k[t].y, fma2(q.x, k[t].x, s2[i][t]));
        }
      }
      float add[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int R = ty + 8 * i;
        if (r0 + R >= rows) continue;
        const int t = (r0 + R) / a.group, g = (r0 + R) - t * a.group;
        const int pq = req.base + it.t0 + t;
        const uint64_t seen = chunk_seen(a, pq, p0) & page_ok;
        const float slope = a.slopes ? a.slopes[j * a.group + g] * kLog2e : 0.f;
        const float l2 = lse2[R];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if (!((seen >> (tx + 16 * k)) & 1) || l2 == -INFINITY) continue;
          float even, odd;
          unpack2(s2[i][k], even, odd);
          add[k] += exp2f(form(even + odd, slope, pq - p0 - tx - 16 * k) - l2);
        }
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float y = add[k] - lost[k], z = total[k] + y;
        lost[k] = (z - total[k]) - y;
        total[k] = z;
      }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) sums[ty * kTok + tx + 16 * k] = total[k];
    __syncthreads();
    if (threadIdx.x < kTok && p0 + (int)threadIdx.x < ctx) {
      float x = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) x += sums[i * kTok + threadIdx.x];
      const int64_t at = ((int64_t)it.b * a.h_kv + j) * a.width + p0 + threadIdx.x;
      if (it.whole)
        a.weights_out[at] = (a.add_to ? a.add_to[at] : 0.f) + x;
      else
        a.ws_acc[((size_t)blockIdx.x * 2 + it.slot) * kTok + threadIdx.x] = x;
    }
    if (!it.whole && it.slot == 1)
      record = WeighRecord{it.b * a.h_kv + j, p0, min(kTok, ctx - p0), it.shares};
  }
  if (threadIdx.x == 0) static_cast<WeighRecord*>(a.ws_rec)[blockIdx.x] = record;
}

// Items that crossed shares: a block for each share adds the partials of the item that begins there.
__global__ void weights_combine_kernel(const ChunkArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const WeighRecord rec = static_cast<const WeighRecord*>(a.ws_rec)[blockIdx.x];
  if (rec.shares == 0 || (int)threadIdx.x >= rec.n) return;
  const int T = a.tile_tokens;
  float x = a.ws_acc[((size_t)blockIdx.x * 2 + 1) * T + threadIdx.x];
  for (int c = 1; c <= rec.shares; ++c)
    x += a.ws_acc[((size_t)(blockIdx.x + c) * 2) * T + threadIdx.x];
  const int64_t at = (int64_t)rec.row * a.width + rec.p0 + threadIdx.x;
  a.weights_out[at] = (a.add_to ? a.add_to[at] : 0.f) + x;
}

template <typename KV, int D>
cudaError_t go(const ChunkArgs& a, cudaStream_t s) {
  static std::atomic<unsigned long long> attr_done{0};  // one bit per device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !((attr_done.load() >> dev) & 1ull)) {
    e = cudaFuncSetAttribute(weights_simt_kernel<KV, D>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, WeighShape<D>::SMEM);
    if (e != cudaSuccess) return e;
    if (dev < 64) attr_done.fetch_or(1ull << dev);
  }
  weights_simt_kernel<KV, D><<<a.ctas, kThreads, WeighShape<D>::SMEM, s>>>(a);
  return cudaGetLastError();
}

template <int D>
cudaError_t types(const ChunkArgs& a, int kv_dtype, cudaStream_t s) {
  if (kv_dtype == PKV_F32) return go<F32, D>(a, s);
  if (kv_dtype == PKV_FP8_E4M3) return go<FP8, D>(a, s);
  return go<INT8, D>(a, s);
}

}  // namespace

cudaError_t launch_chunk_weights_simt(const ChunkArgs& a, int kv_dtype, int head_dim,
                                      cudaStream_t s) {
  return head_dim == 64 ? types<64>(a, kv_dtype, s) : types<128>(a, kv_dtype, s);
}

cudaError_t launch_chunk_weights_combine(const ChunkArgs& a, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.ctas);
  cfg.blockDim = dim3(a.tile_tokens);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, weights_combine_kernel, a);
}

}  // namespace pkv
