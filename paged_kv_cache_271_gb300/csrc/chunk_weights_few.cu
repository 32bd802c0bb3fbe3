// Sums of attention weights for calls of few rows a request (decode steps), bf16 queries over a bf16, FP8 or
// INT8 cache; the mathematics is that of chunk_weights.cu.
//
// Such a call is bound by reading K once: 64 requests' rows are 149 MB of FP8 for some thousand operations a
// row. So K goes from memory straight into registers, in the form the MMA wants: a dot product does not
// mind the order of its terms, so each lane takes 16 consecutive bytes of a row where the MMA
// (m16n8k16: 16 positions x 8 rows) would have it take 2 and 2 of distant ones, and the queries are
// taken in the same order. A warp has a page (16 positions) and the next one in registers, no shared
// memory, no barriers, and 12 to 16 warps on an SM keep 50 to 100 KB of reads under way (through the
// rings of the tcgen05 kernel the same call, 64 requests of 512 .. 4096 FP8 tokens and 8 KV heads, takes
// 142 us instead of 39, or 4.1 TB/s: a step of 4 rows there costs as much as one of 128).
//
// The pages of all requests and KV heads, in order, form one stream, and each warp takes an equal
// contiguous share of it, whole pages: no sum is made in parts, so equal inputs give equal results.
// Rows beyond 8 NB take another pass over the warp's pages of that KV head, which adds to the sums. From three
// passes on that is Kahan's summation (over 32 pages at a time): a request of many rows may be among many of
// one, and its sums are to be as good as in a call of its own. (In a body of its own: with both in one, a
// decode step over FP8 takes 45 us instead of 40; with it from two passes on, 16 rows of each 74, not 70.)
#include <math.h>

#include <type_traits>

#include "chunk_score.cuh"
#include "paged_decode_mma.cuh"
#include "pkv_device.cuh"
#include "pkv_internal.h"
#include "tcgen05.cuh"
#include "weigh_plan.cuh"

namespace pkv {

namespace {

constexpr int kThreads = 128, kWarps = kThreads / 32;
constexpr int kPassPages = 32;  // pages that several passes go over before the next ones

// d += a b, 16 x 8 x 16: a is K (row gid: a0, a2; row gid + 8: a1, a3), b queries.
template <bool F16>
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                    uint32_t b0, uint32_t b1) {
  if constexpr (F16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint4 stream128(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

// A request's length in the stream: its pages, each as long as the passes over it.
template <int NB>
__device__ __forceinline__ int few_passes(const ChunkArgs& a, const WeighReq& w) {
  return max(1, ((w.r.n - w.from) * a.group + 8 * NB - 1) / (8 * NB));
}

struct FewShare {
  int b, page, left;  // first request and page of it (KV heads in turn); length left
};

template <typename KV, int D, int NB>
__global__ void __launch_bounds__(kThreads, NB == 1 ? 4 : 3) weights_few_kernel(const ChunkArgs a) {
  constexpr bool W8 = KV::bytes == 1;
  constexpr int CH = D * KV::bytes / 64;  // 16-byte chunks of a lane's part of a row
  constexpr int KS = D / 16;              // MMA steps along the dims
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, gid = lane >> 2, tig = lane & 3;
  __shared__ int scratch[32];
  __shared__ FewShare shares[kWarps];
  __shared__ float lost[kWarps][kPassPages][kPageSize];  // what a sum of three passes or more has lost
  // ---- this warp's share ----
  {
    const int per = (a.batch + kThreads - 1) / kThreads;
    const int b0 = min(a.batch, (int)threadIdx.x * per), b1 = min(a.batch, b0 + per);
    int mine = 0, err = 0;
    for (int b = b0; b < b1; ++b) {
      const WeighReq w = weigh_request(a, b);
      err |= w.r.err;
      mine += w.items * few_passes<NB>(a, w) * a.h_kv;
    }
    if (err && blockIdx.x == 0) atomicOr(a.err, err);
    if (threadIdx.x < kWarps) shares[threadIdx.x].left = 0;
    if (chunk_rows_overlap(a, err & PKV_DEVERR_BAD_CHUNK)) return;
    int below, total;
    block_scan<kThreads>(mine, scratch, below, total);
    const int warps = a.ctas * kWarps;
    const int share = (int)(((unsigned)total + warps - 1) / (unsigned)warps);
    for (int x = 0; x < kWarps; ++x) {
      const long long start = ((long long)blockIdx.x * kWarps + x) * share;
      if (start < below || start >= (long long)below + mine) continue;
      int at = below, b = b0;
      WeighReq w = weigh_request(a, b);
      while (b < b1 - 1 && start >= at + w.items * few_passes<NB>(a, w) * a.h_kv) {
        at += w.items * few_passes<NB>(a, w) * a.h_kv;
        w = weigh_request(a, ++b);
      }
      const int cost = few_passes<NB>(a, w), page = ((int)start - at + cost - 1) / cost;
      shares[x].b = b;
      shares[x].page = page;  // (the first that begins in the share)
      shares[x].left = min(share, total - (int)start) - (at + page * cost - (int)start);
    }
    __syncthreads();
  }
  int b = shares[warp].b, page = shares[warp].page, left = shares[warp].left;
  const float cap_top = a.softcap * kLog2e, cap_in = a.softcap > 0.f ? kLn2 / a.softcap : 0.f;
  for (; left > 0 && b < a.batch; ++b, page = 0) {
    const WeighReq w = weigh_request(a, b);
    const int passes = few_passes<NB>(a, w);
    const int ctx = w.r.base + w.r.n, rows = (w.r.n - w.from) * a.group, first = w.r.base + w.from;
    const int32_t* table = a.block_tables + (size_t)b * a.max_pages;
    while (left > 0 && page < w.items * a.h_kv) {
      const int j = page / w.items, lo = page - j * w.items;  // this head's pages lo .. hi - 1
      const int most = (left + passes - 1) / passes;
      const int hi = (int)min((long long)w.items, (long long)lo + (passes > 2 ? min(most, kPassPages) : most));
      const float sc = a.scale * kLog2e * (W8 && rows > 0 ? a.k_scales[j] : 1.f);
      float* const out = a.weights_out + ((int64_t)b * a.h_kv + j) * a.width;
      const float* const before = a.add_to ? a.add_to + ((int64_t)b * a.h_kv + j) * a.width : nullptr;
      for (int pass = 0; pass < passes; ++pass) {
        // ---- queries: lane (gid, tig) has its dims of row gid of every block of 8 rows ----
        uint32_t q[NB][KS][2];
        float factor[NB][2], neg_lse[NB][2], slope[NB][2];
        int pos[NB][2];  // of columns 2 tig and 2 tig + 1 (before every position where there is no row)
#pragma unroll
        for (int n = 0; n < NB; ++n) {
          const int row = (pass * NB + n) * 8;
          auto place = [&](int r) {  // of row r in q and lse
            const int t = r / a.group;
            return (size_t)(w.r.q0 + w.from + t) * a.h_q + j * a.group + (r - t * a.group);
          };
          const bool there = row + gid < rows;
          const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(a.q) +
                                     (there ? place(row + gid) : 0) * D;
          uint32_t x[D / 8];  // pairs in the MMAs' order
          constexpr int RUN = 16 / KV::bytes;  // dims of a 16-byte chunk of K
#pragma unroll
          for (int i = 0; i < CH; ++i)
#pragma unroll
            for (int h = 0; h < RUN / 8; ++h) {
              const uint4 v = there ? *reinterpret_cast<const uint4*>(src + (4 * i + tig) * RUN + 8 * h)
                                    : make_uint4(0, 0, 0, 0);
              uint32_t* const y = x + (i * (RUN / 8) + h) * 4;
              y[0] = v.x; y[1] = v.y; y[2] = v.z; y[3] = v.w;
            }
          float mine = sc;  // of row gid
          if constexpr (W8) {
            uint32_t lo_max = 0, hi_max = 0;
#pragma unroll
            for (int i = 0; i < D / 8; ++i) {
              lo_max = max(lo_max, x[i] & 0x7fffu);
              hi_max = max(hi_max, x[i] & 0x7fff0000u);
            }
            uint32_t mx = max(lo_max, hi_max >> 16);
            mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
            mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
            // f16, scaled by 2^e that puts the row's largest value in f16's top binade (as in the tcgen05
            // kernels, the K scale's sign or NaN goes with the queries)
            const int ex = mx >> 7, e = mx != 0 && ex < 255 ? min(126, max(-126, 141 - ex)) : 0;
            const float two_e = __int_as_float((127 + e) << 23);
            const float up = sc < 0.f ? -two_e : sc == sc ? two_e : sc;
#pragma unroll
            for (int i = 0; i < D / 8; ++i) x[i] = pack_f16(bf16lo(x[i]) * up, bf16hi(x[i]) * up);
            mine = fmaxf(fabsf(sc) * __int_as_float((127 - e) << 23), 0x1p-126f);
          }
#pragma unroll
          for (int k = 0; k < KS; ++k) {
            q[n][k][0] = x[2 * k];
            q[n][k][1] = x[2 * k + 1];
          }
#pragma unroll
          for (int m = 0; m < 2; ++m) {
            const int r = row + 2 * tig + m;
            factor[n][m] = __shfl_sync(0xffffffffu, mine, 4 * (2 * tig + m));
            const float lse = r < rows ? a.lse[place(r)] : -INFINITY;
            neg_lse[n][m] = lse == -INFINITY ? -INFINITY : -lse * kLog2e;  // (gives nothing)
            pos[n][m] = r < rows ? first + r / a.group : -1;
            slope[n][m] = a.slopes && r < rows ? a.slopes[j * a.group + r % a.group] * kLog2e : 0.f;
          }
        }
        const int pos_first = first + pass * NB * 8 / a.group;
        const int pos_last = first + (min(rows, (pass + 1) * NB * 8) - 1) / a.group;
        // ---- pages ----
        int ids = -1;
        auto id_of = [&](int pg) {  // -1: no row sees it; -2: it has no id
          if ((pg - lo) % 32 == 0) {
            const int mine = pg + lane, p0 = mine * kPageSize;
            // (a page outside every row's window may have been given back: it is not read)
            const bool wanted = rows > 0 && mine < hi && p0 <= pos_last &&
                                (a.window <= 0 || p0 < a.sink || p0 + kPageSize > first + 1 - a.window);
            ids = -1;
            if (wanted) {
              ids = table[mine];
              if (ids < 0 || ids >= a.num_pages) ids = -2;
            }
            if (ids == -2) atomicOr(a.err, PKV_DEVERR_BAD_PAGE);
          }
          return __shfl_sync(0xffffffffu, ids, (pg - lo) & 31);
        };
        uint4 kv[2][2][CH];  // [this page, the next][row gid, gid + 8]
        auto fetch = [&](int which, int id) {
          if (id < 0) return;
          const uint8_t* src = static_cast<const uint8_t*>(a.k_cache) +
                               (((int64_t)id * a.h_kv + j) * kPageSize + gid) * D * KV::bytes + 16 * tig;
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < CH; ++i) kv[which][h][i] = stream128(src + h * 8 * D * KV::bytes + 64 * i);
        };
        int id = id_of(lo), id_next = -1;
        fetch(0, id);
        auto one = [&](auto several, int which, int pg) {
          const int p0 = pg * kPageSize;
          id_next = pg + 1 < hi ? id_of(pg + 1) : -1;
          fetch(1 - which, id_next);
          // lane tig 0 writes position gid, 1 position gid + 8
          const int at = p0 + gid + 8 * tig;
          const bool writes = tig < 2 && at < ctx;
          const float base = !writes ? 0.f : pass > 0 ? out[at] : before ? before[at] : 0.f;
          float total[2] = {0.f, 0.f};
          if (id >= 0) {
            const bool edge = p0 + kPageSize - 1 > pos_first ||
                              (a.window > 0 && p0 + kPageSize > a.sink && p0 < pos_last + 1 - a.window);
#pragma unroll
            for (int n = 0; n < NB; ++n) {
              float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
              for (int i = 0; i < CH; ++i) {
                const uint4 r0 = kv[which][0][i], r8 = kv[which][1][i];
                if constexpr (W8) {
                  const uint32_t w0[4] = {r0.x, r0.y, r0.z, r0.w}, w8[4] = {r8.x, r8.y, r8.z, r8.w};
#pragma unroll
                  for (int k = 0; k < 4; ++k) {
                    uint32_t a0, a2, a1, a3;
                    widen4<KV>(w0[k], a0, a2);
                    widen4<KV>(w8[k], a1, a3);
                    mma<true>(d, a0, a1, a2, a3, q[n][4 * i + k][0], q[n][4 * i + k][1]);
                  }
                } else {
                  mma<false>(d, r0.x, r8.x, r0.y, r8.y, q[n][2 * i][0], q[n][2 * i][1]);
                  mma<false>(d, r0.z, r8.z, r0.w, r8.w, q[n][2 * i + 1][0], q[n][2 * i + 1][1]);
                }
              }
#pragma unroll
              for (int m = 0; m < 4; ++m) {  // (row gid + 8 (m / 2), column 2 tig + m % 2)
                const int c = m & 1, p = p0 + gid + 8 * (m >> 1);
                float s = d[m] * factor[n][c];
                if (a.softcap > 0.f) s = cap_top * tanhf(s * cap_in);
                if (a.slopes) s = fmaf(slope[n][c], (float)(p - pos[n][c]), s);
                float e = ex2_approx(s + neg_lse[n][c]);
                if (!(a.softcap > 0.f) && !a.slopes) e = ex2_approx(fmaf(d[m], factor[n][c], neg_lse[n][c]));
                const int behind = pos[n][c] - p;
                const bool hidden =
                    edge && (behind < 0 || (a.window > 0 && behind >= a.window && p >= a.sink));
                total[m >> 1] += hidden || neg_lse[n][c] == -INFINITY ? 0.f : e;
              }
            }
          }
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            total[h] += __shfl_xor_sync(0xffffffffu, total[h], 1);
            total[h] += __shfl_xor_sync(0xffffffffu, total[h], 2);
          }
          if constexpr (decltype(several)::value) {
            if (writes) {
              float* const gone = &lost[warp][pg - lo][gid + 8 * tig];
              float add = tig == 0 ? total[0] : total[1];
              if (pass > 0) add -= *gone;
              const float sum = base + add;
              const float left_out = (sum - base) - add;
              *gone = fabsf(left_out) < INFINITY ? left_out : 0.f;  // (infinite sums stay that)
              out[at] = sum;
            }
          } else {
            if (writes) out[at] = base + (tig == 0 ? total[0] : total[1]);
          }
          id = id_next;
        };
        auto walk = [&](auto several) {
          for (int pg = lo; pg < hi; pg += 2) {
            one(several, 0, pg);
            if (pg + 1 < hi) one(several, 1, pg + 1);
          }
        };
        if (passes > 2)
          walk(std::true_type{});
        else
          walk(std::false_type{});
      }
      left -= (hi - lo) * passes;
      page += hi - lo;
    }
  }
}

template <typename KV, int D, int NB>
cudaError_t go(const ChunkArgs& a, cudaStream_t s) {
  weights_few_kernel<KV, D, NB><<<a.ctas, kThreads, 0, s>>>(a);
  return cudaGetLastError();
}

template <int D, int NB>
cudaError_t types(const ChunkArgs& a, int kv_dtype, cudaStream_t s) {
  if constexpr (NB == 1)
    if (kv_dtype == PKV_BF16) return go<BF16, D, NB>(a, s);
  if (kv_dtype == PKV_FP8_E4M3) return go<FP8, D, NB>(a, s);
  return go<INT8, D, NB>(a, s);
}

}  // namespace

cudaError_t launch_chunk_weights_few(const ChunkArgs& a, int kv_dtype, int head_dim, int blocks,
                                     cudaStream_t s) {
  if (blocks == 1 || kv_dtype == PKV_BF16)
    return head_dim == 64 ? types<64, 1>(a, kv_dtype, s) : types<128, 1>(a, kv_dtype, s);
  return head_dim == 64 ? types<64, 4>(a, kv_dtype, s) : types<128, 4>(a, kv_dtype, s);
}

}  // namespace pkv
