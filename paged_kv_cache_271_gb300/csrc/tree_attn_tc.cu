// Tree attention on the fifth-generation tensor cores (tcgen05), bf16 queries over a bf16, FP8 or
// INT8 cache.
//
// The mathematics is that of tree_attn.cu; the work is cut as tree_plan.cuh says, in units of up to
// 256 (node, query head) rows of one KV head and tiles of 64 tokens, one persistent CTA per SM. A
// verification step does 4 rows x D operations per cached K/V row of 2 D values, so up to about 256
// rows it is bound by reading the cache once; the work here is arranged so that everything else
// hides behind those reads:
//
//  * a copy warp streams tiles of K and V into a ring of shared-memory stages, running ahead across
//    units; a bf16 tile arrives by TMA in the 128-byte-swizzled form the MMAs read. The codes of an
//    8-bit tile arrive by bulk copies and four converter warps widen them to f16 (exactly) in that
//    form; the K scale goes into the score factor and the V scale into the output;
//  * an MMA warp (one lane) issues S = Q K^T (M = 128 rows, N = 64 tokens) and O += P V (N = D),
//    with Q and P as A operands in tensor memory and all accumulators there;
//  * two groups of four softmax warps, thread r of a group owning row r. Units of up to 128 rows:
//    the groups take alternate tiles, each with a maximum, a sum and an O of its own, merged at the
//    unit's end (three S buffers); larger units: group g takes rows 128 g .. of every tile (two S
//    buffers), so the cache is still read once. Either way one group's softmax overlaps the other's
//    MMAs;
//  * O is rescaled only when a row's maximum grows by more than 2^8 (P <= 2^8 until then): the final
//    (max, sum, O) is exact whatever maximum it was accumulated against.
//
// P is rounded to the MMA's input type (bf16 for a bf16 cache, f16 otherwise), the only rounding
// before the output's; scores, maxima and sums are fp32. For 8-bit caches a query row is scaled by
// a power of two that puts its largest value in f16's top binade, undone in its score factor.
//
// Tiles with unseen positions (the drafted nodes, the end of the context, bad pages) mask scores
// by the row's 64 mask bits, and their V rows are mended in shared memory before the MMA reads them:
// rows outside the context or on a bad page become 0, and a drafted row's infinite or NaN values,
// which 0 P would still spread to rows that do not see the node, become 0 there and are added to
// the rows that do see it at the unit's end.
//
// Every wait is bounded (PKV_DEVERR_TIMEOUT); the tensor memory is freed on every path.
#include <atomic>
#include <cuda.h>
#include <math.h>

#include "paged_decode_mma.cuh"
#include "pkv_device.cuh"
#include "pkv_internal.h"
#include "tcgen05.cuh"
#include "tree_plan.cuh"

namespace pkv {

namespace {

constexpr int kTok = kTreeTcTokens;        // tokens of a tile
constexpr int kPages = kTok / kPageSize;   // pages of a tile
constexpr int kGroupThreads = 128;         // a softmax group: one row per thread
constexpr int kSoftThreads = 2 * kGroupThreads;
constexpr int kMmaWarp = kSoftThreads / 32;
constexpr int kCopyWarp = kMmaWarp + 1;
constexpr int kConvWarp = kCopyWarp + 1;   // first of four (8-bit caches)
constexpr int kConvThreads = 128;
constexpr int kSBufs = 3;
// tensor memory columns: O of group 0 and 1, Q of the rows 0 .. 127 and 128 .. 255, S (then P)
// buffers; the third S buffer shares the second Q's columns (units of up to 128 rows have one Q)
constexpr uint32_t kColO = 0, kColQ = 256, kColS = 384, kColS2 = 320;
constexpr uint32_t kTmemCols = 512;
constexpr float kLazyLog2 = 8.f;
static_assert(2 * kGroupThreads == kTreeTcRows, "a unit is two groups' rows");

template <typename KV, int D>
struct TcShape {
  static constexpr bool W8 = KV::bytes == 1;
  static constexpr int THREADS = 32 * (W8 ? kConvWarp + kConvThreads / 32 : kConvWarp);
  static constexpr int TILE = kTok * D * 2;       // K (or V) of a tile in MMA form
  static constexpr int STAGE = 2 * TILE;
  static constexpr int RAW_TILE = kTok * D;       // 8-bit codes
  static constexpr int RAW_STAGE = 2 * RAW_TILE;
  // a ring of 192 KB; 8-bit caches: half of it raw codes, half MMA form
  static constexpr int NS = (W8 ? 96 : 192) * 1024 / STAGE;
  static constexpr int NR = W8 ? 96 * 1024 / RAW_STAGE : 0;
  static constexpr int OFF_RAW = NS * STAGE;
  static constexpr int OFF_ML = OFF_RAW + NR * RAW_STAGE;   // [2][128] (max, sum)
  static constexpr int OFF_BAR = OFF_ML + 2 * kGroupThreads * 8;
  static constexpr int BARS = 2 * NS + 2 * NR + 3 * kSBufs + 2;
  static constexpr int OFF_MISC = OFF_BAR + 8 * BARS;       // masks, bad nodes, TMEM address
  static constexpr uint32_t IDESC_S = tc_idesc(128, kTok, false, W8);
  static constexpr uint32_t IDESC_PV = tc_idesc(128, D, true, W8);
  static constexpr int SMEM = 1024 + OFF_MISC + 4 * (NS + NR + 2 * 8 + 1) + 16;
  static_assert(SMEM <= 227 * 1024 && SMEM > 114 * 1024, "one CTA per SM");
};

__device__ __forceinline__ uint32_t s_col(int buf) {
  return buf == 2 ? kColS2 : kColS + 64 * buf;
}

// Steps of a unit in order: with up to 128 rows step u is tile u, otherwise tile u / 2 for rows
// 128 (u % 2) ... Group u % 2 takes it; it uses S buffer u % bufs.
struct Steps {
  int n, bufs;
  bool wide;
  __device__ __forceinline__ explicit Steps(const TreeRun& r)
      : n(r.rows > kGroupThreads ? 2 * r.n : r.n),
        bufs(r.rows > kGroupThreads ? 2 : kSBufs),
        wide(r.rows > kGroupThreads) {}
  __device__ __forceinline__ int tile(int u) const { return wide ? u >> 1 : u; }
  __device__ __forceinline__ int buf(int u) const { return wide ? u & 1 : u % 3; }
  // parity of the buffer's barriers in step u; `ph` holds each buffer's parity at the unit's start
  __device__ __forceinline__ uint32_t parity(uint32_t ph, int u) const {
    return ((ph >> buf(u)) ^ (wide ? u >> 1 : u / 3)) & 1u;
  }
  __device__ __forceinline__ uint32_t after(uint32_t ph) const {
#pragma unroll
    for (int b = 0; b < kSBufs; ++b) {
      if (b >= bufs) break;
      const int uses = wide ? n / 2 : (n + 2 - b) / 3;
      ph ^= (uint32_t)(uses & 1) << b;
    }
    return ph;
  }
};

template <bool F16>
__device__ __forceinline__ uint32_t pack_p(float a, float b) {
  return F16 ? pack_f16(a, b) : pack_bf16(a, b);
}

// Whether a 16-bit value (bits of the MMA input type) is infinite or NaN.
template <bool F16>
__device__ __forceinline__ bool not_finite(uint32_t h) {
  constexpr uint32_t E = F16 ? 0x7c00u : 0x7f80u;
  return (h & E) == E;
}

template <typename KV, int D>
__global__ void __launch_bounds__(TcShape<KV, D>::THREADS, 1) tree_tc_kernel(
    const TreeArgs a, const __grid_constant__ CUtensorMap tm_k,
    const __grid_constant__ CUtensorMap tm_v) {
  using S = TcShape<KV, D>;
  constexpr bool W8 = S::W8;
  constexpr int NS = S::NS, NR = S::NR;
  constexpr int PAGE_MMA = kPageSize * D * 2;  // V bytes of a page in MMA form
  constexpr int PAGE_RAW = kPageSize * D;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t ring = smem_u32(smem);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + S::OFF_BAR);  // [NS] tile in MMA form
  uint64_t* freed = full + NS;                                       // [NS] its P V done
  uint64_t* raw_full = freed + NS;                                   // [NR] codes arrived
  uint64_t* raw_freed = raw_full + NR;                               // [NR] codes widened
  uint64_t* s_done = raw_freed + NR;                                 // [3] S in its buffer
  uint64_t* p_ready = s_done + kSBufs;                               // [3] P in its buffer
  uint64_t* pv_done = p_ready + kSBufs;                              // [3] that P V complete
  uint64_t* q_ready = pv_done + kSBufs;  // Q of a unit stored, the last unit's O read
  uint64_t* mma_idle = q_ready + 1;
  int* page_mask = reinterpret_cast<int*>(smem + S::OFF_MISC);       // [NS] good pages of the tile
  int* raw_mask = page_mask + NS;                                    // [NR]
  uint32_t* bad_nodes = reinterpret_cast<uint32_t*>(raw_mask + NR);  // [2][8] V row not finite
  uint32_t* s_taddr = bad_nodes + 16;
  float2* ml = reinterpret_cast<float2*>(smem + S::OFF_ML);          // [2][128]

  __shared__ long long scratch[33];
  __shared__ TreeShare share;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (threadIdx.x == kCopyWarp * 32) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(&full[s], W8 ? kConvThreads : 1);
      mbar_init(&freed[s], 1);
    }
    for (int s = 0; s < NR; ++s) {
      mbar_init(&raw_full[s], 1);
      mbar_init(&raw_freed[s], kConvThreads);
    }
    for (int s = 0; s < kSBufs; ++s) {
      mbar_init(&s_done[s], 1);
      mbar_init(&p_ready[s], kGroupThreads);
      mbar_init(&pv_done[s], 1);
    }
    mbar_init(q_ready, kSoftThreads);
    mbar_init(mma_idle, 1);
    mbar_fence_init();
    if constexpr (!W8) {
      asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tm_k)) : "memory");
      asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tm_v)) : "memory");
    }
  }
  if (threadIdx.x < 16) bad_nodes[threadIdx.x] = 0;
  tree_share<S::THREADS>(a, scratch, &share);
  if (share.count == 0) return;  // (the whole CTA)
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(s_taddr)),
                 "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *s_taddr;
  TreeWalk walk{share.b, share.off, share.count};
  TreeRun run;

  if (warp == kCopyWarp) {
    // ===================== copies: the share's tiles, in order =====================
    constexpr int N = W8 ? NR : NS;
    uint64_t* const arrive = W8 ? raw_full : full;
    uint64_t* const leave = W8 ? raw_freed : freed;
    int* const masks = W8 ? raw_mask : page_mask;
    // the row units of more than 256 rows read the same tiles again
    const uint64_t pol =
        a.nodes * a.group > kTreeTcRows ? l2_evict_last_policy() : l2_evict_first_policy();
    uint32_t gt = 0;
    bool ok = true;
    while (ok && walk.next(a, run)) {
      const int pages = (run.req.read + kPageSize - 1) / kPageSize;
      const int32_t* table = a.block_tables + (size_t)run.b * a.max_pages;
      const int first = run.tile0 * kPages;
      int ids = -1;  // lane L: the id of page 32 m + L of the run (8 tiles a batch)
      for (int i = 0; i < run.n; ++i, ++gt) {
        if ((i & 7) == 0) {
          const int lp = first + kPages * i + lane;
          ids = lp < pages ? table[lp] : -1;
        }
        int pid[kPages];
#pragma unroll
        for (int p = 0; p < kPages; ++p)
          pid[p] = __shfl_sync(0xffffffffu, ids, (kPages * i + p) & 31);
        const uint32_t st = gt % N;
        if (gt >= N) {
          ok = mbar_wait(&leave[st], (gt / N - 1) & 1u, a.err);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
        }
        if (lane != 0) continue;
        int mask = 0;
#pragma unroll
        for (int p = 0; p < kPages; ++p) {
          if (first + kPages * i + p >= pages) continue;
          if (pid[p] < 0 || pid[p] >= a.num_pages)
            atomicOr(a.err, PKV_DEVERR_BAD_PAGE);
          else
            mask |= 1 << p;
        }
        masks[st] = mask;
        if constexpr (W8) fence_proxy_async_smem();
        mbar_arrive_expect_tx(&arrive[st],
                              __popc(mask) * 2 * (W8 ? PAGE_RAW : PAGE_MMA));
#pragma unroll
        for (int p = 0; p < kPages; ++p) {
          if (!((mask >> p) & 1)) continue;
          if constexpr (W8) {
            const int64_t src = ((int64_t)pid[p] * a.h_kv + run.j) * PAGE_RAW;
            uint8_t* dst = smem + S::OFF_RAW + st * S::RAW_STAGE + p * PAGE_RAW;
            bulk_g2s(dst, static_cast<const uint8_t*>(a.k_cache) + src, PAGE_RAW, &arrive[st], pol);
            bulk_g2s(dst + S::RAW_TILE, static_cast<const uint8_t*>(a.v_cache) + src, PAGE_RAW,
                     &arrive[st], pol);
          } else {
            const int row = (pid[p] * a.h_kv + run.j) * kPageSize;
            const uint32_t dst = ring + st * S::STAGE;
            // K: 64-dim blocks of all 64 rows (one N = 64 operand); V: one block per page (K = 16)
#pragma unroll
            for (int bx = 0; bx < D / 64; ++bx)
              tma_load_2d(dst + bx * (kTok * 128) + p * 2048, &tm_k, bx * 64, row, &arrive[st], pol);
            tma_tile<D / 64, 64>(dst + S::TILE + p * PAGE_MMA, &tm_v, a.tma_rank, row, &arrive[st],
                                 pol);
          }
        }
      }
    }
    if (lane == 0)  // before leaving, every copy issued has landed
      for (uint32_t t = gt > N ? gt - N : 0; t < gt; ++t)
        mbar_wait(&arrive[t % N], (t / N) & 1u, a.err);
  } else if (warp == kMmaWarp) {
    // ===================== MMAs (lane 0) =====================
    if (lane == 0) {
      bool ok = true;
      uint32_t ph = 0, unit = 0;
      uint32_t gt = 0;  // tiles of earlier runs
      for (; ok && walk.next(a, run); ++unit) {
        const Steps st(run);
        ok = mbar_wait(q_ready, unit & 1, a.err);
        tc_fence_after();
        auto s_mma = [&](int u) {
          const uint32_t t = gt + st.tile(u), stage = t % NS;
          if (!mbar_wait(&full[stage], (t / NS) & 1u, a.err)) return false;
          tc_fence_after();
          const uint32_t kb = ring + stage * S::STAGE;
          const uint32_t q = tmem + kColQ + (st.wide && (u & 1) ? 64 : 0);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            tc_mma_ta(tmem + s_col(st.buf(u)), q + 8 * kk,
                      tc_desc(kb + (kk >> 2) * (kTok * 128) + (kk & 3) * 32, 16, 1024), S::IDESC_S,
                      kk > 0 ? 1u : 0u);
          tc_commit(&s_done[st.buf(u)]);
          return true;
        };
        for (int u = 0; ok && u < st.bufs && u < st.n; ++u) ok = s_mma(u);
        for (int u = 0; ok && u < st.n; ++u) {
          const int b = st.buf(u);
          ok = mbar_wait(&p_ready[b], st.parity(ph, u), a.err);
          if (!ok) break;
          tc_fence_after();
          const uint32_t stage = (gt + st.tile(u)) % NS;
          const uint32_t vb = ring + stage * S::STAGE + S::TILE;
#pragma unroll
          for (int kk = 0; kk < kPages; ++kk)
            tc_mma_ta(tmem + kColO + 128 * (u & 1), tmem + s_col(b) + 8 * kk,
                      tc_desc(vb + kk * PAGE_MMA, 2048, 1024), S::IDESC_PV, u < 2 && kk == 0 ? 0u : 1u);
          tc_commit(&pv_done[b]);
          if (!st.wide || (u & 1)) tc_commit(&freed[stage]);
          if (u + st.bufs < st.n) {  // its S overwrites the buffer that this P lives in
            ok = mbar_wait(&pv_done[b], st.parity(ph, u), a.err);
            if (ok) ok = s_mma(u + st.bufs);
          }
        }
        ph = st.after(ph);
        gt += run.n;
      }
      tc_commit(mma_idle);  // before leaving, every MMA issued is complete
      mbar_wait(mma_idle, 0, a.err);
    }
  } else if (W8 && warp >= kConvWarp) {
    // ===================== 8-bit codes to f16 in MMA form =====================
    if constexpr (W8) {
      const int i0 = threadIdx.x - kConvWarp * 32;
      bool ok = true;
      const uint32_t count = (uint32_t)share.count;
      for (uint32_t gt = 0; ok && gt < count; ++gt) {
        const uint32_t rs = gt % NR, cs = gt % NS;
        ok = mbar_wait(&raw_full[rs], (gt / NR) & 1u, a.err);
        if (ok && gt >= NS) ok = mbar_wait(&freed[cs], (gt / NS - 1) & 1u, a.err);
        if (!ok) break;
        const uint32_t src = ring + S::OFF_RAW + rs * S::RAW_STAGE;
        const uint32_t dst = ring + cs * S::STAGE;
        constexpr int CPR = D / 16;  // 16-code chunks of a row
#pragma unroll 2
        for (int i = i0; i < 2 * kTok * CPR; i += kConvThreads) {
          const bool v = i >= kTok * CPR;
          const int e = v ? i - kTok * CPR : i;
          // eight threads read and write distinct banks: four chunks each of two rows
          int row, c;
          if constexpr (CPR == 8) {
            row = 2 * (e >> 4) + ((e >> 2) & 1);
            c = (e & 3) + 4 * (((e >> 2) ^ (e >> 3)) & 1);
          } else {
            row = e >> 2;
            c = e & 3;
          }
          const uint4 w = lds128(src + (v ? S::RAW_TILE : 0) + row * D + c * 16);
          uint4 lo, hi;
          widen4<KV>(w.x, lo.x, lo.y);
          widen4<KV>(w.y, lo.z, lo.w);
          widen4<KV>(w.z, hi.x, hi.y);
          widen4<KV>(w.w, hi.z, hi.w);
          const int ch = 2 * c, x = row & 7;  // 16-byte chunks ch and ch + 1 of the row's f16
          const uint32_t at =
              v ? dst + S::TILE + (row >> 4) * PAGE_MMA + (ch >> 3) * 2048 + (row & 15) * 128
                : dst + (ch >> 3) * (kTok * 128) + row * 128;
          sts128(at + (((ch & 7) ^ x) << 4), lo);
          sts128(at + ((((ch & 7) + 1) ^ x) << 4), hi);
        }
        if (i0 == 0) page_mask[cs] = raw_mask[rs];
        fence_proxy_async_smem();
        mbar_arrive(&full[cs]);
        mbar_arrive(&raw_freed[rs]);
      }
    }
  } else if (warp < kMmaWarp) {
    // ===================== softmax =====================
    const int wg = warp >> 2;             // group
    const int r = threadIdx.x & 127;      // row of the group
    const uint32_t lane_t = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    bool ok = true;
    uint32_t ph = 0, unit = 0, gt = 0;
    for (; walk.next(a, run); ++unit) {
      const Steps st(run);
      const int b = run.b, j = run.j;
      const int R = run.row0 + (st.wide ? wg * kGroupThreads : 0) + r;
      const bool live = R < run.row0 + run.rows;
      const int t = live ? R / a.group : 0, head = j * a.group + (live ? R % a.group : 0);
      uint32_t* const bad = bad_nodes + 8 * (unit & 1);
      float sc = a.scale_log2 * (W8 ? a.k_scales[j] : 1.f);
      // ---- the row's query into tensor memory (both groups' reads of the last unit's O are done) ----
      {
        const uint4* qrow = reinterpret_cast<const uint4*>(
            static_cast<const __nv_bfloat16*>(a.q) +
            (((size_t)b * a.nodes + t) * a.h_q + head) * D);
        uint4 qv[D / 8];
#pragma unroll
        for (int c = 0; c < D / 8; ++c) qv[c] = live ? qrow[c] : make_uint4(0, 0, 0, 0);
        float up = 1.f;
        if constexpr (W8) {
          uint32_t mx = 0;  // largest |q| as bits (bf16 magnitudes order like integers)
#pragma unroll
          for (int c = 0; c < D / 8; ++c) {
            const uint32_t w[4] = {qv[c].x, qv[c].y, qv[c].z, qv[c].w};
#pragma unroll
            for (int k = 0; k < 4; ++k)
              mx = max(mx, max(w[k] & 0x7fffu, (w[k] >> 16) & 0x7fffu));
          }
          const int ex = mx >> 7;  // biased exponent: mx * 2^e in [2^14, 2^15), none for 0, inf, NaN
          const int e = mx != 0 && ex < 255 ? min(126, max(-126, 141 - ex)) : 0;
          up = __int_as_float((127 + e) << 23);
          // (at least the smallest normal number: an unseen score of -inf must stay one)
          sc = fmaxf(sc * __int_as_float((127 - e) << 23), 0x1p-126f);
        }
        if (ok && (st.wide || wg == 0)) {
          const uint32_t q_col = kColQ + (st.wide ? 64 * wg : 0);
#pragma unroll
          for (int h = 0; h < D / 64; ++h) {
            uint32_t w[32];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const uint32_t x[4] = {qv[8 * h + k].x, qv[8 * h + k].y, qv[8 * h + k].z,
                                     qv[8 * h + k].w};
#pragma unroll
              for (int m = 0; m < 4; ++m)
                w[4 * k + m] = W8 ? pack_f16(bf16lo(x[m]) * up, bf16hi(x[m]) * up) : x[m];
            }
            tmem_st32(lane_t + q_col + 32 * h, w);
          }
          tmem_wait_st();
        }
        tc_fence_before();
        mbar_arrive(q_ready);
      }
      float m_used = -INFINITY, l = 0.f;
      for (int u = wg; ok && u < st.n; u += 2) {
        const uint32_t tl = gt + st.tile(u), stage = tl % NS;
        const int buf = st.buf(u);
        ok = mbar_wait(&full[stage], (tl / NS) & 1u, a.err) &&
             mbar_wait(&s_done[buf], st.parity(ph, u), a.err);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        const int mask = page_mask[stage];
        const int p0 = (run.tile0 + st.tile(u)) * kTok;
        tc_fence_after();
        uint32_t sr[64];
        const uint32_t scol = s_col(buf);
        tmem_ld32(lane_t + scol, *reinterpret_cast<uint32_t(*)[32]>(&sr[0]));
        tmem_ld32(lane_t + scol + 32, *reinterpret_cast<uint32_t(*)[32]>(&sr[32]));
        tmem_wait_ld();
        const bool masked = mask != (1 << kPages) - 1 || p0 + kTok > min(run.req.base, run.req.read);
        if (masked) {
          uint64_t seen = live ? tree_seen(a, run.req, b, t, p0) : 0ull;
#pragma unroll
          for (int p = 0; p < kPages; ++p)
            if (!((mask >> p) & 1)) seen &= ~(0xffffull << (16 * p));
#pragma unroll
          for (int k = 0; k < 64; ++k)
            if (!((seen >> k) & 1)) sr[k] = __float_as_uint(-INFINITY);
          if (!st.wide || wg == 0) {  // mend V: two threads to a row
            const int vr = r >> 1, pos = p0 + vr;
            constexpr int CH = D / 16;  // 16-byte chunks of half a row
            const uint32_t vrow = ring + stage * S::STAGE + S::TILE + (vr >> 4) * PAGE_MMA +
                                  (vr & 15) * 128 + (D == 128 ? (r & 1) * 2048 : 0);
            const int c0 = D == 128 ? 0 : (r & 1) * CH;
            if (pos >= run.req.read || !((mask >> (vr >> 4)) & 1)) {
#pragma unroll
              for (int c = 0; c < CH; ++c)
                sts128(vrow + (((c0 + c) ^ (vr & 7)) << 4), make_uint4(0, 0, 0, 0));
            } else if (KV::code != PKV_INT8 && pos >= run.req.base) {
              bool hot = false;
#pragma unroll
              for (int c = 0; c < CH; ++c) {
                const uint32_t at = vrow + (((c0 + c) ^ (vr & 7)) << 4);
                uint4 x = lds128(at);
                uint32_t* w = &x.x;
                bool here = false;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                  if (not_finite<W8>(w[k])) {
                    w[k] &= 0xffff0000u;
                    here = true;
                  }
                  if (not_finite<W8>(w[k] >> 16)) {
                    w[k] &= 0xffffu;
                    here = true;
                  }
                }
                if (here) sts128(at, x);
                hot |= here;
              }
              if (hot) {
                const int node = pos - run.req.base;
                atomicOr(&bad[node >> 5], 1u << (node & 31));
              }
            }
            fence_proxy_async_smem();
          }
        }
        float mx8[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) mx8[k] = -INFINITY;
#pragma unroll
        for (int k = 0; k < 64; ++k) mx8[k & 7] = fmaxf(mx8[k & 7], __uint_as_float(sr[k]));
        const float mx = sc * fmaxf(fmaxf(fmaxf(mx8[0], mx8[1]), fmaxf(mx8[2], mx8[3])),
                                    fmaxf(fmaxf(mx8[4], mx8[5]), fmaxf(mx8[6], mx8[7])));
        if (u == wg) {
          m_used = mx;
        } else {
          const bool need = mx > m_used + kLazyLog2;
          if (__any_sync(0xffffffffu, need)) {  // rescale this warp's rows of O (in TMEM)
            ok = mbar_wait(&pv_done[st.buf(u - 2)], st.parity(ph, u - 2), a.err);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            tc_fence_after();
            const float m_new = need ? mx : m_used;
            const float alpha = m_new == -INFINITY ? 1.f : exp2f(m_used - m_new);
#pragma unroll
            for (int cb = 0; cb < D / 32; ++cb) {
              uint32_t o[32];
              tmem_ld32(lane_t + kColO + 128 * wg + 32 * cb, o);
              tmem_wait_ld();
#pragma unroll
              for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * alpha);
              tmem_st32(lane_t + kColO + 128 * wg + 32 * cb, o);
            }
            tmem_wait_st();
            l *= alpha;
            m_used = m_new;
          }
        }
        // P = 2^(s - m) over the first 32 columns of the tile's S buffer
        const float m_use = m_used == -INFINITY ? 0.f : m_used;
        uint32_t pw[32];
        float sum8[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) sum8[k] = 0.f;
#pragma unroll
        for (int k = 0; k < 32; ++k) {
          const float e0 = ex2_approx(fmaf(__uint_as_float(sr[2 * k]), sc, -m_use));
          const float e1 = ex2_approx(fmaf(__uint_as_float(sr[2 * k + 1]), sc, -m_use));
          sum8[(2 * k) & 7] += e0;
          sum8[(2 * k + 1) & 7] += e1;
          pw[k] = pack_p<W8>(e0, e1);
        }
        tmem_st32(lane_t + scol, pw);
        l += ((sum8[0] + sum8[1]) + (sum8[2] + sum8[3])) +
             ((sum8[4] + sum8[5]) + (sum8[6] + sum8[7]));
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(&p_ready[buf]);
      }
      // ---- the unit's rows ----
      const int last = wg < st.n ? ((st.n - 1 - wg) & ~1) + wg : -1;  // this group's last step
      if (ok && last >= 0) ok = mbar_wait(&pv_done[st.buf(last)], st.parity(ph, last), a.err);
      ok = __all_sync(0xffffffffu, ok);
      tc_fence_after();
      if (!st.wide) ml[wg * kGroupThreads + r] = make_float2(m_used, l);
      tc_fence_before();
      // both groups are here whatever became of their waits
      asm volatile("bar.sync 1, 256;" ::: "memory");
      tc_fence_after();
      if (threadIdx.x < 8) bad_nodes[8 * ((unit + 1) & 1) + threadIdx.x] = 0;
      if (ok) {
        // wide: the group's own rows, all dims; else group wg takes dims wg D/2 .. of every row and
        // merges the two groups' O
        float M = m_used, L = l, w0 = 1.f, w1 = 0.f;
        const bool two = !st.wide && st.n > 1;
        if (!st.wide) {
          const float2 x = ml[r], y = ml[kGroupThreads + r];
          M = fmaxf(x.x, y.x);
          const float Mu = M == -INFINITY ? 0.f : M;
          w0 = exp2f(x.x - Mu);
          w1 = two ? exp2f(y.x - Mu) : 0.f;
          L = w0 * x.y + (two ? w1 * y.y : 0.f);
        }
        const float vs = W8 ? a.v_scales[j] : 1.f;
        const float f = run.whole ? (L != 0.f ? vs / L : 0.f) : vs;
        const size_t part = ((size_t)blockIdx.x * 2 + run.slot) * kTreeTcRows + (R - run.row0);
        __nv_bfloat16* orow = static_cast<__nv_bfloat16*>(a.out) +
                              (((size_t)b * a.nodes + t) * a.h_q + head) * D;
        uint32_t any_bad = 0;
#pragma unroll
        for (int k = 0; k < 8; ++k) any_bad |= bad[k];
        const int c_lo = st.wide ? 0 : wg * (D / 2), c_hi = st.wide ? D : c_lo + D / 2;
        for (int c = c_lo; c < c_hi; c += 32) {
          uint32_t o[32];
          tmem_ld32(lane_t + kColO + (st.wide ? 128 * wg : 0) + c, o);
          if (two) {
            uint32_t o1[32];
            tmem_ld32(lane_t + kColO + 128 + c, o1);
            tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < 32; ++k)
              o[k] = __float_as_uint(w0 * __uint_as_float(o[k]) + w1 * __uint_as_float(o1[k]));
          } else {
            tmem_wait_ld();
            if (!st.wide)
#pragma unroll
              for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(w0 * __uint_as_float(o[k]));
          }
          if (any_bad && live) {  // the infinite and NaN values of the nodes this row sees
            for (int n = 0; n < run.req.nodes; ++n) {
              if (!((bad[n >> 5] >> (n & 31)) & 1)) continue;
              const int pos = run.req.base + n;
              if (!(tree_seen(a, run.req, b, t, pos) & 1)) continue;
              const int id = a.block_tables[(size_t)b * a.max_pages + pos / kPageSize];
              const int64_t at =
                  ((((int64_t)id * a.h_kv + j) * kPageSize + pos % kPageSize) * D + c) * KV::bytes;
              const uint8_t* v = static_cast<const uint8_t*>(a.v_cache) + at;
#pragma unroll
              for (int k = 0; k < 32; k += 4) {
                float x[4];
                RowLoad<KV, 4>::run(v + k * KV::bytes, x);
#pragma unroll
                for (int m = 0; m < 4; ++m)
                  if (!(fabsf(x[m]) < INFINITY))
                    o[k + m] = __float_as_uint(__uint_as_float(o[k + m]) + x[m]);
              }
            }
          }
          if (live) {
            if (run.whole) {
#pragma unroll
              for (int k = 0; k < 32; k += 8) {
                uint4 v;
                uint32_t* w = &v.x;
#pragma unroll
                for (int m = 0; m < 4; ++m)
                  w[m] = L != 0.f ? pack_bf16(__uint_as_float(o[k + 2 * m]) * f,
                                              __uint_as_float(o[k + 2 * m + 1]) * f)
                                  : 0u;
                *reinterpret_cast<uint4*>(orow + c + k) = v;
              }
            } else {
              float* dst = a.ws_acc + part * D + c;
#pragma unroll
              for (int k = 0; k < 32; k += 4)
                *reinterpret_cast<float4*>(dst + k) =
                    make_float4(__uint_as_float(o[k]) * f, __uint_as_float(o[k + 1]) * f,
                                __uint_as_float(o[k + 2]) * f, __uint_as_float(o[k + 3]) * f);
              if (c == 0) *reinterpret_cast<float2*>(a.ws_ml + 2 * part) = make_float2(M, L);
            }
          }
        }
      }
      ph = st.after(ph);
      gt += run.n;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    __syncwarp();
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                 "r"(kTmemCols)
                 : "memory");
  }
}

template <typename KV, int D>
cudaError_t launch_t(const TreeArgs& a, const CUtensorMap& tk, const CUtensorMap& tv,
                     cudaStream_t s) {
  using S = TcShape<KV, D>;
  static std::atomic<unsigned long long> attr_done{0};  // one bit per device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !((attr_done.load() >> dev) & 1ull)) {
    e = cudaFuncSetAttribute(tree_tc_kernel<KV, D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             S::SMEM);
    if (e != cudaSuccess) return e;
    if (dev < 64) attr_done.fetch_or(1ull << dev);
  }
  tree_tc_kernel<KV, D><<<a.ctas, S::THREADS, S::SMEM, s>>>(a, tk, tv);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_tree_tc(const TreeArgs& a, int kv_dtype, int head_dim, const void* tk,
                           const void* tv, cudaStream_t s) {
  const CUtensorMap& mk = *static_cast<const CUtensorMap*>(tk);
  const CUtensorMap& mv = *static_cast<const CUtensorMap*>(tv);
  if (head_dim == 64) {
    if (kv_dtype == PKV_BF16) return launch_t<BF16, 64>(a, mk, mv, s);
    if (kv_dtype == PKV_FP8_E4M3) return launch_t<FP8, 64>(a, mk, mv, s);
    return launch_t<INT8, 64>(a, mk, mv, s);
  }
  if (kv_dtype == PKV_BF16) return launch_t<BF16, 128>(a, mk, mv, s);
  if (kv_dtype == PKV_FP8_E4M3) return launch_t<FP8, 128>(a, mk, mv, s);
  return launch_t<INT8, 128>(a, mk, mv, s);
}

}  // namespace pkv
