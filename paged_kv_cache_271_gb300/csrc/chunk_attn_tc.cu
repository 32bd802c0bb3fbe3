// Attention of chunks of new tokens on the fifth-generation tensor cores (tcgen05), bf16 queries over a
// bf16, FP8 or INT8 cache.
//
// The mathematics is that of chunk_attn.cu; the work is cut as chunk_plan.cuh says, in units of up to
// 256 (token, query head) rows of one KV head and tiles of 128 tokens, one persistent CTA per SM. A
// tile of a full unit takes 4 x 256 x 128 x D operations, 2048 cycles of the tensor cores at D = 128, and
// reads 64 KB of K and V from L2 or memory; everything else is arranged beside that:
//
//  * copy warps stream the share's tiles through rings of shared memory, running ahead across units;
//    a bf16 tile arrives by TMA in the 128-byte-swizzled form the MMAs read, the codes of an 8-bit
//    tile by bulk copies, which four converter warps widen to f16 (exactly) in that form;
//  * one MMA warp issues S = Q K^T (128 rows x 128 tokens) and O += P V, with P as an A operand in the
//    tensor memory that held S and all accumulators there;
//  * two groups of eight softmax warps, two threads to a row: thread (h, r) of a group has tokens 64 h ..
//    of row r's scores, and the two agree on the row's maximum through shared memory. In a unit of more
//    than 128 rows group g takes rows 128 g .. of every tile: while one group works on its scores, the
//    tensor cores have the other's P V and next S. In a smaller unit both groups have the same rows and
//    take alternate tiles, and the sums are merged at the unit's end;
//  * O is rescaled only when a row's maximum grows by more than 2^8 (8-bit caches: 2^7): the final
//    (max, sum, O) is exact whatever reference it was accumulated against.
//
// P is rounded to the MMA's input type (bf16 for a bf16 cache, f16 otherwise), the only rounding
// before the output's; scores, maxima and sums are fp32. (Outputs' relative error against 64 bits, over a
// bf16 cache: 0.0019 to 0.0023, where weights in 32 bits give 0.0017, the output's own rounding; over 8-bit
// caches no more than that. What bf16 leaves out, as a second operand, would be half as many MMAs again.)
// For 8-bit caches a query row is scaled by a power of two that puts its largest value in f16's top binade,
// undone in its score factor; the sign of the K scale goes with it, so that score factors are positive.
//
// Tiles with unseen positions (the chunk's own, the window's edge, bad pages) mask scores by the row's
// mask bits, and their V rows are mended in shared memory before the MMA reads them: rows outside the
// context or on a page that is not there become 0, and infinite or NaN values, which a weight of 0
// would still spread to rows that do not see them, become 0 there and are added to the rows that do
// see them at the unit's end.
//
// Measured: an 8191-token prompt, 32 heads on 8 of 128 dims, bf16, 436 us (1.26 PFLOP/s of the 1.91 that a
// library product reaches); 2048 tokens over 32768 cached ones, 64 heads, FP8, 2.04 ms (1.11); 64 decode steps
// with biases 133 us (4.5 TB/s), without 114 (5.2), over FP8 152 (2.0). A tile of a full unit takes about 3300
// cycles: S is issued in 640 a group (both its operands come from shared memory, 128 bytes a clock), and of a
// group's chain of S, maximum, exchange, exponentials, P and P V two are under way at a time.
//
// Every wait is bounded (PKV_DEVERR_TIMEOUT); the tensor memory is freed on every path.
#include <atomic>
#include <cuda.h>
#include <limits.h>
#include <math.h>

#include "chunk_plan.cuh"
#include "chunk_score.cuh"
#include "paged_decode_mma.cuh"
#include "pkv_device.cuh"
#include "pkv_internal.h"
#include "tc_pipe.cuh"
#include "tcgen05.cuh"

namespace pkv {

namespace {

constexpr int kTok = kChunkTcTokens;       // tokens of a tile
constexpr int kPages = kTok / kPageSize;   // pages of a tile
constexpr int kGroupRows = 128;            // rows of a softmax group
constexpr int kGroupWarps = 8;             // its warps: four for each half of a row's scores
constexpr int kSoftThreads = 2 * kGroupWarps * 32;
constexpr int kMmaWarp = kSoftThreads / 32;
constexpr int kCopyWarp = kMmaWarp + 1;    // K; the next one V (8-bit caches: one for both)
constexpr int kConvWarp = kMmaWarp + 4;    // first of four (8-bit caches; one warp before is idle)
constexpr int kConvThreads = 128;
// Runs on their way from the first copy warp, which walks the share, to the other warps. It is ahead
// of the slowest by the tiles in the rings at most, each a run of its own at worst, besides the run whose
// rows are being written, the one after it and the one it is about to copy.
constexpr int kRuns = 16;
constexpr uint32_t kTmemCols = 512;        // O of group g at 128 g, S (then P) at 256 + 128 g
// tiles of a unit in which some rows see a position that others do not: those that cross the sinks'
// end, and those of the at most 256 positions from the first to the last row's end or window
constexpr int kEdgeTiles = 8;
static_assert(2 * kGroupRows == kChunkTcRows, "a unit is two groups' rows");

template <typename KV, int D>
struct TcShape {
  static constexpr bool W8 = KV::bytes == 1;
  static constexpr int THREADS = 32 * (W8 ? kConvWarp + kConvThreads / 32 : kConvWarp);
  // registers of the softmax warps, of MMA and copies, and of the converters, out of what the launch
  // gives every warp
  static constexpr int LAUNCH_REGS = W8 ? 80 : 96;
  static constexpr int SOFT_REGS = W8 ? 88 : 104, REGS = W8 ? 48 : 64, CONV_REGS = 80;
  static_assert(kSoftThreads * SOFT_REGS + 128 * REGS + (W8 ? 128 * CONV_REGS : 0) <=
                    THREADS * LAUNCH_REGS,
                "the split takes no more registers than the launch brings");
  static constexpr int TILE = kTok * D * 2;       // K (or V) of a tile in MMA form
  static constexpr int NK = 64 * 1024 / TILE, NV = NK;
  static constexpr int RAW = kTok / 2 * D;        // codes of half a tile's K or V
  static constexpr int NR = W8 ? (D == 128 ? 3 : 8) : 0;
  static constexpr int OFF_V = NK * TILE;
  static constexpr int OFF_RAW = OFF_V + NV * TILE;
  static constexpr int OFF_Q = OFF_RAW + NR * RAW;
  static constexpr int Q_GROUP = kGroupRows * D * 2;
  static constexpr int OFF_HALF = OFF_Q + 2 * Q_GROUP;             // [2][2][128] of the half rows
  static constexpr int OFF_REF = OFF_HALF + kSoftThreads * 4;      // [2][128] the rows' maxima
  static constexpr int OFF_FAC = OFF_REF + 2 * kGroupRows * 4;     // [2][128] score factors (8-bit)
  static constexpr int OFF_BAR = OFF_FAC + (W8 ? 2 * kGroupRows * 4 : 0);
  static constexpr int BARS = 2 * NK + 2 * NV + 2 * NR + 2 * 4 + 8 + 3 + kRuns;
  static_assert(NK + (NR + 3) / 4 + 3 <= kRuns, "runs in flight");
  static constexpr int OFF_MISC = OFF_BAR + 8 * BARS;              // masks, TMEM address
  static constexpr uint32_t IDESC_S = tc_idesc(128, kTok, false, W8);
  static constexpr uint32_t IDESC_PV = tc_idesc(128, D, true, W8);
  static constexpr int SMEM = 1024 + OFF_MISC + 4 * (NV + NR + 1) + 16;
  static_assert(SMEM <= 223 * 1024 && SMEM > 114 * 1024, "one CTA per SM");
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

// z + 0 w for the two 16-bit values of a word: NaN from the first infinite or NaN one on.
template <bool F16>
__device__ __forceinline__ uint32_t add_zero_times(uint32_t w, uint32_t z) {
  uint32_t r;
  if constexpr (F16)
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(w), "r"(0u), "r"(z));
  else
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(w), "r"(0u), "r"(z));
  return r;
}

// FORM: scores are capped or have a bias (otherwise they are the products, scaled).
template <typename KV, int D, bool FORM>
__global__ void __launch_bounds__(TcShape<KV, D>::THREADS, 1) chunk_tc_kernel(
    const ChunkArgs a, const __grid_constant__ CUtensorMap tm_k,
    const __grid_constant__ CUtensorMap tm_v) {
  using S = TcShape<KV, D>;
  constexpr bool W8 = S::W8;
  constexpr int NK = S::NK, NV = S::NV, NR = S::NR;
  constexpr int PAGE_MMA = kPageSize * D * 2;  // V bytes of a page in MMA form
  constexpr int PAGE_RAW = kPageSize * D;
  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t ring = smem_u32(smem);
  uint64_t* full_k = reinterpret_cast<uint64_t*>(smem + S::OFF_BAR);  // [NK] K of a tile is there
  uint64_t* free_k = full_k + NK;                                    // [NK] its S done
  uint64_t* full_v = free_k + NK;                                    // [NV] V of a tile is there
  uint64_t* free_v = full_v + NV;                                    // [NV] its P V done
  uint64_t* raw_full = free_v + NV;                                  // [NR] codes arrived
  uint64_t* raw_freed = raw_full + NR;                               // [NR] codes in registers
  uint64_t* s_done = raw_freed + NR;                                 // [2] S of a group's step
  uint64_t* p_ready = s_done + 2;                                    // [2] its P
  uint64_t* o_done = p_ready + 2;                                    // [2] a group's last P V of a run
  uint64_t* q_ready = o_done + 2;                                    // [2] Q of a run stored
  uint64_t* paired = q_ready + 2;      // [2][4] the two warps of 32 rows have left word of a half row
  uint64_t* met = paired + 8;          // both groups ended a small run
  uint64_t* parted = met + 1;          // and are done with what the other reads or writes
  uint64_t* mma_idle = parted + 1;
  uint64_t* run_there = mma_idle + 1;  // [kRuns]
  int* page_mask = reinterpret_cast<int*>(smem + S::OFF_MISC);       // [NV] good pages of the tile
  int* raw_mask = page_mask + NV;                                    // [NR] of the half tile
  uint32_t* s_taddr = reinterpret_cast<uint32_t*>(raw_mask + NR);
  float* half_row = reinterpret_cast<float*>(smem + S::OFF_HALF);
  float* row_max = reinterpret_cast<float*>(smem + S::OFF_REF);
  float* row_fac = reinterpret_cast<float*>(smem + S::OFF_FAC);

  __shared__ int scratch[64];
  __shared__ ChunkShare share;
  __shared__ ChunkRun runs[kRuns];  // (n = 0: the share's end)
  __shared__ uint32_t bad_rows[kRuns][kEdgeTiles * 4];  // of a run's edge tiles: V row not finite
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (threadIdx.x == kCopyWarp * 32) {
    for (int s = 0; s < NK; ++s) {
      mbar_init(&full_k[s], W8 ? kConvThreads / 32 : 1);
      mbar_init(&free_k[s], 1);
    }
    for (int s = 0; s < NV; ++s) {
      mbar_init(&full_v[s], W8 ? kConvThreads / 32 : 1);
      mbar_init(&free_v[s], 1);
    }
    for (int s = 0; s < NR; ++s) {
      mbar_init(&raw_full[s], 1);
      mbar_init(&raw_freed[s], kConvThreads / 32);
    }
    for (int g = 0; g < 2; ++g) {
      mbar_init(&s_done[g], 1);
      mbar_init(&p_ready[g], kGroupWarps);
      mbar_init(&o_done[g], 1);
      mbar_init(&q_ready[g], kGroupWarps);
      for (int w = 0; w < 4; ++w) mbar_init(&paired[4 * g + w], 2);
    }
    mbar_init(met, kSoftThreads / 32);
    mbar_init(parted, kSoftThreads / 32);
    mbar_init(mma_idle, 1);
    for (int i = 0; i < kRuns; ++i) mbar_init(&run_there[i], 1);
    mbar_fence_init();
    if constexpr (!W8) {
      asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tm_k)) : "memory");
      asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tm_v)) : "memory");
    }
  }
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(s_taddr)),
                 "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  chunk_share<S::THREADS>(a, scratch, &share);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = (uint32_t)uniform((int)*s_taddr);
  auto release = [&] {
    __syncwarp();
    if (warp == kMmaWarp)
      asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols)
                   : "memory");
  };
  if (share.count == 0) {  // (the whole CTA)
    if (threadIdx.x == 0) static_cast<ChunkRecord*>(a.ws_rec)[blockIdx.x] = ChunkRecord{0, 1, 0, 0};
    release();
    return;
  }
  // run i of the share, or nullptr after the last (or a wait that gave up)
  auto get_run = [&](uint32_t i) -> const ChunkRun* {
    const bool got = mbar_wait(&run_there[i % kRuns], (i / kRuns) & 1u, a.err);
    const ChunkRun* r = &runs[i % kRuns];
    return __all_sync(0xffffffffu, got && r->n > 0) ? r : nullptr;
  };
  // Steps of a run: wide (more than 128 rows): step u is tile u / 2 for group u % 2, otherwise tile u
  // for group u % 2. Every barrier of a group completes once per step of its own.
  auto is_wide = [](const ChunkRun* run) { return uniform(run->rows) > kGroupRows; };

  if (warp >= kMmaWarp && warp < kConvWarp) {
    regs_down<S::REGS>();
    if (warp == kCopyWarp || (!W8 && warp == kCopyWarp + 1)) {
      // ===================== copies: the share's tiles, in order =====================
      const bool is_k = warp == kCopyWarp;
      const uint64_t once = l2_evict_first_policy(), again = l2_evict_last_policy();
      const int stages = W8 ? NR : is_k ? NK : NV;
      uint64_t* const there = W8 ? raw_full : is_k ? full_k : full_v;
      uint64_t* const gone = W8 ? raw_freed : is_k ? free_k : free_v;
      const uint32_t ring0 = ring + (is_k ? 0 : S::OFF_V);
      int st = 0, issued = 0;
      uint32_t par = 0;
      bool ok = true;
      ChunkWalk walk(a, share);
      ChunkRecord record{0, 1, 0, 0};
      for (uint32_t unit = 0;; ++unit) {
        const ChunkRun* run = nullptr;
        if (is_k) {  // (a wait that gave up ends the share for every warp)
          ChunkRun* r = &runs[unit % kRuns];
          bad_rows[unit % kRuns][lane] = 0;
          __syncwarp();
          if (lane == 0) {
            if (!ok || !walk.next(a, *r)) r->n = 0;
            mbar_arrive(&run_there[unit % kRuns]);
          }
          __syncwarp();
          if (r->n > 0) run = r;
          if (run && !run->whole && run->slot == 1)
            record = ChunkRecord{(int)chunk_row(a, *run, 0), run->heads, run->rows, run->shares};
        } else if (ok) {
          run = get_run(unit);
        }
        if (!run) break;
        const int n = uniform(run->n), j = uniform(run->j), i0 = uniform(run->i0);
        const ChunkTiles tiles{0, uniform(run->tiles.sinks), uniform(run->tiles.first)};
        const int first = uniform(run->req.base + run->t0), ctx = uniform(run->req.base + run->req.n);
        const int32_t* table = a.block_tables + (size_t)uniform(run->b) * a.max_pages;
        // later units of the request read the same rows again
        const uint64_t pol = uniform(run->req.n) > a.unit_tokens ? again : once;
        // lane p: the id of page p of a tile; -1 where it is not read, -2 where it is but has no id
        auto page_of = [&](int i) {
          const int lp = tiles[i0 + i] * kPages + (lane & (kPages - 1)), p0 = lp * kPageSize;
          // (a page outside every row's window may have been given back: it is not read)
          if (i >= n || p0 >= ctx || (a.window > 0 && p0 >= a.sink &&
                                      p0 + kPageSize <= first + 1 - a.window))
            return -1;
          const int id = table[lp];
          return id >= 0 && id < a.num_pages ? id : -2;
        };
        int next = page_of(0);
        for (int i = 0; i < n; ++i) {
          const int mine = next;
          next = page_of(i + 1);
          int id[kPages];
          const uint32_t mask = __ballot_sync(0xffffffffu, mine >= 0) & ((1u << kPages) - 1);
          if (is_k && __any_sync(0xffffffffu, mine == -2) && lane == 0)
            atomicOr(a.err, PKV_DEVERR_BAD_PAGE);
#pragma unroll
          for (int p = 0; p < kPages; ++p) id[p] = __shfl_sync(0xffffffffu, mine, p);
          // a stage: a bf16 tile of K or V, or the codes of half of one (K, K, V, V)
#pragma unroll 1
          for (int part = 0; part < (W8 ? 4 : 1); ++part) {
            if (issued >= stages) {
              ok = __all_sync(0xffffffffu, mbar_wait(&gone[st], par ^ 1u, a.err));
              if (!ok) break;
            }
            if (elect_one()) {
              if constexpr (W8) {
                constexpr int HALF = kPages / 2;
                const uint32_t m = (mask >> ((part & 1) * HALF)) & ((1u << HALF) - 1);
                raw_mask[st] = (int)m;
                fence_proxy_async_smem();
                mbar_arrive_expect_tx(&there[st], __popc(m) * PAGE_RAW);
                const uint8_t* pool = static_cast<const uint8_t*>(part < 2 ? a.k_cache : a.v_cache);
#pragma unroll
                for (int p = 0; p < HALF; ++p) {
                  const int page = part & 1 ? id[HALF + p] : id[p];
                  if ((m >> p) & 1)
                    bulk_g2s(smem + S::OFF_RAW + st * S::RAW + p * PAGE_RAW,
                             pool + ((int64_t)page * a.h_kv + j) * PAGE_RAW, PAGE_RAW, &there[st],
                             pol);
                }
              } else {
                if (!is_k) page_mask[st] = (int)mask;
                mbar_arrive_expect_tx(&there[st], __popc(mask) * PAGE_MMA);
                const uint32_t dst = ring0 + st * S::TILE;
#pragma unroll
                for (int p = 0; p < kPages; ++p) {
                  if (!((mask >> p) & 1)) continue;
                  const int row = (id[p] * a.h_kv + j) * kPageSize;
                  if (is_k) {  // 64-dim blocks of all 128 rows (one N = 128 operand)
#pragma unroll
                    for (int bx = 0; bx < D / 64; ++bx)
                      tma_load_2d(dst + bx * (kTok * 128) + p * 2048, &tm_k, bx * 64, row,
                                  &there[st], pol);
                  } else {  // a block per page (K = 16)
                    tma_tile<D / 64, 64>(dst + p * PAGE_MMA, &tm_v, a.tma_rank, row, &there[st],
                                         pol);
                  }
                }
              }
            }
            __syncwarp();
            if (++st == stages) {
              st = 0;
              par ^= 1u;
            }
            ++issued;
          }
          if (!ok) break;
        }
      }
      if (is_k && lane == 0) static_cast<ChunkRecord*>(a.ws_rec)[blockIdx.x] = record;
      if (lane == 0)  // before leaving, every copy issued has landed
        for (int t = max(0, issued - stages); t < issued; ++t)
          mbar_wait(&there[t % stages], (uint32_t)(t / stages) & 1u, a.err);
    } else if (warp == kMmaWarp) {
      // ===================== MMAs (one elected lane issues) =====================
      // They run in the order of their issue: an S overwrites a P after the P V before it.
      const uint64_t k_desc = tc_desc(ring, 16, 1024), v_desc = tc_desc(ring + S::OFF_V, 2048, 1024);
      const uint64_t q_desc = tc_desc(ring + S::OFF_Q, 16, 1024);
      bool ok = true;
      uint32_t ph_p = 0, ph_q = 0;  // parities of the next phases of p_ready and q_ready, bit g
      Place<NK> ks;       // K of the next S
      Place<NV> vs;       // V of the next P V
      auto wait = [&](uint64_t* bar, uint32_t par) {
        const bool got = __all_sync(0xffffffffu, mbar_wait(bar, par, a.err));
        tc_fence_after();
        return got;
      };
      auto s_mma = [&](int group, bool last_use) {
        const uint64_t kd = k_desc + (uint32_t)(ks.st * (S::TILE >> 4));
        const uint64_t qd = q_desc + (uint32_t)(group * (S::Q_GROUP >> 4));
        const uint32_t d = tmem + 256 + 128 * group;
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t at = ((kk >> 2) * (kTok * 128) + (kk & 3) * 32) >> 4;
            tc_mma_sa(d, qd + at, kd + at, S::IDESC_S, kk > 0 ? 1u : 0u);
          }
          tc_commit(&s_done[group]);
          if (last_use) tc_commit(&free_k[ks.st]);
        }
        __syncwarp();
        if (last_use) ks.advance(1);
      };
      static_assert(kTok == kGroupRows && kEdgeTiles * 4 == 32, "Q and K tiles have one form");
      auto pv_mma = [&](int group, bool first, bool last_use, bool last_step) {
        const uint64_t vd = v_desc + (uint32_t)(vs.st * (S::TILE >> 4));
        const uint32_t pc = tmem + 256 + 128 * group, o = tmem + 128 * group;
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < kPages; ++kk)
            tc_mma_ta(o, pc + 8 * kk, vd + ((kk * PAGE_MMA) >> 4), S::IDESC_PV,
                      first && kk == 0 ? 0u : 1u);
          if (last_use) tc_commit(&free_v[vs.st]);
          if (last_step) tc_commit(&o_done[group]);
        }
        __syncwarp();
        if (last_use) vs.advance(1);
      };
      for (uint32_t unit = 0; ok; ++unit) {
        const ChunkRun* run = get_run(unit);
        if (!run) break;
        const bool wide = is_wide(run);
        const int n = wide ? 2 * uniform(run->n) : uniform(run->n);
        auto step_s = [&](int u) {  // S of step u; in a run's first two steps the queries are waited for
          const int group = u & 1;
          if (u < 2) {
            ok = wait(&q_ready[group], (ph_q >> group) & 1u);
            ph_q ^= 1u << group;
          }
          if (ok && (!wide || group == 0)) ok = wait(&full_k[ks.st], ks.par);
          if (ok) s_mma(group, !wide || group == 1);
        };
        step_s(0);
        if (ok && n > 1) step_s(1);
        for (int u = 0; ok && u < n; ++u) {
          const int group = u & 1;
          ok = wait(&p_ready[group], (ph_p >> group) & 1u);
          ph_p ^= 1u << group;
          if (ok && (!wide || group == 0)) ok = wait(&full_v[vs.st], vs.par);
          if (ok) pv_mma(group, u < 2, !wide || group == 1, u + 2 >= n);
          if (ok && u + 2 < n) step_s(u + 2);
        }
      }
      if (elect_one()) tc_commit(mma_idle);  // before leaving, every MMA issued is complete
      __syncwarp();
      wait(mma_idle, 0);
    }
  } else if (warp >= kConvWarp) {
    // ===================== 8-bit codes to f16 in MMA form =====================
    if constexpr (W8) {
      static_assert(S::CONV_REGS == S::LAUNCH_REGS, "no change");
      constexpr int CPR = D / 16;                          // 16-code chunks of a row
      constexpr int PER = kTok / 2 * CPR / kConvThreads;   // chunks of a thread in half a tile
      const int i0 = threadIdx.x - kConvWarp * 32;
      // a thread's chunks are PER rows, ROWS rows apart. Eight threads read and write distinct banks:
      // four chunks each of two rows.
      constexpr int ROWS = kConvThreads / CPR;
      int row0, c;
      if constexpr (CPR == 8) {
        row0 = 2 * (i0 >> 4) + ((i0 >> 2) & 1);
        c = (i0 & 3) + 4 * (((i0 >> 2) ^ (i0 >> 3)) & 1);
      } else {
        row0 = i0 >> 2;
        c = i0 & 3;
      }
      const int ch = 2 * c;  // 16-byte chunks ch and ch + 1 of the row's f16
      const uint32_t x0 = ((ch & 7) ^ (row0 & 7)) << 4, x1 = (((ch & 7) + 1) ^ (row0 & 7)) << 4;
      static_assert(ROWS % 8 == 0, "a thread's rows share their swizzle");
      const uint32_t src0 = ring + S::OFF_RAW + row0 * D + c * 16;
      const uint32_t k0 = ring + (ch >> 3) * (kTok * 128) + row0 * 128;
      const uint32_t v0 = ring + S::OFF_V + (ch >> 3) * 2048;
      Place<W8 ? NR : 1> raw;
      Place<NK> pk;
      Place<NV> pv;
      bool ok = true;
      int t = 0, end = 0;  // tiles done, tiles of the runs so far
      uint32_t unit = 0;
      for (;; ++t, pk.advance(1), pv.advance(1)) {
        if (t == end) {
          const ChunkRun* run = get_run(unit++);
          if (!run) break;
          end += run->n;
        }
        int mask = 0;
#pragma unroll
        for (int part = 0; part < 4; ++part) {  // K, K, V, V
          ok = mbar_wait(&raw_full[raw.st], raw.par, a.err);
          if (!ok) break;
          const uint32_t src = src0 + raw.st * S::RAW;
          if (part >= 2) mask |= raw_mask[raw.st] << ((part & 1) * (kPages / 2));
          uint4 w[PER];
#pragma unroll
          for (int i = 0; i < PER; ++i) w[i] = lds128(src + i * ROWS * D);
          __syncwarp();
          if (lane == 0) mbar_arrive(&raw_freed[raw.st]);
          raw.advance(1);
          if (part == 0 && t >= NK) ok = mbar_wait(&free_k[pk.st], pk.par ^ 1u, a.err);
          if (part == 2 && t >= NV) ok = mbar_wait(&free_v[pv.st], pv.par ^ 1u, a.err);
          if (!ok) break;
#pragma unroll
          for (int i = 0; i < PER; ++i) {
            const int r = (part & 1) * (kTok / 2) + i * ROWS;  // row of the tile, less row0
            const int rv = r + row0;
            const uint32_t at = part < 2 ? k0 + pk.st * S::TILE + r * 128
                                         : v0 + pv.st * S::TILE + (rv >> 4) * PAGE_MMA +
                                               (rv & 15) * 128;
            uint4 lo, hi;
            widen4<KV>(w[i].x, lo.x, lo.y);
            widen4<KV>(w[i].y, lo.z, lo.w);
            widen4<KV>(w[i].z, hi.x, hi.y);
            widen4<KV>(w[i].w, hi.z, hi.w);
            sts128(at + x0, lo);
            sts128(at + x1, hi);
          }
          if (part & 1) {
            if (part == 3 && i0 == 0) page_mask[pv.st] = mask;
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(part == 1 ? &full_k[pk.st] : &full_v[pv.st]);
          }
        }
        if (!ok) break;
      }
    }
  } else {
    // ===================== softmax =====================
    regs_up<S::SOFT_REGS>();
    const int wg = warp >> 3, h = (warp >> 2) & 1, quad = warp & 3;  // group, half of a row, rows / 32
    const int r = quad * 32 + lane;                                  // row of the group
    const uint32_t lane_t = tmem + ((uint32_t)(quad * 32) << 16);
    const uint32_t s_all = lane_t + 256 + 128 * wg;
    const uint32_t scol = s_all + 64 * h, pcol = s_all + 32 * h, ocol = lane_t + 128 * wg;
    uint64_t* const pair = &paired[4 * wg + quad];
    float* const mine = half_row + (2 * wg + h) * kGroupRows + r;
    const float* const theirs = half_row + (2 * wg + 1 - h) * kGroupRows + r;
    bool ok = true;
    uint32_t unit = 0, ph_s = 0, ph_o = 0, ph_pair = 0, ph_met = 0;  // parities of the next phases
    Place<NV> base;                                                  // V of the run's first tile
    // What this warp says in shared memory and the other warp of its rows, exchanged.
    auto exchange = [&](float x) {
      *mine = x;
      __syncwarp();
      if (lane == 0) mbar_arrive(pair);
      ok = mbar_wait(pair, ph_pair, a.err) && ok;
      ok = __all_sync(0xffffffffu, ok);
      ph_pair ^= 1u;
      return *theirs;
    };
    // The row of this thread in a run (row `row` of its unit, at position pq), its offset in q and
    // out in rows.
    struct Row {
      int row, pq;
      size_t at;
      bool live;
      float slope;
    };
    auto find_row = [&](const ChunkRun& run) {
      Row x;
      x.row = (run.rows > kGroupRows ? wg * kGroupRows : 0) + r;
      x.live = x.row < run.rows;
      const unsigned R = x.live ? x.row : 0, t = R / (unsigned)run.heads;
      x.pq = run.req.base + run.t0 + (int)t;
      x.at = (size_t)(run.req.q0 + run.t0 + (int)t) * a.h_q + run.j * a.group + run.g0 +
             (R - t * run.heads);
      x.slope = FORM && a.slopes ? a.slopes[run.j * a.group + run.g0 + R - t * run.heads] * kLog2e : 0.f;
      return x;
    };
    // A run's queries go straight into shared memory in MMA form while the last step of the run before
    // is worked on, 16 rows a warp, four lanes copying 64 consecutive bytes of a row; for an 8-bit cache
    // the lanes that copied a row then make f16 of it and leave its score factor.
    constexpr int RND = D / 32;  // rounds of 64 bytes
    const int row0 = quad * 32 + 16 * h + (lane >> 2);  // rows row0 and row0 + 8 of the group
    const uint32_t q_at = ring + S::OFF_Q + wg * S::Q_GROUP + row0 * 128;
    auto q_chunk = [&](int d, int g) {
      return q_at + (d >> 1) * (kGroupRows * 128) + g * 1024 +
             ((((4 * d & 7) + (lane & 3)) ^ (row0 & 7)) << 4);
    };
    // Queries are brought for runs in which the group has a step: the MMAs wait for each of them.
    auto has_step = [&](const ChunkRun& run) { return run.rows > kGroupRows || wg < run.n; };
    auto load_query = [&](const ChunkRun& run, const Row& x) {
      if (!has_step(run)) return;
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        const int from = 16 * h + 8 * g + (lane >> 2);
        const size_t at = __shfl_sync(0xffffffffu, (unsigned long long)x.at, from);
        const bool there = __shfl_sync(0xffffffffu, (int)x.live, from) != 0;
        const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(a.q) + at * D + 8 * (lane & 3);
#pragma unroll
        for (int d = 0; d < RND; ++d)
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(q_chunk(d, g)),
                       "l"(src + 32 * d), "r"(there ? 16 : 0)
                       : "memory");
      }
    };
    auto store_query = [&](const ChunkRun& run) {
      if (!has_step(run)) return;
      asm volatile("cp.async.wait_all;" ::: "memory");
      if constexpr (W8) {
        const float sc = a.scale * kLog2e * a.k_scales[run.j];
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          uint4 in[RND];
#pragma unroll
          for (int d = 0; d < RND; ++d) in[d] = lds128(q_chunk(d, g));
          const float factor = query_to_f16<RND>(in, sc);
#pragma unroll
          for (int d = 0; d < RND; ++d) sts128(q_chunk(d, g), in[d]);
          if ((lane & 3) == 0) row_fac[wg * kGroupRows + row0 + 8 * g] = factor;
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&q_ready[wg]);
    };
    Row me{};
    const ChunkRun* next = get_run(0);
    if (next) {
      me = find_row(*next);
      load_query(*next, me);
      store_query(*next);
    }
    float sc = a.scale * kLog2e;  // of the row's scores (log2 domain)
    for (; next; ++unit) {
      const ChunkRun& run = *next;
      const bool wide = run.rows > kGroupRows;
      const bool live = me.live;
      const int ctx = run.req.base + run.req.n;
      const int stride = wide ? 1 : 2;  // tiles between this group's steps
      uint32_t* const bad = bad_rows[unit % kRuns];
      // tiles that begin behind edge_from, or before edge_win and not wholly among the sinks, have
      // positions that some rows do not see (chunk_edge)
      const int edge_from = run.req.base + run.t0 - kTok + 1;
      const int edge_win = a.window > 0 ? run.req.base + run.t0 + run.tokens - a.window : INT_MIN;
      float m_used = -INFINITY, l = 0.f;
      Place<NV> at = base;
      if (!wide) at.advance(wg);
      const int i_first = wide ? 0 : wg;
      const bool any = i_first < run.n;  // the group has a step in the run
      Row then{};
      const ChunkRun* after = nullptr;
      for (int i = i_first; ok && i < run.n; i += stride) {
        const int p0 = run.tiles[run.i0 + i] * kTok;
        // V of the tile too: what it says of its pages, and rows of it may have to be mended. S first: it
        // is issued behind P V of two steps before, so that V's stage is past its last use, which may have
        // been the other group's (before, a phase could look over that has not begun).
        static_assert(NV >= 2, "P V of two steps before");
        ok = mbar_wait(&s_done[wg], ph_s, a.err) && mbar_wait(&full_v[at.st], at.par, a.err);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        ph_s ^= 1u;
        const int mask = page_mask[at.st];
        tc_fence_after();
        uint32_t sr[64];
        tmem_ld32(scol, *reinterpret_cast<uint32_t(*)[32]>(&sr[0]));
        tmem_ld32(scol + 32, *reinterpret_cast<uint32_t(*)[32]>(&sr[32]));
        if constexpr (W8) {
          if (i == i_first) sc = row_fac[wg * kGroupRows + r];
        }
        if (i + stride >= run.n) {  // the group's last S of the run: its queries are used up
          after = get_run(unit + 1);
          if (after) {
            then = find_row(*after);
            load_query(*after, then);
          }
        }
        tmem_wait_ld();
        const bool edge = p0 > edge_from || (p0 < edge_win && p0 + kTok > a.sink);
        // which of its positions this thread's row sees, in tiles where that need not be all
        const bool part = edge || mask != (1 << kPages) - 1;
        auto seen_now = [&] {
          uint64_t seen = live ? chunk_seen(a, me.pq, p0 + 64 * h) : 0ull;
#pragma unroll
          for (int p = 0; p < 4; ++p)
            if (!((mask >> (4 * h + p)) & 1)) seen &= ~(0xffffull << (16 * p));
          return seen;
        };
        if constexpr (FORM) {  // the scores themselves, log2 domain
          if (a.softcap > 0.f) {
            // (what is not seen may be whatever memory held, and has no say in how the cap is taken)
            if (part) {  // (bits made twice, kept they cost registers in every tile: INT8 mix 930 us, not 866)
              const uint64_t seen = seen_now();
              const uint32_t lo = (uint32_t)seen, hi = (uint32_t)(seen >> 32);
#pragma unroll
              for (int k = 0; k < 32; ++k) {
                sr[k] &= 0u - ((lo >> k) & 1u);
                sr[32 + k] &= 0u - ((hi >> k) & 1u);
              }
            }
            cap_scores<64>(sr, sc * (kLn2 / a.softcap), a.softcap * kLog2e);
          } else {
            const uint64_t sc2 = pack2(sc, sc);
#pragma unroll
            for (int k = 0; k < 64; k += 2) put2(&sr[k], mul2(get2(&sr[k]), sc2));
          }
          if (a.slopes) {
            const float far0 = (float)(p0 + 64 * h - me.pq);
            const uint64_t slope2 = pack2(me.slope, me.slope), far2 = pack2(far0, far0);
#pragma unroll
            for (int k = 0; k < 64; k += 2)
              put2(&sr[k], fma2(slope2, add2(far2, pack2((float)k, (float)(k + 1))), get2(&sr[k])));
          }
        }
        if (part) {
          const uint64_t seen = seen_now();
#pragma unroll
          for (int k = 0; k < 64; ++k)
            if (!((seen >> k) & 1)) sr[k] = __float_as_uint(-INFINITY);
          // Mend V, two threads to a row. In a wide unit both groups do (and write every row they
          // mend): each group's P V waits for its own group only. A row is noted before it is mended:
          // who finds it mended finds the note.
          constexpr int CH = D / 16;  // 16-byte chunks of half a row
          const uint32_t vrow = ring + S::OFF_V + at.st * S::TILE + (r >> 4) * PAGE_MMA + (r & 15) * 128;
          auto chunk_at = [&](int c) {
            const int k = CH * h + c;
            return vrow + (k >> 3) * 2048 + (((k & 7) ^ (r & 7)) << 4);
          };
          if (p0 + r >= ctx || !((mask >> (r >> 4)) & 1)) {
#pragma unroll
            for (int c = 0; c < CH; ++c) sts128(chunk_at(c), make_uint4(0, 0, 0, 0));
          } else if (KV::code != PKV_INT8 && edge) {
            uint32_t z = 0;
#pragma unroll
            for (int c = 0; c < CH; ++c) {
              const uint4 x = lds128(chunk_at(c));
              z = add_zero_times<W8>(x.x, z);
              z = add_zero_times<W8>(x.y, z);
              z = add_zero_times<W8>(x.z, z);
              z = add_zero_times<W8>(x.w, z);
            }
            if (not_finite<W8>(z) || not_finite<W8>(z >> 16)) {
              int e = 0;  // which of the run's edge tiles this is
              for (int k = 0; k < i; ++k)
                e += chunk_edge(a, run, run.tiles[run.i0 + k] * kTok, kTok) ? 1 : 0;
              if (e < kEdgeTiles) atomicOr(&bad[4 * e + (r >> 5)], 1u << (r & 31));
              __threadfence_block();
#pragma unroll 1
              for (int c = 0; c < CH; ++c) {
                uint4 x = lds128(chunk_at(c));
                uint32_t* w = &x.x;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                  if (not_finite<W8>(w[k])) w[k] &= 0xffff0000u;
                  if (not_finite<W8>(w[k] >> 16)) w[k] &= 0xffffu;
                }
                sts128(chunk_at(c), x);
              }
            }
          }
          fence_proxy_async_smem();
        }
        float mx4[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) mx4[k] = __uint_as_float(sr[k]);
#pragma unroll
        for (int k = 4; k < 60; k += 8) {
#pragma unroll
          for (int m = 0; m < 4; ++m)
            mx4[m] = max3(mx4[m], __uint_as_float(sr[k + 2 * m]), __uint_as_float(sr[k + 2 * m + 1]));
        }
        float mx = max3(max3(mx4[0], mx4[1], mx4[2]),
                        max3(mx4[3], __uint_as_float(sr[60]), __uint_as_float(sr[61])),
                        fmaxf(__uint_as_float(sr[62]), __uint_as_float(sr[63])));
        if constexpr (!FORM) mx *= sc;
        mx = fmaxf(mx, exchange(mx));  // (both halves' scores have left S, where P goes)
        if (!ok) break;
        // s sc - m is one FMA below: m is a rounded product, the product in the FMA is not, so that a row's
        // weights are all off by one factor, which their sum shares: up to 2^0.5 for |m| <= 2^24. For
        // larger m it would soon leave f16's range and then every range: there s sc is rounded as m is.
        // (A tile that counts has its maximum near m.)
        const bool huge = !FORM && fabsf(mx) > 0x1p24f && mx != -INFINITY;
        // The reference that P and O are scaled by: from the first tile's maximum, then moved only when
        // passed by far (the difference, not a sum: past 2^26 that would round to several times as far).
        const bool first = i == i_first;
        const bool moved = !first && mx - m_used > kLazyLog2<W8> + kLiftLog2<W8>;
        float factor = FORM ? 1.f : sc;
        if (__any_sync(0xffffffffu, moved || huge)) {  // (one vote for the two: most steps have neither)
          if (__any_sync(0xffffffffu, moved)) {
            // rescale half the dims of this warp's rows of O: this step's S was issued after the last
            // P V, and is there
            const float m_new = moved ? mx - kLiftLog2<W8> : m_used;
            const float alpha = moved ? exp2f(m_used - m_new) : 1.f;
#pragma unroll 1
            for (int c = h * (D / 2); c < (h + 1) * (D / 2); c += 16) {
              uint32_t o[16];
              tmem_ld16(ocol + c, o);
              tmem_wait_ld();
#pragma unroll
              for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * alpha);
              tmem_st16(ocol + c, o);
            }
            l *= alpha;
            m_used = m_new;
          }
          if (__any_sync(0xffffffffu, huge)) {
#pragma unroll
            for (int k = 0; k < 64; ++k)
              sr[k] = __float_as_uint(__fmul_rn(__uint_as_float(sr[k]), sc));
            factor = 1.f;
          }
        }
        if (first) m_used = mx - kLiftLog2<W8>;
        // P = 2^(s - m), the two halves over the first 64 columns of S
        const float m_use = m_used == -INFINITY ? 0.f : m_used;
        uint64_t sum[4] = {0, 0, 0, 0};  // (pairs of zeros)
        const uint64_t sc2 = pack2(factor, factor), m2 = pack2(-m_use, -m_use);
        uint32_t pw[32];
#pragma unroll
        for (int k = 0; k < 32; ++k) {
          float e0, e1;
          unpack2(fma2(pack2(__uint_as_float(sr[2 * k]), __uint_as_float(sr[2 * k + 1])), sc2, m2),
                  e0, e1);
          e0 = ex2_approx(e0);
          e1 = ex2_approx(e1);
          sum[k & 3] = add2(sum[k & 3], pack2(e0, e1));
          pw[k] = pack_p<W8>(e0, e1);
        }
        tmem_st32(pcol, pw);
        float s0, s1;
        unpack2(add2(add2(sum[0], sum[1]), add2(sum[2], sum[3])), s0, s1);
        l += s0 + s1;
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();  // (one arrival per warp: arrivals on one barrier go one by one)
        if (lane == 0) mbar_arrive(&p_ready[wg]);
        at.advance(stride);
      }
      // ---- the run's rows ----
      // the next run's queries first, so that its first scores run while this one's rows are written
      if (!any || !ok) {
        after = get_run(unit + 1);
        if (after) {
          then = find_row(*after);
          load_query(*after, then);
        }
      }
      if (after) store_query(*after);
      if (ok && any) {
        ok = mbar_wait(&o_done[wg], ph_o, a.err);
        ok = __all_sync(0xffffffffu, ok);
      }
      if (any) ph_o ^= 1u;
      tc_fence_after();
      // The row's maximum and sum; wide: over the group's two halves, and warp (group, h) writes dims
      // h D/2 .. of its rows; else over both groups' halves, and it writes dims 32 (2 group + h) ...
      float M = m_used, L, w0 = 1.f, w1 = 0.f;
      if (wide) {
        const float x = exchange(l);
        L = h == 0 ? l + x : x + l;
        __syncwarp();
        if (lane == 0) mbar_arrive(pair);  // (read: waited for below)
      } else {
        *mine = l;
        if (h == 0) row_max[wg * kGroupRows + r] = m_used;
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(met);
        ok = mbar_wait(met, ph_met, a.err) && ok;
        ok = __all_sync(0xffffffffu, ok);
        tc_fence_after();
        const float m0 = row_max[r], m1 = row_max[kGroupRows + r];
        M = fmaxf(m0, m1);
        const float Mu = M == -INFINITY ? 0.f : M;
        w0 = exp2f(m0 - Mu);
        w1 = exp2f(m1 - Mu);
        L = w0 * (half_row[r] + half_row[kGroupRows + r]) +
            w1 * (half_row[2 * kGroupRows + r] + half_row[3 * kGroupRows + r]);
      }
      const float vs = W8 ? a.v_scales[run.j] : 1.f;
      const float f = run.whole ? (L != 0.f ? vs / L : 0.f) : vs;
      const bool none = run.whole && L == 0.f;
      const bool any_bad = __any_sync(0xffffffffu, bad[lane] != 0);
      const size_t part0 = ((size_t)blockIdx.x * 2 + run.slot) * kChunkTcRows;
      if (ok && live && h == 0 && (wide || wg == 0)) {
        if (!run.whole)
          *reinterpret_cast<float2*>(a.ws_ml + 2 * (part0 + me.row)) = make_float2(M, L);
        else if (a.lse)
          a.lse[me.at] = L != 0.f ? (M + log2f(L)) * kLn2 : -INFINITY;
      }
      // O in blocks of 16 rows x 32 dims: a lane has dims 8 n + 2 (lane % 4) + {0, 1}, n < 4, of rows
      // lane / 4 and lane / 4 + 8, so that four lanes write a row's 64 (bf16) or 32 (fp32) consecutive
      // bytes
      const int c_lo = wide ? h * (D / 2) : 32 * (2 * wg + h);
      const int c_hi = min(D, c_lo + (wide ? D / 2 : 32));
      const int q4 = lane & 3;
      for (int b16 = 0; ok && c_lo < D && b16 < 2; ++b16) {
        if (!__any_sync(0xffffffffu, live && (lane >> 4) == b16)) break;  // (rows are in order)
        // (with the rows' factors, offsets, parts)
        const int ra = 16 * b16 + (lane >> 2), rb = ra + 8;
        const float fa = __shfl_sync(0xffffffffu, f, ra), fb = __shfl_sync(0xffffffffu, f, rb);
        const float w0a = __shfl_sync(0xffffffffu, w0, ra), w0b = __shfl_sync(0xffffffffu, w0, rb);
        const float w1a = __shfl_sync(0xffffffffu, w1, ra), w1b = __shfl_sync(0xffffffffu, w1, rb);
        const size_t at_a = __shfl_sync(0xffffffffu, (unsigned long long)me.at, ra);
        const size_t at_b = __shfl_sync(0xffffffffu, (unsigned long long)me.at, rb);
        const uint32_t lives = __ballot_sync(0xffffffffu, live);
        const uint32_t nones = __ballot_sync(0xffffffffu, none);
        const bool live_a = (lives >> ra) & 1, live_b = (lives >> rb) & 1;
        const bool none_a = (nones >> ra) & 1, none_b = (nones >> rb) & 1;
        for (int c = c_lo; c < c_hi; c += 32) {
          uint32_t o[16];
          const uint32_t rows_t = ((uint32_t)(16 * b16) << 16) + c;
          tmem_ld_16x256(( wide ? ocol : lane_t) + rows_t, o);
          tmem_wait_ld();
          if (!wide && run.n > 1) {
            uint32_t o1[16];
            tmem_ld_16x256(lane_t + 128 + rows_t, o1);
            tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              const float x0 = k & 2 ? w0b : w0a, x1 = k & 2 ? w1b : w1a;
              o[k] = __float_as_uint(x0 * __uint_as_float(o[k]) + x1 * __uint_as_float(o1[k]));
            }
          }
          if (any_bad) {  // the infinite and NaN values of the positions that a row sees
            const int pq_a = __shfl_sync(0xffffffffu, me.pq, ra), pq_b = __shfl_sync(0xffffffffu, me.pq, rb);
            int e = 0;
            for (int k = 0; k < run.n && e < kEdgeTiles; ++k) {
              const int q0 = run.tiles[run.i0 + k] * kTok;
              if (!chunk_edge(a, run, q0, kTok)) continue;
              for (int x = 0; x < kTok; ++x) {
                if (!((bad[4 * e + (x >> 5)] >> (x & 31)) & 1)) continue;
                const int pos = q0 + x;
                const bool see_a = chunk_seen(a, pq_a, pos) & 1, see_b = chunk_seen(a, pq_b, pos) & 1;
                const int id = a.block_tables[(size_t)run.b * a.max_pages + pos / kPageSize];
                const uint8_t* v = static_cast<const uint8_t*>(a.v_cache) +
                                   ((((int64_t)id * a.h_kv + run.j) * kPageSize + pos % kPageSize) * D +
                                    c + 2 * q4) * KV::bytes;
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                  float y[2];
                  RowLoad<KV, 2>::run(v + 8 * n * KV::bytes, y);
#pragma unroll
                  for (int m = 0; m < 2; ++m) {
                    if (fabsf(y[m]) < INFINITY) continue;
                    if (see_a) o[4 * n + m] = __float_as_uint(__uint_as_float(o[4 * n + m]) + y[m]);
                    if (see_b) o[4 * n + 2 + m] = __float_as_uint(__uint_as_float(o[4 * n + 2 + m]) + y[m]);
                  }
                }
              }
              ++e;
            }
          }
          if (run.whole) {
            uint32_t va[4], vb[4];
#pragma unroll
            for (int n = 0; n < 4; ++n) {
              va[n] = none_a ? 0u : pack_bf16(__uint_as_float(o[4 * n]) * fa,
                                              __uint_as_float(o[4 * n + 1]) * fa);
              vb[n] = none_b ? 0u : pack_bf16(__uint_as_float(o[4 * n + 2]) * fb,
                                              __uint_as_float(o[4 * n + 3]) * fb);
            }
            quad_transpose(va, q4);
            quad_transpose(vb, q4);
            __nv_bfloat16* const out = static_cast<__nv_bfloat16*>(a.out) + c + 8 * q4;
            if (live_a)
              *reinterpret_cast<uint4*>(out + at_a * D) = make_uint4(va[0], va[1], va[2], va[3]);
            if (live_b)
              *reinterpret_cast<uint4*>(out + at_b * D) = make_uint4(vb[0], vb[1], vb[2], vb[3]);
          } else {
            const int first_row = me.row - lane;  // (of the warp)
            float* const out = a.ws_acc + c + 2 * q4;
#pragma unroll
            for (int n = 0; n < 4; ++n) {
              if (live_a)
                *reinterpret_cast<float2*>(out + (part0 + first_row + ra) * D + 8 * n) = make_float2(
                    __uint_as_float(o[4 * n]) * fa, __uint_as_float(o[4 * n + 1]) * fa);
              if (live_b)
                *reinterpret_cast<float2*>(out + (part0 + first_row + rb) * D + 8 * n) = make_float2(
                    __uint_as_float(o[4 * n + 2]) * fb, __uint_as_float(o[4 * n + 3]) * fb);
            }
          }
        }
      }
      if (wide) {  // the other warp has read this one's sums
        ok = mbar_wait(pair, ph_pair, a.err) && ok;
        ok = __all_sync(0xffffffffu, ok);
        ph_pair ^= 1u;
      } else {  // the other group reads this one's O and sums
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(parted);
        ok = mbar_wait(parted, ph_met, a.err) && ok;
        ok = __all_sync(0xffffffffu, ok);
        tc_fence_after();
        ph_met ^= 1u;
      }
      base.skip(run.n);
      me = then;
      next = after;
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  release();
}

template <typename KV, int D, bool FORM>
cudaError_t launch_shape(const ChunkArgs& a, const CUtensorMap& tk, const CUtensorMap& tv,
                         cudaStream_t s) {
  using S = TcShape<KV, D>;
  static std::atomic<unsigned long long> attr_done{0};  // one bit per device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !((attr_done.load() >> dev) & 1ull)) {
    e = cudaFuncSetAttribute(chunk_tc_kernel<KV, D, FORM>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             S::SMEM);
    if (e != cudaSuccess) return e;
    // the softmax warps may take no more registers than the launch brings and the others give up
    cudaFuncAttributes fa{};
    e = cudaFuncGetAttributes(&fa, chunk_tc_kernel<KV, D, FORM>);
    if (e != cudaSuccess) return e;
    if (fa.numRegs < S::LAUNCH_REGS) return cudaErrorLaunchOutOfResources;
    if (dev < 64) attr_done.fetch_or(1ull << dev);
  }
  chunk_tc_kernel<KV, D, FORM><<<a.ctas, S::THREADS, S::SMEM, s>>>(a, tk, tv);
  return cudaGetLastError();
}

template <typename KV, int D>
cudaError_t launch_t(const ChunkArgs& a, const CUtensorMap& tk, const CUtensorMap& tv,
                     cudaStream_t s) {
  return a.softcap > 0.f || a.slopes ? launch_shape<KV, D, true>(a, tk, tv, s)
                                     : launch_shape<KV, D, false>(a, tk, tv, s);
}

}  // namespace

cudaError_t launch_chunk_tc(const ChunkArgs& a, int kv_dtype, int head_dim, const void* tk,
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
