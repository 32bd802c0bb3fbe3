// Sums of attention weights on the fifth-generation tensor cores (tcgen05), bf16 queries over a bf16, FP8
// or INT8 cache; the mathematics is that of chunk_weights.cu, the work is cut as weigh_plan.cuh says, in
// items of 256 positions of one KV head and steps of 128 (token, query head) rows, one persistent CTA
// per SM.
//
// The scores come transposed, S^T = K Q^T with the positions as the MMA's 128 rows and the queries as its
// columns, so that a thread owns a position and its sum never leaves the thread: no exchange between
// lanes, no atomics. A step of both halves of an item is 2 x 512 cycles of MMAs at D = 128, reads 32 KB of
// queries from L2 (with 128 positions an item it would be twice that for the same work, 64 bytes a
// clock and SM), and 2 x 512 cycles of exponentials:
//
//  * a copy warp streams the tiles' K by TMA (bf16) or as codes that four converter warps widen to f16;
//  * four loader warps bring the rows' queries into shared memory in MMA form and each row's numbers: minus
//    its lse, its score factor, slope and position. The queries come by TMA where a step's rows are whole
//    tokens (a bf16 cache, a group that divides 128: 92 us instead of 97 for 4095 rows over themselves),
//    else by copies of 16 bytes; for 8-bit caches they are then made f16, scaled by a row's power of two;
//  * one MMA warp; four groups of four warps that add up weights: group 2 q + h takes half h of the item
//    in every second step, reading S^T from its own 128 columns of tensor memory, 32 at a time.
//
// 4095 prompt rows over themselves, 32 query heads on 8, bf16: 81 us for 69 GFLOP, 0.85 PFLOP/s (the rings
// and MMAs alone, without the sums, took 62).
//
// A wait for a phase by its parity means something only to a warp that has seen the phase before end. So
// every warp of the sums waits for both halves' K, though it needs one; the rows' numbers have a ring for even
// and one for odd steps; and each warp gives a run's place back (items without rows take no place in any
// ring, so nothing else would keep the copy warp from lapping a slow reader).
//
// A step's weights are summed in eight chains of 16 and join the position's sum by a compensated addition
// (Kahan's), so that sums over thousands of rows are good to fp32. Every wait is bounded
// (PKV_DEVERR_TIMEOUT); the tensor memory is freed on every path.
#include <atomic>
#include <climits>
#include <cuda.h>
#include <math.h>
#include <type_traits>

#include "chunk_score.cuh"
#include "paged_decode_mma.cuh"
#include "pkv_device.cuh"
#include "pkv_internal.h"
#include "tc_pipe.cuh"
#include "tcgen05.cuh"
#include "weigh_plan.cuh"

namespace pkv {

namespace {

constexpr int kItem = kWeighTcTokens;      // positions of an item: two halves
constexpr int kHalf = 128;                 // positions of a half: one tile of K
constexpr int kStep = kWeighTcRows;        // rows of a step
constexpr int kPages = kHalf / kPageSize;  // pages of a half
constexpr int kGroupThreads = 128;
constexpr int kSumThreads = 4 * kGroupThreads;
constexpr int kMmaWarp = kSumThreads / 32;
constexpr int kCopyWarp = kMmaWarp + 1;
constexpr int kLoadWarp = kMmaWarp + 4;    // first of four (two warps before are idle)
constexpr int kConvWarp = kLoadWarp + 4;   // first of four (8-bit caches)
constexpr int kCols = 4;                   // steps whose rows' numbers are kept: two even, two odd
constexpr int kRuns = 16;
constexpr uint32_t kTmemCols = 512;        // S^T of group g at 128 g
static_assert(kItem == 2 * kHalf && kStep == 128, "two halves, M = 128, N = 128");

template <typename KV, int D>
struct WeighTcShape {
  static constexpr bool W8 = KV::bytes == 1;
  static constexpr int THREADS = 32 * (W8 ? kConvWarp + 4 : kConvWarp);
  // Registers: the block's at launch, and the warps' own: those of the sums take what the others leave.
  static constexpr int LAUNCH_REGS = W8 ? 72 : 80, SUM_REGS = W8 ? 88 : 96, REGS = 48;
  static_assert(kSumThreads * SUM_REGS + (THREADS - kSumThreads) * REGS <= THREADS * LAUNCH_REGS,
                "the block's own registers");
  static constexpr int TILE = kHalf * D * 2;  // K of a half, or the queries of a step, in MMA form
  static constexpr int NK = D == 128 ? 3 : 6, NQ = D == 128 ? (W8 ? 2 : 3) : 4;
  static constexpr uint32_t IDESC = tc_idesc(128, 0, false, W8);  // (N: the step's columns)
  static constexpr int RAW = kHalf / 2 * D;   // codes of half a tile
  static constexpr int NR = W8 ? 6 : 0;
  static constexpr int OFF_Q = NK * TILE;
  static constexpr int OFF_RAW = OFF_Q + NQ * TILE;
  static constexpr int OFF_COL = OFF_RAW + NR * RAW;        // [kCols][4][128] a step's rows' numbers
  static constexpr int OFF_SUM = OFF_COL + kCols * 4 * kStep * 4;  // [2][256] the second steps' sums
  static constexpr int OFF_BAR = OFF_SUM + 2 * kItem * 4;
  static constexpr int BARS = 2 * NK + 2 * NQ + 2 * NR + 2 * 4 + 2 * kCols + 8 + 1 + 2 * kRuns;
  static constexpr int READERS = kSumThreads / 32 + 1 + 4 + (W8 ? 4 : 0);  // warps that follow the runs
  static constexpr int OFF_MISC = OFF_BAR + 8 * BARS;       // masks, TMEM address
  static constexpr int SMEM = 1024 + OFF_MISC + 4 * (NK + NR + 1) + 16;
  static_assert(SMEM <= 224 * 1024 && SMEM > 114 * 1024, "one CTA per SM");
};

constexpr float kNanLse = 0x1p127f;  // stands for minus a NaN lse: an infinite weight wherever seen

// A step's rows' numbers in shared memory.
struct Columns {
  const float* neg_lse;  // log2 domain; -inf where there is no row, or its lse is -inf; kNanLse
  const float* factor;   // scores (log2 domain) are factor times the product (8-bit caches: a row's own)
  const float* slope;    // log2 domain
  const int* pos;        // the row's position
};
template <typename T>
__device__ __forceinline__ Columns columns(T* base, int st) {
  float* p = reinterpret_cast<float*>(base) + st * 4 * kStep;
  return Columns{p, p + kStep, p + 2 * kStep, reinterpret_cast<const int*>(p + 3 * kStep)};
}

template <typename KV, int D, bool FORM>
__global__ void __launch_bounds__(WeighTcShape<KV, D>::THREADS, 1) weights_tc_kernel(
    const ChunkArgs a, const __grid_constant__ CUtensorMap tm_k,
    const __grid_constant__ CUtensorMap tm_q) {
  using S = WeighTcShape<KV, D>;
  constexpr bool W8 = S::W8;
  constexpr int NK = S::NK, NQ = S::NQ, NR = S::NR;
  constexpr int PAGE_MMA = kPageSize * D * 2, PAGE_RAW = kPageSize * D;
  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t ring = smem_u32(smem);
  uint64_t* full_k = reinterpret_cast<uint64_t*>(smem + S::OFF_BAR);  // [NK] K of a half is there
  uint64_t* free_k = full_k + NK;                                    // [NK] its last S done
  uint64_t* full_q = free_k + NK;                                    // [NQ] queries of a step
  uint64_t* free_q = full_q + NQ;                                    // [NQ] their S done
  uint64_t* raw_full = free_q + NQ;                                  // [NR] codes arrived
  uint64_t* raw_freed = raw_full + NR;                               // [NR] codes in registers
  uint64_t* s_done = raw_freed + NR;                                 // [4] S of a group's step
  uint64_t* s_read = s_done + 4;                                     // [4] it is in registers
  uint64_t* full_c = s_read + 4;                                     // [kCols] the rows' numbers
  uint64_t* free_c = full_c + kCols;                                 // [kCols] used up
  uint64_t* handed = free_c + kCols;                                 // [2][half] second steps' sums
  uint64_t* taken = handed + 4;                                      // [2][half] read
  uint64_t* mma_idle = taken + 4;
  uint64_t* run_there = mma_idle + 1;                                // [kRuns]
  uint64_t* run_gone = run_there + kRuns;                            // [kRuns] its place is free again
  int* page_mask = reinterpret_cast<int*>(smem + S::OFF_MISC);       // [NK] good pages of the half
  int* raw_mask = page_mask + NK;                                    // [NR]
  uint32_t* s_taddr = reinterpret_cast<uint32_t*>(raw_mask + NR);
  uint8_t* const col = smem + S::OFF_COL;
  float* const hand = reinterpret_cast<float*>(smem + S::OFF_SUM);

  __shared__ int scratch[32];
  __shared__ WeighShare share;
  __shared__ WeighRun runs[kRuns];  // (n = 0: the share's end)
  __shared__ uint32_t no_lse[kCols][4];  // of a step's rows, bits: its lse is -inf
  // whether there is one among 32 rows; one whose lse is NaN
  __shared__ __align__(4) uint8_t some_none[kCols][4], some_nan[kCols][4];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (threadIdx.x == kCopyWarp * 32) {
    for (int s = 0; s < NK; ++s) {
      mbar_init(&full_k[s], W8 ? 4 : 1);
      mbar_init(&free_k[s], 1 + kSumThreads / 32);  // the MMAs and every warp of the sums
    }
    for (int s = 0; s < NQ; ++s) {
      mbar_init(&full_q[s], 4);
      mbar_init(&free_q[s], 1);
    }
    for (int s = 0; s < NR; ++s) {
      mbar_init(&raw_full[s], 1);
      mbar_init(&raw_freed[s], 4);
    }
    for (int g = 0; g < 4; ++g) {
      mbar_init(&s_done[g], 1);
      mbar_init(&s_read[g], 4);
    }
    for (int s = 0; s < kCols; ++s) {
      mbar_init(&full_c[s], 4);
      mbar_init(&free_c[s], 8);  // the two groups of the step
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&handed[i], 4);
      mbar_init(&taken[i], 4);
    }
    mbar_init(mma_idle, 1);
    for (int i = 0; i < kRuns; ++i) {
      mbar_init(&run_there[i], 1);
      mbar_init(&run_gone[i], S::READERS);
    }
    mbar_fence_init();
    if constexpr (!W8)
      if (a.num_rows > 0)  // (else there is no map)
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tm_k)) : "memory");
  }
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(s_taddr)),
                 "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  weigh_share<S::THREADS>(a, scratch, &share);
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
    if (threadIdx.x == 0) static_cast<WeighRecord*>(a.ws_rec)[blockIdx.x] = WeighRecord{0, 0, 0, 0};
    release();
    return;
  }
  // run i of the share, or nullptr after the last (or a wait that gave up); run i - 2 is done with
  auto get_run = [&](uint32_t i) -> const WeighRun* {
    const bool got = mbar_wait(&run_there[i % kRuns], (i / kRuns) & 1u, a.err);
    const WeighRun* r = &runs[i % kRuns];
    if (i >= 2 && lane == 0) mbar_arrive(&run_gone[(i - 2) % kRuns]);
    return __all_sync(0xffffffffu, got && r->n > 0) ? r : nullptr;
  };
  // Step u of a run (from its first on) belongs to the groups 2 (u % 2) + h; a run without rows has no
  // steps here, and one whose positions end in the first half no half 1.
  auto steps_of = [](const WeighRun* r) { return r->rows > 0 ? uniform(r->n) : 0; };
  auto halves_of = [](const WeighRun* r) {
    return uniform(r->req.base + r->req.n - r->item * kItem) > kHalf ? 2 : 1;
  };

  if (warp >= kMmaWarp && warp < kLoadWarp) {
    regs_down<S::REGS>();
    if (warp == kCopyWarp) {
      // ===================== copies of K, half by half =====================
      const uint64_t pol = l2_evict_first_policy();
      constexpr int stages = W8 ? NR : NK;
      uint64_t* const there = W8 ? raw_full : full_k;
      uint64_t* const gone = W8 ? raw_freed : free_k;
      int st = 0, issued = 0;
      uint32_t par = 0;
      bool ok = true;
      WeighWalk walk(a, share);
      WeighRecord record{0, 0, 0, 0};
      for (uint32_t unit = 0;; ++unit) {
        WeighRun* run = &runs[unit % kRuns];
        if (lane == 0) {  // (a wait that gave up ends the share for every warp)
          // (items without rows take no place in the rings: nothing else holds this warp back there)
          if (unit >= kRuns)
            ok = mbar_wait(&run_gone[unit % kRuns], (unit / kRuns - 1) & 1u, a.err) && ok;
          if (!ok || !walk.next(a, *run)) run->n = 0;
          mbar_arrive(&run_there[unit % kRuns]);
        }
        __syncwarp();
        if (run->n == 0) break;
        const int j = uniform(run->j), first = uniform(run->req.base + run->t0);
        const int ctx = uniform(run->req.base + run->req.n), item0 = uniform(run->item) * kItem;
        if (!run->whole && run->slot == 1)
          record = WeighRecord{run->b * a.h_kv + j, item0, min(kItem, ctx - item0), run->shares};
        if (steps_of(run) == 0) continue;
        const int32_t* table = a.block_tables + (size_t)uniform(run->b) * a.max_pages;
        const int halves = halves_of(run);
        // lane p: the id of page p of the item; -1 where it is not read, -2 where it is but has no id
        const int p0 = item0 + (lane & 15) * kPageSize;
        int mine = -1;
        // (a page outside every row's window may have been given back: it is not read)
        if (p0 < ctx && (a.window <= 0 || p0 < a.sink || p0 + kPageSize > first + 1 - a.window)) {
          const int id = table[p0 / kPageSize];
          mine = id >= 0 && id < a.num_pages ? id : -2;
        }
        const uint32_t all = __ballot_sync(0xffffffffu, mine >= 0);
        if (__any_sync(0xffffffffu, mine == -2) && lane == 0) atomicOr(a.err, PKV_DEVERR_BAD_PAGE);
        // a stage: K of a half (bf16), or the codes of a quarter
        constexpr int PART = W8 ? kPages / 2 : kPages;
#pragma unroll 1
        for (int part = 0; part < halves * (kPages / PART); ++part) {
          if (issued >= stages) {
            ok = __all_sync(0xffffffffu, mbar_wait(&gone[st], par ^ 1u, a.err));
            if (!ok) break;
          }
          int id[PART];
          const uint32_t m = (all >> (part * PART)) & ((1u << PART) - 1);
#pragma unroll
          for (int p = 0; p < PART; ++p) id[p] = __shfl_sync(0xffffffffu, mine, part * PART + p);
          if (elect_one()) {
            if constexpr (W8) {
              raw_mask[st] = (int)m;
              fence_proxy_async_smem();
              mbar_arrive_expect_tx(&there[st], __popc(m) * PAGE_RAW);
#pragma unroll
              for (int p = 0; p < PART; ++p)
                if ((m >> p) & 1)
                  bulk_g2s(smem + S::OFF_RAW + st * S::RAW + p * PAGE_RAW,
                           static_cast<const uint8_t*>(a.k_cache) +
                               ((int64_t)id[p] * a.h_kv + j) * PAGE_RAW,
                           PAGE_RAW, &there[st], pol);
            } else {
              page_mask[st] = (int)m;
              mbar_arrive_expect_tx(&there[st], __popc(m) * PAGE_MMA);
#pragma unroll
              for (int p = 0; p < PART; ++p) {
                if (!((m >> p) & 1)) continue;
                const int row = (id[p] * a.h_kv + j) * kPageSize;
#pragma unroll
                for (int bx = 0; bx < D / 64; ++bx)
                  tma_load_2d(ring + st * S::TILE + bx * (kHalf * 128) + p * 2048, &tm_k, bx * 64,
                              row, &there[st], pol);
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
      }
      if (lane == 0) {
        static_cast<WeighRecord*>(a.ws_rec)[blockIdx.x] = record;
        for (int t = max(0, issued - stages); t < issued; ++t)  // every copy issued has landed
          mbar_wait(&there[t % stages], (uint32_t)(t / stages) & 1u, a.err);
      }
    } else if (warp == kMmaWarp) {
      // ===================== MMAs (one elected lane issues) =====================
      const uint64_t k_desc = tc_desc(ring, 16, 1024), q_desc = tc_desc(ring + S::OFF_Q, 16, 1024);
      bool ok = true;
      uint32_t uses = 0, seen = 0;  // bit g: parity of the group's next s_read; whether there was one
      Place<NK> ks;
      Place<NQ> qs;
      auto wait = [&](uint64_t* bar, uint32_t par) {
        const bool got = __all_sync(0xffffffffu, mbar_wait(bar, par, a.err));
        tc_fence_after();
        return got;
      };
      for (uint32_t unit = 0; ok; ++unit) {
        const WeighRun* run = get_run(unit);
        if (!run) break;
        const int n = steps_of(run), halves = halves_of(run);
        const int rows = uniform(run->rows - run->s0 * kStep);
        if (n == 0) continue;
        Place<NK> k1 = ks;
        k1.advance(1);
        for (int u = 0; ok && u < n; ++u) {
          const int q = u & 1;
          // columns in use, in blocks of 32
          const int cols = min(kStep, (rows - u * kStep + 31) & ~31);
          const uint32_t idesc = S::IDESC | ((uint32_t)(cols >> 3) << 17);
          ok = wait(&full_q[qs.st], qs.par);
          for (int h = 0; ok && h < halves; ++h) {
            const Place<NK>& k = h ? k1 : ks;
            const int g = 2 * q + h;
            if (u == 0) ok = wait(&full_k[k.st], k.par);
            if (ok && ((seen >> g) & 1)) {  // the group has read the last S there
              ok = wait(&s_read[g], (uses >> g) & 1u);
              uses ^= 1u << g;
            }
            seen |= 1u << g;
            if (!ok) break;
            const uint64_t kd = k_desc + (uint32_t)(k.st * (S::TILE >> 4));
            const uint64_t qd = q_desc + (uint32_t)(qs.st * (S::TILE >> 4));
            if (elect_one()) {
#pragma unroll
              for (int kk = 0; kk < D / 16; ++kk) {
                const uint32_t at = ((kk >> 2) * (kHalf * 128) + (kk & 3) * 32) >> 4;
                tc_mma_sa(tmem + 128 * g, kd + at, qd + at, idesc, kk > 0 ? 1u : 0u);
              }
              tc_commit(&s_done[g]);
              if (h == halves - 1) tc_commit(&free_q[qs.st]);
              if (u == n - 1) tc_commit(&free_k[k.st]);
            }
            __syncwarp();
          }
          qs.advance(1);
        }
        ks.advance(halves);
      }
      if (elect_one()) tc_commit(mma_idle);  // before leaving, every MMA issued is complete
      __syncwarp();
      wait(mma_idle, 0);
    }
  } else if (warp >= kLoadWarp && warp < kConvWarp) {
    // ===================== queries and the rows' numbers =====================
    regs_down<S::REGS>();
    // A step's loads are issued before the step ahead of it is waited for, if there is a place for them
    // yet, whatever runs they belong to.
    // Four lanes copy 64 consecutive bytes of a row; for an 8-bit cache they then make f16 of the row in
    // its place.
    const int w = warp - kLoadWarp, r = 32 * w + lane;  // this lane's row of a step
    const int row0 = 32 * w + (lane >> 2);              // it copies pieces of rows row0 + 8 g
    constexpr int RND = D / 32;
    bool ok = true;
    struct Step {
      const WeighRun* run;
      int u, pos;                 // step of the run; position of this lane's row
      float lse, slope, k_scale;  // (as they come: used when the step is finished)
    };
    uint32_t unit = 0;
    auto next_run = [&](Step& x) {  // to the first step of the next run that has any, or nullptr
      do {
        x.run = get_run(unit++);
      } while (x.run && steps_of(x.run) == 0);
      x.u = 0;
    };
    auto q_chunk = [&](int st, int d, int g) {
      return ring + S::OFF_Q + st * S::TILE + row0 * 128 + (d >> 1) * (kStep * 128) + g * 1024 +
             ((((4 * d & 7) + (lane & 3)) ^ (row0 & 7)) << 4);
    };
    Place<NQ> q_in, q_out;
    uint32_t used[2] = {0, 0};  // places taken for even and odd steps of runs
    int issued = 0;
    auto issue = [&](Step& x) {
      if (issued >= NQ) ok = __all_sync(0xffffffffu, mbar_wait(&free_q[q_in.st], q_in.par ^ 1u, a.err));
      if (!ok) return;
      const WeighRun& run = *x.run;
      const unsigned first = (unsigned)(run.s0 + x.u) * kStep, R = first + r;
      const bool live = R < (unsigned)run.rows;
      const unsigned t = live ? R / (unsigned)a.group : 0, g = live ? R - t * a.group : 0;
      const size_t at = (size_t)(run.req.q0 + run.t0 + (int)t) * a.h_q + run.j * a.group + g;
      x.lse = live ? a.lse[at] : INFINITY;  // (gives nothing)
      x.slope = FORM && a.slopes ? a.slopes[run.j * a.group + g] : 0.f;
      x.k_scale = W8 ? a.k_scales[run.j] : 1.f;
      x.pos = run.req.base + run.t0 + (int)t;
      if (!W8 && a.step_tokens > 0) {  // the step's tokens in a box for each 64 dims, by the first warp
        if (w == 0 && elect_one()) {
          mbar_arrive_expect_tx(&full_q[q_in.st], kStep * D * 2);
          const int token = run.req.q0 + run.t0 + (run.s0 + x.u) * a.step_tokens;
#pragma unroll
          for (int bx = 0; bx < D / 64; ++bx)
            tma_load_box(ring + S::OFF_Q + q_in.st * S::TILE + bx * (kStep * 128), &tm_q, bx * 64,
                         run.j * a.group, token, &full_q[q_in.st]);
        }
        __syncwarp();
      } else if (32 * w < run.rows - (int)first) {  // (columns beyond the last block of 32 are not used)
#pragma unroll
        for (int g4 = 0; g4 < 4; ++g4) {
          const int from = 8 * g4 + (lane >> 2);
          const size_t src_at = __shfl_sync(0xffffffffu, (unsigned long long)at, from);
          const bool there = __shfl_sync(0xffffffffu, (int)live, from) != 0;
          const __nv_bfloat16* src =
              static_cast<const __nv_bfloat16*>(a.q) + src_at * D + 8 * (lane & 3);
#pragma unroll
          for (int d = 0; d < RND; ++d)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(q_chunk(q_in.st, d, g4)),
                         "l"(src + 32 * d), "r"(there ? 16 : 0)
                         : "memory");
        }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
      ++issued;
      q_in.advance(1);
    };
    auto finish = [&](const Step& x) {
      // (a ring for each pair of groups, so that a group sees every phase of its barriers)
      const int q = x.u & 1;
      const uint32_t use = q ? used[1] : used[0];
      const int cs = 2 * q + (int)(use & 1u);
      if (use >= 2)
        ok = __all_sync(0xffffffffu, mbar_wait(&free_c[cs], ((use >> 1) & 1u) ^ 1u, a.err));
      if (!ok) return;
      const float sc = a.scale * kLog2e * x.k_scale;
      float* const p = reinterpret_cast<float*>(col) + cs * 4 * kStep;
      // A row that saw nothing gives nothing: -inf. One whose lse is NaN gives an infinite weight to what
      // it sees, which the sums then call NaN (NaN itself would also reach what it does not see: those
      // scores are -inf).
      p[r] = x.lse != x.lse ? kNanLse : x.lse == -INFINITY ? -INFINITY : -x.lse * kLog2e;
      const uint32_t none = __ballot_sync(0xffffffffu, x.lse == -INFINITY);
      const bool nan = __any_sync(0xffffffffu, x.lse != x.lse);
      if (lane == 0) {
        no_lse[cs][w] = none;
        some_none[cs][w] = none != 0;
        some_nan[cs][w] = nan;
      }
      if constexpr (FORM) p[2 * kStep + r] = x.slope * kLog2e;
      reinterpret_cast<int*>(p)[3 * kStep + r] = x.pos;
      if constexpr (W8) {
        if (32 * w < x.run->rows - (x.run->s0 + x.u) * kStep) {
#pragma unroll
          for (int g4 = 0; g4 < 4; ++g4) {
            uint4 in[RND];
#pragma unroll
            for (int d = 0; d < RND; ++d) in[d] = lds128(q_chunk(q_out.st, d, g4));
            const float f = query_to_f16<RND>(in, sc);
#pragma unroll
            for (int d = 0; d < RND; ++d) sts128(q_chunk(q_out.st, d, g4), in[d]);
            if ((lane & 3) == 0) p[kStep + row0 + 8 * g4] = f;
          }
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        if (W8 || a.step_tokens == 0 || w > 0) mbar_arrive(&full_q[q_out.st]);  // (else: its copy's word)
        mbar_arrive(&full_c[cs]);
      }
      if (q)
        ++used[1];
      else
        ++used[0];
      q_out.advance(1);
    };
    Step now{}, then{};
    next_run(now);
    if (now.run) issue(now);
    while (ok && now.run) {
      then = now;
      // The step behind this one, if it is known already: a run that is still to come may wait for this step,
      // and this step's run is held until then (a warp gives run i back when it takes run i + 2).
      bool known = ++then.u < steps_of(now.run), last = false;
      if (!known &&
          __all_sync(0xffffffffu, mbar_test(&run_there[unit % kRuns], (unit / kRuns) & 1u))) {
        then.run = get_run(unit++);
        then.u = 0;
        last = !then.run;
        known = then.run && steps_of(then.run) > 0;
      }
      // (the place of two or three steps ago: not waited for while this step's work can be done)
      const bool ahead =
          known && (issued < NQ || __all_sync(0xffffffffu, mbar_test(&free_q[q_in.st], q_in.par ^ 1u)));
      if (ahead) {
        issue(then);
        asm volatile("cp.async.wait_group 1;" ::: "memory");
      } else {
        asm volatile("cp.async.wait_group 0;" ::: "memory");
      }
      finish(now);
      if (ok && !known && !last) next_run(then);
      if (ok && then.run && !ahead) issue(then);
      now = then;
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (!ok && !W8 && a.step_tokens > 0 && w == 0)  // (else the MMAs have waited for every box)
      for (int t = max(0, issued - NQ); t < issued; ++t)
        mbar_wait(&full_q[t % NQ], (uint32_t)(t / NQ) & 1u, a.err);
  } else if (warp >= kConvWarp) {
    // ===================== 8-bit codes to f16 in MMA form =====================
    regs_down<S::REGS>();
    if constexpr (W8) {
        constexpr int CPR = D / 16;                       // 16-code chunks of a row
      constexpr int PER = kHalf / 2 * CPR / 128;        // chunks of a thread in half a tile
      constexpr int ROWS = 128 / CPR;
      const int i0 = threadIdx.x - kConvWarp * 32;
      int row0, c;  // eight threads read and write distinct banks: four chunks each of two rows
      if constexpr (CPR == 8) {
        row0 = 2 * (i0 >> 4) + ((i0 >> 2) & 1);
        c = (i0 & 3) + 4 * (((i0 >> 2) ^ (i0 >> 3)) & 1);
      } else {
        row0 = i0 >> 2;
        c = i0 & 3;
      }
      const int ch = 2 * c;  // 16-byte chunks ch and ch + 1 of the row's f16
      const uint32_t x0 = ((ch & 7) ^ (row0 & 7)) << 4, x1 = (((ch & 7) + 1) ^ (row0 & 7)) << 4;
      const uint32_t src0 = ring + S::OFF_RAW + row0 * D + c * 16;
      const uint32_t k0 = ring + (ch >> 3) * (kHalf * 128) + row0 * 128;
      Place<W8 ? NR : 1> raw;
      Place<NK> pk;
      bool ok = true;
      int tiles = 0;
      for (uint32_t unit = 0; ok; ++unit) {
        const WeighRun* run = get_run(unit);
        if (!run) break;
        const int halves = steps_of(run) > 0 ? halves_of(run) : 0;
        for (int h = 0; ok && h < halves; ++h, ++tiles, pk.advance(1)) {
          int mask = 0;
#pragma unroll
          for (int part = 0; part < 2; ++part) {
            ok = mbar_wait(&raw_full[raw.st], raw.par, a.err);
            if (!ok) break;
            const uint32_t src = src0 + raw.st * S::RAW;
            mask |= raw_mask[raw.st] << (part * (kPages / 2));
            uint4 x[PER];
#pragma unroll
            for (int i = 0; i < PER; ++i) x[i] = lds128(src + i * ROWS * D);
            __syncwarp();
            if (lane == 0) mbar_arrive(&raw_freed[raw.st]);
            raw.advance(1);
            if (part == 0 && tiles >= NK) ok = mbar_wait(&free_k[pk.st], pk.par ^ 1u, a.err);
            if (!ok) break;
#pragma unroll
            for (int i = 0; i < PER; ++i) {
              const uint32_t at = k0 + pk.st * S::TILE + (part * (kHalf / 2) + i * ROWS) * 128;
              uint4 lo, hi;
              widen4<KV>(x[i].x, lo.x, lo.y);
              widen4<KV>(x[i].y, lo.z, lo.w);
              widen4<KV>(x[i].z, hi.x, hi.y);
              widen4<KV>(x[i].w, hi.z, hi.w);
              sts128(at + x0, lo);
              sts128(at + x1, hi);
            }
          }
          if (!ok) break;
          if (i0 == 0) page_mask[pk.st] = mask;
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&full_k[pk.st]);
        }
      }
    }
  } else {
    // ===================== sums =====================
    regs_up<S::SUM_REGS>();
    const int group = warp >> 2, h = group & 1, q = group >> 1;
    const int r = threadIdx.x & 127;  // position of the half
    const uint32_t scol = tmem + ((uint32_t)((warp & 3) * 32) << 16) + 128 * group;
    bool ok = true;
    uint32_t ph_s = 0, hands = 0;  // parity of s_done's next phase; runs that handed sums over
    Place<NK> ks;
    Place<2> cs;  // of the group's steps
    const float sc = a.scale * kLog2e;
    const bool cap = FORM && a.softcap > 0.f;
    const float in = cap ? (W8 ? kLn2 : kLn2 * sc) / a.softcap : 0.f, top = a.softcap * kLog2e;
    for (uint32_t unit = 0;; ++unit) {
      const WeighRun* run = get_run(unit);
      if (!run) break;
      const int n = steps_of(run), halves = halves_of(run);
      const int p0 = run->item * kItem + h * kHalf, p = p0 + r, ctx = run->req.base + run->req.n;
      const int64_t at = ((int64_t)run->b * a.h_kv + run->j) * a.width + p;
      const bool writes = q == 0 && h < halves && p < ctx;
      const float before = writes && run->whole && a.add_to ? a.add_to[at] : 0.f;  // (on its way meanwhile)
      float total = 0.f, lost = 0.f;
      bool good = false;
      // (Every warp waits for the other half's K too: a phase that a warp does not see could still be to
      // come when it asks for the one behind it, whose parity then looks as if it were over.)
      for (int i = 0; i < halves && n > 0; ++i) {
        Place<NK> k = ks;
        k.advance(i);
        ok = ok && mbar_wait(&full_k[k.st], k.par, a.err);
        if (i == h) good = ok && ((page_mask[k.st] >> (r >> 4)) & 1);
        __syncwarp();
        if (lane == 0) mbar_arrive(&free_k[k.st]);
      }
      // Rows in order see positions in order: of the run's rows, this position is seen from `from` on and up
      // to the last or, with a window that it can leave, up to `end`. (Rows that are not there hold what
      // lies behind the request's, or zeros.)
      const unsigned rows = (unsigned)(run->rows - run->s0 * kStep);
      const long long first = (long long)(p - run->req.base - run->t0) * a.group - (long long)run->s0 * kStep;
      // (a page that is not there is seen by none)
      const unsigned from = good ? (unsigned)max(0ll, min((long long)INT_MAX, first)) : INT_MAX;
      const unsigned end = a.window > 0 && p >= a.sink
                               ? (unsigned)max(0ll, min((long long)rows, first + (long long)a.window * a.group))
                               : rows;
      const unsigned from_any = __reduce_min_sync(0xffffffffu, from);
      const unsigned from_all = __reduce_max_sync(0xffffffffu, from);
      const unsigned end_any = __reduce_max_sync(0xffffffffu, end);
      const unsigned end_all = __reduce_min_sync(0xffffffffu, end);
      for (int u = q; ok && u < n; u += 2, cs.advance(1)) {
        const int at_c = 2 * q + cs.st;
        ok = mbar_wait(&full_c[at_c], cs.par, a.err);
        const bool none = *reinterpret_cast<const uint32_t*>(some_none[at_c]) != 0;
        if (ok && h < halves) ok = mbar_wait(&s_done[group], ph_s, a.err);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        if (h < halves) {
          ph_s ^= 1u;
          tc_fence_after();
          const unsigned u0 = (unsigned)u * kStep;
          const int cols = (int)min((unsigned)kStep, rows - u0);
          const Columns cn = columns(col, at_c);
          uint64_t sum[4] = {0, 0, 0, 0};
          const uint64_t sc2 = pack2(sc, sc);
          // With the tests of what its positions see, or, where every row sees them all and has an lse,
          // without: in one body the tests cost more than the few steps that need them (4095 rows over
          // themselves: 85 us instead of 75). What gives a position nothing has a score of -inf there,
          // whatever its product is.
          auto step = [&](auto edge) {
#pragma unroll 1
            for (int c = 0; c < cols; c += 32) {
              uint32_t s[32];
              tmem_ld32(scol + c, s);
              tmem_wait_ld();
              if (c + 32 >= cols) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&s_read[group]);
              }
              // (columns that see no position of the warp are left out)
              if (decltype(edge)::value && (u0 + c + 32 <= from_any || u0 + c >= end_any)) continue;
              uint32_t gives = ~0u;  // the columns that give this position something
              if constexpr (decltype(edge)::value)
                gives = (uint32_t)(low_bits((int)(end - (u0 + c))) & ~low_bits((int)(from - (u0 + c)))) &
                        ~no_lse[at_c][c >> 5];
              if constexpr (FORM && decltype(edge)::value) {
                // (what is not seen may be whatever memory held, and has no say in how the cap is taken)
                if (cap) {
#pragma unroll
                  for (int k = 0; k < 32; ++k)
                    if (!((gives >> k) & 1)) s[k] = 0u;
                }
              }
              if constexpr (FORM) {
                if (W8 || !cap) {
#pragma unroll
                  for (int k = 0; k < 32; ++k)
                    s[k] = __float_as_uint(__uint_as_float(s[k]) * (W8 ? cn.factor[c + k] : sc));
                }
                if (cap) cap_scores<32>(s, in, top);
                if (a.slopes) {
#pragma unroll
                  for (int k = 0; k < 32; ++k)
                    s[k] = __float_as_uint(fmaf(cn.slope[c + k], (float)(p - cn.pos[c + k]),
                                                __uint_as_float(s[k])));
                }
              }
              if constexpr (decltype(edge)::value) {
#pragma unroll
                for (int k = 0; k < 32; ++k)
                  if (!((gives >> k) & 1)) s[k] = __float_as_uint(-INFINITY);
              }
#pragma unroll
              for (int k = 0; k < 32; k += 4) {
                const ulonglong2 nl = *reinterpret_cast<const ulonglong2*>(cn.neg_lse + c + k);
                uint64_t x01 = get2(&s[k]), x23 = get2(&s[k + 2]);
                if constexpr (FORM) {
                  x01 = add2(x01, nl.x);
                  x23 = add2(x23, nl.y);
                } else if constexpr (W8) {
                  const ulonglong2 f = *reinterpret_cast<const ulonglong2*>(cn.factor + c + k);
                  x01 = fma2(x01, f.x, nl.x);
                  x23 = fma2(x23, f.y, nl.y);
                } else {
                  x01 = fma2(x01, sc2, nl.x);
                  x23 = fma2(x23, sc2, nl.y);
                }
                float e0, e1, e2, e3;
                unpack2(x01, e0, e1);
                unpack2(x23, e2, e3);
                sum[(k >> 1) & 3] = add2(sum[(k >> 1) & 3], pack2(ex2_approx(e0), ex2_approx(e1)));
                sum[((k >> 1) & 3) + 1] =
                    add2(sum[((k >> 1) & 3) + 1], pack2(ex2_approx(e2), ex2_approx(e3)));
              }
            }
          };
          if (none || u0 < from_all || u0 + ((cols + 31) & ~31) > end_all)
            step(std::true_type{});
          else
            step(std::false_type{});
          float x, y;
          unpack2(add2(add2(sum[0], sum[1]), add2(sum[2], sum[3])), x, y);
          const float add = (x + y) - lost, z = total + add;
          lost = (z - total) - add;
          total = z;
          if (!(total < INFINITY) && *reinterpret_cast<const uint32_t*>(some_nan[at_c]) != 0) total = NAN;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&free_c[at_c]);
      }
      // ---- the run's sums: the second steps' group hands its own to the first's, which writes ----
      if (n > 1 && h < halves) {
        const int spot = hands & 1;  // runs take turns between two places
        float* const place = hand + spot * kItem + h * kHalf + r;
        if (q == 1) {
          if (hands >= 2)
            ok = mbar_wait(&taken[2 * spot + h], ((hands >> 1) - 1) & 1u, a.err) && ok;
          *place = total;
          __syncwarp();
          if (lane == 0) mbar_arrive(&handed[2 * spot + h]);
        } else {
          ok = mbar_wait(&handed[2 * spot + h], (hands >> 1) & 1u, a.err) && ok;
          total += *place;
          __syncwarp();
          if (lane == 0) mbar_arrive(&taken[2 * spot + h]);
        }
        ++hands;
      }
      ok = __all_sync(0xffffffffu, ok);
      if (writes && ok) {
        const float x = good ? total : 0.f;
        if (run->whole)
          a.weights_out[at] = before + x;
        else
          a.ws_acc[((size_t)blockIdx.x * 2 + run->slot) * kItem + h * kHalf + r] = x;
      }
      if (n > 0) ks.skip(halves);
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  release();
}

template <typename KV, int D, bool FORM>
cudaError_t launch_shape(const ChunkArgs& a, const CUtensorMap& tk, const CUtensorMap& tq,
                         cudaStream_t s) {
  using S = WeighTcShape<KV, D>;
  static std::atomic<unsigned long long> attr_done{0};  // one bit per device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !((attr_done.load() >> dev) & 1ull)) {
    cudaFuncAttributes fa{};  // (a launch with fewer could not give the sums theirs: they would wait)
    e = cudaFuncGetAttributes(&fa, weights_tc_kernel<KV, D, FORM>);
    if (e != cudaSuccess) return e;
    if (fa.numRegs < S::LAUNCH_REGS) return cudaErrorLaunchOutOfResources;
    e = cudaFuncSetAttribute(weights_tc_kernel<KV, D, FORM>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, S::SMEM);
    if (e != cudaSuccess) return e;
    if (dev < 64) attr_done.fetch_or(1ull << dev);
  }
  weights_tc_kernel<KV, D, FORM><<<a.ctas, S::THREADS, S::SMEM, s>>>(a, tk, tq);
  return cudaGetLastError();
}

template <typename KV, int D>
cudaError_t launch_t(const ChunkArgs& a, const CUtensorMap& tk, const CUtensorMap& tq,
                     cudaStream_t s) {
  return a.softcap > 0.f || a.slopes ? launch_shape<KV, D, true>(a, tk, tq, s)
                                     : launch_shape<KV, D, false>(a, tk, tq, s);
}

}  // namespace

cudaError_t launch_chunk_weights_tc(const ChunkArgs& a, int kv_dtype, int head_dim, const void* tk,
                                    const void* tq, cudaStream_t s) {
  const CUtensorMap& mk = *static_cast<const CUtensorMap*>(tk);
  const CUtensorMap& mq = *static_cast<const CUtensorMap*>(tq);
  if (head_dim == 64) {
    if (kv_dtype == PKV_BF16) return launch_t<BF16, 64>(a, mk, mq, s);
    if (kv_dtype == PKV_FP8_E4M3) return launch_t<FP8, 64>(a, mk, mq, s);
    return launch_t<INT8, 64>(a, mk, mq, s);
  }
  if (kv_dtype == PKV_BF16) return launch_t<BF16, 128>(a, mk, mq, s);
  if (kv_dtype == PKV_FP8_E4M3) return launch_t<FP8, 128>(a, mk, mq, s);
  return launch_t<INT8, 128>(a, mk, mq, s);
}

}  // namespace pkv
