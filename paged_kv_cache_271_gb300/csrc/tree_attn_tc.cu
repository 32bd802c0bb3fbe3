// Tree attention on the fifth-generation tensor cores (tcgen05), bf16 queries over a bf16, FP8 or
// INT8 cache.
//
// The mathematics is that of tree_attn.cu; the work is cut as tree_plan.cuh says, in units of up to
// 256 (node, query head) rows of one KV head and tiles of 64 tokens, one persistent CTA per SM. A
// verification step does 4 rows x D operations per cached K/V row of 2 D values, so up to about 256
// rows it is bound by reading the cache once; the work here is arranged so that everything else
// hides behind those reads:
//
//  * two copy warps stream the share's tiles, one K and one V, through rings of shared memory,
//    running ahead across units; a bf16 tile arrives by TMA in the 128-byte-swizzled form the MMAs
//    read. The codes of an 8-bit tile arrive by bulk copies and four converter warps widen them to
//    f16 (exactly) in that form; the K scale goes into the score factor and the V scale into the
//    output. The K warp also walks the share and hands its runs to the others;
//  * two MMA warps: one issues S = Q K^T (M = 128 rows, N = 64 tokens) up to four steps ahead, the
//    other O += P V (N = D), with P as an A operand in the tensor memory that held S and all
//    accumulators there (one warp issuing both was the limit of an 8-bit cache's small units);
//  * two groups of four softmax warps, thread r of a group owning row r. Units of up to 128 rows: the
//    groups take alternate tiles, which add into one O; a row's reference maximum goes from step to
//    step through shared memory, set before anything else of a step is done, and each group keeps
//    its own sum. Larger units: group g takes rows 128 g .. of every tile with an O of its own, so the
//    cache is still read once;
//  * O is rescaled only when a row's maximum grows by more than 2^8 (8-bit caches: 2^7): the final
//    (max, sum, O) is exact whatever reference it was accumulated against.
//
// Two kernels: a call whose drafts have at most 128 rows a KV head keeps a unit's queries in tensor
// memory beside an O and four S buffers and has the whole of shared memory for the rings; with more
// rows the tensor memory holds two O and four S, and the queries are read from 64 KB of shared memory
// (in tensor memory they left room for two S buffers: 425 us instead of 380 for 128 requests of 128
// .. 8192 FP8 tokens and 192 rows a head; 169 instead of 142 for ragged bf16 drafts). The queries of
// the larger kernel are prefetched into L2 when a run is handed out (wide FP8 208 us without, 204
// with; in the smaller kernel the prefetch costs more than it gives: 64 dims 83 without, 92 with).
//
// P is rounded to the MMA's input type (bf16 for a bf16 cache, f16 otherwise), the only rounding
// before the output's; scores, maxima and sums are fp32. For 8-bit caches a query row is scaled by
// a power of two that puts its largest value in f16's top binade, undone in its score factor; the sign
// of the K scale goes with it, so that score factors are positive.
//
// Tiles with unseen positions (the drafted nodes, the end of the context, bad pages) mask scores
// by the row's 64 mask bits, and their V rows are mended in shared memory before the MMA reads them:
// rows outside the context or on a bad page become 0, and a drafted row's infinite or NaN values,
// which 0 P would still spread to rows that do not see the node, become 0 there and are added to
// the rows that do see it at the unit's end.
//
// Measured with the combine in graphs of calls over two states, in brackets the bytes of those states
// and their time at the copy's 6.78 TB/s: 64 requests of 512 .. 4096 bf16 tokens, 64 rows a head: 111 us
// (648 MB, 96); ragged drafts of up to 256 rows: 149 (651 MB, 96); 4 requests of 8191 .. 65536 INT8
// tokens, 96 rows: 68 (210 MB, 31); 128 requests of 128 .. 8192 FP8 tokens, 192 rows: 388 (1108 MB, 163).
// (The figures above, and beside the split's constants, are of single calls after a flush of the L2.)
// Large units are bound by the softmax steps, about 1400 cycles of waits, tensor-memory loads and
// exponentials for 128 rows x 64 tokens, two at a time on an SM, and by 4 to 8 thousand cycles from the
// last step of a unit to the first of the next. Small units take, from whole calls, about 900 cycles a
// tile of a 64-dim bf16 cache and 1200 to 1350 of an 8-bit one with 128 dims, for which the copy's rate
// would allow 700: two steps at a time overlap in part only. Whether the hand-over of the maximum or the
// converters, which widen one tile from end to end, set that pace has not been told apart.
//
// Every wait is bounded (PKV_DEVERR_TIMEOUT); the tensor memory is freed on every path.
#include <atomic>
#include <cuda.h>
#include <math.h>

#include "paged_decode_mma.cuh"
#include "pkv_device.cuh"
#include "pkv_internal.h"
#include "tcgen05.cuh"
#include "tree_exchange.h"
#include "tree_plan.cuh"

namespace pkv {

namespace {

constexpr int kTok = kTreeTcTokens;        // tokens of a tile
constexpr int kPages = kTok / kPageSize;   // pages of a tile
constexpr int kGroupThreads = 128;         // a softmax group: one row per thread
constexpr int kSoftThreads = 2 * kGroupThreads;
constexpr int kMmaWarp = kSoftThreads / 32;  // two: S and P V
constexpr int kCopyWarp = kMmaWarp + 2;      // two: copies of K and of V
constexpr int kConvWarp = kMmaWarp + 4;      // first of four (8-bit caches)
constexpr int kConvThreads = 128;
constexpr int kSBufs = 4;
// Runs on their way from the K copy warp, which walks the share, to the other warps. It is ahead by
// the tiles of the rings at most, each a run of its own at worst, besides the run whose rows are
// being written and the one it is about to copy.
constexpr int kRuns = 32;
// tensor memory columns. WIDE: two O and four S (then P) buffers; otherwise an O, a Q and the same
constexpr uint32_t kColO = 0, kColQ = 256;
constexpr uint32_t kTmemCols = 512;
static_assert(2 * kGroupThreads == kTreeTcRows, "a unit is two groups' rows");
static_assert(kExchangeRows == kGroupThreads, "a place for each row of a group");

template <typename KV, int D, bool WIDE>
struct TcShape {
  static constexpr bool W8 = KV::bytes == 1;
  static constexpr int THREADS = 32 * (W8 ? kConvWarp + kConvThreads / 32 : kConvWarp);
  // registers of the softmax warps and of the others, out of what the launch gives every warp
  static constexpr int SOFT_REGS = W8 ? 176 : 208, REGS = W8 ? 72 : 80;
  static constexpr int TILE = kTok * D * 2;       // K (or V) of a tile in MMA form
  static constexpr int RAW_TILE = kTok * D;       // 8-bit codes
  static constexpr int RAW_STAGE = 2 * RAW_TILE;
  // rings: K tiles, needed until their S is done, and V tiles, needed until their P V is done, go
  // round separately; 8-bit caches have raw codes before them
  static constexpr int NK = (WIDE ? W8 ? 32 : 64 : W8 ? 48 : 96) * 1024 / TILE;
  static constexpr int NV = (WIDE ? W8 ? 48 : 80 : W8 ? 64 : 96) * 1024 / TILE;
  static constexpr int NR = W8 ? (WIDE ? 64 : 80) * 1024 / RAW_STAGE : 0;
  static constexpr int OFF_V = NK * TILE;
  static constexpr int OFF_RAW = OFF_V + NV * TILE;
  static constexpr int OFF_Q = OFF_RAW + NR * RAW_STAGE;    // WIDE: 256 queries in MMA form
  static constexpr int Q_GROUP = WIDE ? kGroupThreads * D * 2 : 0;
  static constexpr int PIECE = WIDE ? 32 : 64;              // bytes of a row that change hands at once
  static constexpr int OFF_STAGE = OFF_Q + 2 * Q_GROUP;     // 32 rows' pieces for each softmax warp
  static constexpr int OFF_ML = OFF_STAGE + kSoftThreads * PIECE;  // (max, sum) exchanged
  static constexpr int OFF_REF = OFF_ML + kExchangeSlots * 8;      // [128] reference maxima
  static constexpr int OFF_BAR = OFF_REF + kGroupThreads * 4;
  static constexpr int BARS = 2 * NK + 2 * NV + 2 * NR + 3 * kSBufs + 6 + kRuns;
  static_assert(NK + NR + 3 <= kRuns, "runs in flight");
  static constexpr int OFF_MISC = OFF_BAR + 8 * BARS;       // masks, bad nodes, TMEM address
  static constexpr uint32_t IDESC_S = tc_idesc(128, kTok, false, W8);
  static constexpr uint32_t IDESC_PV = tc_idesc(128, D, true, W8);
  static constexpr int SMEM = 1024 + OFF_MISC + 4 * (NV + NR + 2 * 8 + 1) + 16;
  static_assert(SMEM <= 227 * 1024 && SMEM > 114 * 1024, "one CTA per SM");
};

template <bool WIDE>
__device__ __forceinline__ uint32_t s_col(int buf) {
  return WIDE || buf >= 2 ? (WIDE ? 256 : 0) + 64 * buf : 384 + 64 * buf;
}

// A unit's steps in order: with up to 128 rows step u is tile u, otherwise ("wide") tile u / 2 for
// rows 128 (u % 2) ... Group u % 2 takes it, in S buffer u % 4. Every buffer's three barriers
// complete once per step that uses it.
// parity of the buffer's barriers in step u; ph holds each buffer's at the unit's start
__device__ __forceinline__ uint32_t parity_of(uint32_t ph, int u) {
  return ((ph >> (u & 3)) ^ (uint32_t)(u >> 2)) & 1u;
}
// the buffers' parities after a unit of n steps
__device__ __forceinline__ uint32_t after_steps(uint32_t ph, int n) {
  if ((n >> 2) & 1) ph ^= 15u;
  return ph ^ ((1u << (n & 3)) - 1u);
}

// A place in a ring of N stages and the parity of its current use.
template <int N>
struct Place {
  int st = 0;
  uint32_t par = 0;
  __device__ __forceinline__ void advance(int k) {  // k <= N
    st += k;
    if (st >= N) {
      st -= N;
      par ^= 1u;
    }
  }
  __device__ __forceinline__ void skip(int k) {  // any k
    const int t = st + k, w = t / N;
    st = t - w * N;
    par ^= (uint32_t)w & 1u;
  }
};

template <bool B>
struct BoolConst {
  static constexpr bool value = B;
};

template <int N>
__device__ __forceinline__ void regs_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

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

// WIDE: units may have more than 128 rows.
template <typename KV, int D, bool WIDE>
__global__ void __launch_bounds__(TcShape<KV, D, WIDE>::THREADS, 1) tree_tc_kernel(
    const TreeArgs a, const __grid_constant__ CUtensorMap tm_k,
    const __grid_constant__ CUtensorMap tm_v) {
  using S = TcShape<KV, D, WIDE>;
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
  uint64_t* raw_freed = raw_full + NR;                               // [NR] codes widened
  uint64_t* s_done = raw_freed + NR;                                 // [4] S in its buffer
  uint64_t* p_ready = s_done + kSBufs;                               // [4] P in its buffer
  uint64_t* pv_done = p_ready + kSBufs;                              // [4] that P V complete
  // Q of a unit stored; the MMA warps arrive too, for the unit after the one they have seen, so
  // that no phase completes before both have seen the last (one may have no step in a unit)
  uint64_t* q_ready = pv_done + kSBufs;
  uint64_t* o_read = q_ready + 1;                                    // O of a unit read
  uint64_t* met = o_read + 1;                                        // both groups ended a unit
  uint64_t* mma_idle = met + 1;
  uint64_t* ref_set = mma_idle + 1;                                  // [2] a group's step set it
  uint64_t* run_there = ref_set + 2;                                 // [kRuns]
  int* page_mask = reinterpret_cast<int*>(smem + S::OFF_MISC);       // [NV] good pages of the tile
  int* raw_mask = page_mask + NV;                                    // [NR]
  uint32_t* bad_nodes = reinterpret_cast<uint32_t*>(raw_mask + NR);  // [2][8] V row not finite
  uint32_t* s_taddr = bad_nodes + 16;
  float2* ml = reinterpret_cast<float2*>(smem + S::OFF_ML);          // (tree_exchange.h)
  float* ref = reinterpret_cast<float*>(smem + S::OFF_REF);          // [128]

  __shared__ int scratch[64];
  __shared__ TreeShare share;
  __shared__ TreeRun runs[kRuns];  // (n = 0: the share's end)
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (threadIdx.x == kCopyWarp * 32) {
    for (int s = 0; s < NK; ++s) {
      mbar_init(&full_k[s], W8 ? kConvThreads / 32 : 1);
      mbar_init(&free_k[s], 2);
    }
    for (int s = 0; s < NV; ++s) {
      mbar_init(&full_v[s], W8 ? kConvThreads / 32 : 1);
      mbar_init(&free_v[s], 2);
    }
    for (int s = 0; s < NR; ++s) {
      mbar_init(&raw_full[s], 2);
      mbar_init(&raw_freed[s], kConvThreads / 32);
    }
    for (int s = 0; s < kSBufs; ++s) {
      mbar_init(&s_done[s], 1);
      mbar_init(&p_ready[s], kGroupThreads / 32);
      mbar_init(&pv_done[s], 1);
    }
    mbar_init(q_ready, kSoftThreads / 32 + 2);
    mbar_init(o_read, kSoftThreads / 32);
    mbar_init(met, kSoftThreads / 32);
    mbar_init(mma_idle, 2);
    for (int g = 0; g < 2; ++g) mbar_init(&ref_set[g], kGroupThreads / 32);
    for (int i = 0; i < kRuns; ++i) mbar_init(&run_there[i], 1);
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
  const uint32_t tmem = (uint32_t)uniform((int)*s_taddr);
  // run i of the share, or nullptr after the last (or a wait that gave up)
  auto get_run = [&](uint32_t i) -> const TreeRun* {
    const bool got = mbar_wait(&run_there[i % kRuns], (i / kRuns) & 1u, a.err);
    const TreeRun* r = &runs[i % kRuns];
    return __all_sync(0xffffffffu, got && r->n > 0) ? r : nullptr;
  };

  if (warp >= kMmaWarp && warp < kConvWarp) {
    regs_down<S::REGS>();
    if (warp == kCopyWarp || warp == kCopyWarp + 1) {
      // ===================== copies: the share's tiles, in order =====================
      // One warp copies K, one V, each through its own ring (8-bit caches: both into the same
      // stages): a copy's issue takes a while, and a tile of 64 tokens is 8 to 12 of them.
      const bool is_k = warp == kCopyWarp;
      // the row units of more than 256 rows read the same tiles again
      const uint64_t pol =
          a.nodes * a.group > kTreeTcRows ? l2_evict_last_policy() : l2_evict_first_policy();
      const int stages = W8 ? NR : is_k ? NK : NV;
      uint64_t* const there = W8 ? raw_full : is_k ? full_k : full_v;
      uint64_t* const gone = W8 ? raw_freed : is_k ? free_k : free_v;
      int* const masks = W8 ? raw_mask : page_mask;  // (written by the V warp)
      const uint32_t ring0 = ring + (is_k ? 0 : S::OFF_V);
      uint8_t* const raw0 = smem + S::OFF_RAW + (is_k ? 0 : S::RAW_TILE);
      const uint8_t* const pool = static_cast<const uint8_t*>(is_k ? a.k_cache : a.v_cache);
      int st = 0, issued = 0;
      uint32_t par = 0;
      bool ok = true;
      TreeWalk walk(a, share);
      for (uint32_t unit = 0;; ++unit) {
        const TreeRun* run = nullptr;
        if (is_k) {  // (a wait that gave up ends the share for every warp)
          TreeRun* r = &runs[unit % kRuns];
          if (lane == 0) {
            if (!ok || !walk.next(a, *r)) r->n = 0;
            mbar_arrive(&run_there[unit % kRuns]);
          }
          __syncwarp();
          if (r->n > 0) run = r;
        } else if (ok) {
          run = get_run(unit);
        }
        if (!run) break;
        const int pages = uniform((run->req.read + kPageSize - 1) / kPageSize);
        const int n = uniform(run->n), j = uniform(run->j);
        const int32_t* table = a.block_tables + (size_t)run->b * a.max_pages;
        if (WIDE && is_k) {  // the run's queries into L2, some tiles before their rows are read
          const int t0 = uniform(run->row0) / a.group;
          const int t1 = (uniform(run->row0 + run->rows) - 1) / a.group;
          const uint8_t* q = static_cast<const uint8_t*>(a.q) +
                             2 * (((size_t)run->b * a.nodes * a.h_q) + (size_t)j * a.group) * D;
          for (int t = t0 + lane; t <= t1; t += 32)
            bulk_prefetch_l2(q + 2 * (size_t)t * a.h_q * D, 2 * a.group * D);
        }
        int lp = uniform(run->tile0 * kPages);  // first page of the tile
        int ids = -1;                          // lane L: the id of page 32 m + L of the run
        for (int i = 0; i < n; ++i, lp += kPages) {
          if ((i & 7) == 0) ids = lp + lane < pages ? table[lp + lane] : -1;
          int id[kPages];
          uint32_t mask = 0;
#pragma unroll
          for (int p = 0; p < kPages; ++p) {
            id[p] = __shfl_sync(0xffffffffu, ids, (kPages * i + p) & 31);
            if (lp + p < pages && id[p] >= 0 && id[p] < a.num_pages) mask |= 1u << p;
          }
          if (is_k && mask != (1u << min(kPages, pages - lp)) - 1 && lane == 0)
            atomicOr(a.err, PKV_DEVERR_BAD_PAGE);
          if (issued >= stages) {
            ok = __all_sync(0xffffffffu, mbar_wait(&gone[st], par ^ 1u, a.err));
            if (!ok) break;
          }
          if (elect_one()) {
            if (!is_k) masks[st] = (int)mask;
            if constexpr (W8) fence_proxy_async_smem();
            mbar_arrive_expect_tx(&there[st], __popc(mask) * (W8 ? PAGE_RAW : PAGE_MMA));
#pragma unroll
            for (int p = 0; p < kPages; ++p) {
              if (!((mask >> p) & 1)) continue;
              if constexpr (W8) {
                bulk_g2s(raw0 + st * S::RAW_STAGE + p * PAGE_RAW,
                         pool + ((int64_t)id[p] * a.h_kv + j) * PAGE_RAW, PAGE_RAW, &there[st], pol);
              } else {
                const int row = (id[p] * a.h_kv + j) * kPageSize;
                const uint32_t dst = ring0 + st * S::TILE;
                if (is_k) {  // 64-dim blocks of all 64 rows (one N = 64 operand)
#pragma unroll
                  for (int bx = 0; bx < D / 64; ++bx)
                    tma_load_2d(dst + bx * (kTok * 128) + p * 2048, &tm_k, bx * 64, row, &there[st],
                                pol);
                } else {  // a block per page (K = 16)
                  tma_tile<D / 64, 64>(dst + p * PAGE_MMA, &tm_v, a.tma_rank, row, &there[st], pol);
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
      }
      if (lane == 0)  // before leaving, every copy issued has landed
        for (int t = max(0, issued - stages); t < issued; ++t)
          mbar_wait(&there[t % stages], (uint32_t)(t / stages) & 1u, a.err);
    } else {
      // ===================== MMAs (one elected lane issues) =====================
      // Two warps, since issuing a step's MMAs takes about as long as they run: one issues the S, up
      // to four steps ahead, the other the P V.
      const int w = warp - kMmaWarp;
      const uint64_t k_desc = tc_desc(ring, 16, 1024), v_desc = tc_desc(ring + S::OFF_V, 2048, 1024);
      const uint64_t q_desc = tc_desc(ring + S::OFF_Q, 16, 1024);
      bool ok = true;
      uint32_t ph = 0, unit = 0;
      Place<NK> k_base;  // the run's first tile
      Place<NV> v_base;
      auto wait = [&](uint64_t* bar, uint32_t par) {
        const bool got = __all_sync(0xffffffffu, mbar_wait(bar, par, a.err));
        tc_fence_after();
        return got;
      };
      auto s_mma = [&](const Place<NK>& k, int group, int buf) {
        const uint64_t kd = k_desc + (uint32_t)(k.st * (S::TILE >> 4));
        const uint64_t qd = q_desc + (uint32_t)(group * (S::Q_GROUP >> 4));
        const uint32_t d = tmem + s_col<WIDE>(buf);
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint64_t kb = kd + (((kk >> 2) * (kTok * 128) + (kk & 3) * 32) >> 4);
            if constexpr (WIDE)
              tc_mma_sa(d, qd + (((kk >> 2) * (kGroupThreads * 128) + (kk & 3) * 32) >> 4), kb,
                        S::IDESC_S, kk > 0 ? 1u : 0u);
            else
              tc_mma_ta(d, tmem + kColQ + 8 * kk, kb, S::IDESC_S, kk > 0 ? 1u : 0u);
          }
          tc_commit(&s_done[buf]);
        }
        __syncwarp();
      };
      auto pv_mma = [&](const Place<NV>& v, uint32_t o, int buf, bool first) {
        const uint64_t vd = v_desc + (uint32_t)(v.st * (S::TILE >> 4));
        const uint32_t pc = tmem + s_col<WIDE>(buf);
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < kPages; ++kk)
            tc_mma_ta(o, pc + 8 * kk, vd + ((kk * PAGE_MMA) >> 4), S::IDESC_PV,
                      first && kk == 0 ? 0u : 1u);
          tc_commit(&pv_done[buf]);
          tc_commit(&free_v[v.st]);
        }
        __syncwarp();
      };
      if (elect_one()) mbar_arrive(q_ready);
      __syncwarp();
      for (; ok; ++unit) {
        const TreeRun* run = get_run(unit);
        if (!run) break;
        const int tiles = uniform(run->n);
        const bool wide = WIDE && uniform(run->rows) > kGroupThreads;
        const int n = wide ? 2 * tiles : tiles;
        Place<NK> ks = k_base;  // K of the next S
        Place<NV> vs = v_base;  // V of the next P V
        ok = wait(q_ready, unit & 1);
        if (elect_one()) mbar_arrive(q_ready);  // (the next unit's: this phase has been seen)
        __syncwarp();
        if (w == 0) {
          for (int u = 0; ok && u < n; ++u) {
            const int group = wide ? u & 1 : 0;
            if (group == 0) ok = wait(&full_k[ks.st], ks.par);
            if (ok && u >= 4) ok = wait(&pv_done[u & 3], parity_of(ph, u - 4));  // P used up
            if (ok) s_mma(ks, group, u & 3);
            if (!wide || group) ks.advance(1);
          }
        } else {
          for (int u = 0; ok && u < n; ++u) {
            const int group = wide ? u & 1 : 0;
            ok = wait(&p_ready[u & 3], parity_of(ph, u));
            if (ok && u == 0 && unit > 0) ok = wait(o_read, (unit - 1) & 1);  // the last unit's
            if (ok) pv_mma(vs, tmem + kColO + 128 * group, u & 3, u == group);
            if (!wide || group) vs.advance(1);
          }
        }
        ph = after_steps(ph, n);
        k_base.skip(tiles);
        v_base.skip(tiles);
      }
      if (elect_one()) tc_commit(mma_idle);  // before leaving, every MMA issued is complete
      __syncwarp();
      wait(mma_idle, 0);
    }
  } else if (warp >= kConvWarp) {
    // ===================== 8-bit codes to f16 in MMA form =====================
    if constexpr (W8) {
      regs_down<S::REGS>();
      constexpr int CPR = D / 16;                               // 16-code chunks of a row
      constexpr int PER = 2 * kTok * CPR / kConvThreads;        // chunks of a thread, half K half V
      const int i0 = threadIdx.x - kConvWarp * 32;
      // a thread's chunks are PER / 2 rows of K and the same of V, ROWS rows apart. Eight threads
      // read and write distinct banks: four chunks each of two rows.
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
      for (;; ++t, raw.advance(1), pk.advance(1), pv.advance(1)) {
        if (t == end) {
          const TreeRun* run = get_run(unit++);
          if (!run) break;
          end += run->n;
        }
        ok = mbar_wait(&raw_full[raw.st], raw.par, a.err);
        if (!ok) break;
        const uint32_t src = src0 + raw.st * S::RAW_STAGE;
        const int mask = raw_mask[raw.st];
        uint4 w[PER];  // K, then V
#pragma unroll
        for (int i = 0; i < PER / 2; ++i) {
          w[i] = lds128(src + i * ROWS * D);
          w[PER / 2 + i] = lds128(src + S::RAW_TILE + i * ROWS * D);
        }
        auto widen_to = [&](const uint4& v, uint32_t at) {
          uint4 lo, hi;
          widen4<KV>(v.x, lo.x, lo.y);
          widen4<KV>(v.y, lo.z, lo.w);
          widen4<KV>(v.z, hi.x, hi.y);
          widen4<KV>(v.w, hi.z, hi.w);
          sts128(at + x0, lo);
          sts128(at + x1, hi);
        };
        if (t >= NK) ok = mbar_wait(&free_k[pk.st], pk.par ^ 1u, a.err);
        if (!ok) break;
#pragma unroll
        for (int i = 0; i < PER / 2; ++i) widen_to(w[i], k0 + pk.st * S::TILE + i * ROWS * 128);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&full_k[pk.st]);
          mbar_arrive(&raw_freed[raw.st]);  // (K and V codes are in registers)
        }
        if (t >= NV) ok = mbar_wait(&free_v[pv.st], pv.par ^ 1u, a.err);
        if (!ok) break;
#pragma unroll
        for (int i = 0; i < PER / 2; ++i) {
          const int r = row0 + i * ROWS;
          widen_to(w[PER / 2 + i],
                   v0 + pv.st * S::TILE + (r >> 4) * PAGE_MMA + (r & 15) * 128);
        }
        if (i0 == 0) page_mask[pv.st] = mask;
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&full_v[pv.st]);
      }
    }
  } else {
    // ===================== softmax =====================
    regs_up<S::SOFT_REGS>();
    const int wg = warp >> 2;             // group
    const int r = threadIdx.x & 127;      // row of the group
    const uint32_t lane_t = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    bool ok = true;
    uint32_t ph = 0, ph_ref = 0, unit = 0;  // ph_ref: parities of ref_set at the unit's start
    Place<NV> base;  // V and K of the run's first tile
    Place<NK> k_base;
    // The row of this thread in a run (row `row` of its unit, node t, query head `head`) and its
    // score factor; the factor of V.
    struct Row {
      int row, t, head;
      bool live;
      float sc, vs;
    };
    auto find_row = [&](const TreeRun& run) {
      Row x;
      x.row = (WIDE && run.rows > kGroupThreads ? wg * kGroupThreads : 0) + r;
      x.live = x.row < run.rows;
      const unsigned R = x.live ? run.row0 + x.row : 0;
      x.t = (int)(R / (unsigned)a.group);
      x.head = run.j * a.group + (int)(R - x.t * (unsigned)a.group);
      x.sc = W8 ? a.scale_log2 * a.k_scales[run.j] : a.scale_log2;
      x.vs = W8 ? a.v_scales[run.j] : 1.f;
      return x;
    };
    auto row_at = [&](const TreeRun& run, const Row& x) {  // its offset in q and out
      return (((size_t)run.b * a.nodes + x.t) * a.h_q + x.head) * D;
    };
    // A unit's queries come in two steps. load_query: four lanes read 64 consecutive bytes of a row,
    // eight rows an instruction (a lane reading its own row would touch 32 lines an instruction).
    // store_query, once the S of the last unit are done: 32 rows x 64 bytes at a time change hands
    // through shared memory, and each lane puts its row into tensor memory.
    constexpr int RND = D / 32;  // rounds of 64 bytes
    auto needs_query = [&](const TreeRun& run) {  // (8-bit caches: both groups need a row's scale)
      return ok && (W8 || (WIDE && run.rows > kGroupThreads) || wg == 0);
    };
    auto load_query = [&](const TreeRun& run, const Row& x, uint4 (&in)[RND][4]) {
      if (!needs_query(run)) return;
      const size_t off = row_at(run, x);
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const int from = 8 * g + (lane >> 2);
        const size_t at = __shfl_sync(0xffffffffu, (unsigned long long)off, from);
        const bool there = __shfl_sync(0xffffffffu, (int)x.live, from) != 0;
        const uint4* src =
            reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.q) + at) + (lane & 3);
#pragma unroll
        for (int d = 0; d < RND; ++d) in[d][g] = there ? src[4 * d] : make_uint4(0, 0, 0, 0);
      }
    };
    auto store_query = [&](const TreeRun& run, Row& x, uint4 (&in)[RND][4]) {
      const bool wide = WIDE && run.rows > kGroupThreads;
      if (needs_query(run)) {
        if constexpr (W8) {  // f16, scaled by a row's 2^e (the four lanes that hold a row agree)
          const float sc = x.sc;
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            uint32_t lo = 0, hi = 0;  // largest |q| as bits (bf16 magnitudes order like integers)
#pragma unroll
            for (int d = 0; d < RND; ++d) {
              const uint32_t* w = &in[d][g].x;
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                lo = max(lo, w[k] & 0x7fffu);
                hi = max(hi, w[k] & 0x7fff0000u);
              }
            }
            uint32_t mx = max(lo, hi >> 16);
            mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
            mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
            const int ex = mx >> 7;  // biased exponent: mx 2^e in [2^14, 2^15), none for 0, inf, NaN
            const int e = mx != 0 && ex < 255 ? min(126, max(-126, 141 - ex)) : 0;
            // the factor of the scores stays positive, and at least the smallest normal number (an
            // unseen score of -inf must stay one): a K scale's sign, or a NaN one, is in the query
            const float two_e = __int_as_float((127 + e) << 23);
            const float up = sc < 0.f ? -two_e : sc == sc ? two_e : sc;
            const float of = fmaxf(fabsf(sc) * __int_as_float((127 - e) << 23), 0x1p-126f);
            const float mine = __shfl_sync(0xffffffffu, of, 4 * (lane & 7));
            if ((lane >> 3) == g) x.sc = mine;
            if (wide || wg == 0) {
#pragma unroll
              for (int d = 0; d < RND; ++d) {
                uint32_t* w = &in[d][g].x;
#pragma unroll
                for (int k = 0; k < 4; ++k) w[k] = pack_f16(bf16lo(w[k]) * up, bf16hi(w[k]) * up);
              }
            }
          }
        }
        if constexpr (WIDE) {
          if (wide || wg == 0) {
            const int row0 = (warp & 3) * 32 + (lane >> 2);  // rows row0 + 8 g of the group
            const uint32_t at = ring + S::OFF_Q + wg * S::Q_GROUP + row0 * 128;
#pragma unroll
            for (int d = 0; d < RND; ++d) {
              const uint32_t ch = (((4 * d & 7) + (lane & 3)) ^ (row0 & 7)) << 4;
#pragma unroll
              for (int g = 0; g < 4; ++g)
                sts128(at + (d >> 1) * (kGroupThreads * 128) + g * 1024 + ch, in[d][g]);
            }
            fence_proxy_async_smem();
          }
        } else if (wg == 0) {
          const uint32_t stage = ring + S::OFF_STAGE + warp * 2048;
#pragma unroll
          for (int h = 0; h < RND / 2; ++h) {
            uint32_t w[32];  // 128 bytes of this lane's row
#pragma unroll
            for (int d = 0; d < 2; ++d) {
              __syncwarp();
#pragma unroll
              for (int g = 0; g < 4; ++g) {
                const int row = 8 * g + (lane >> 2);
                sts128(stage + row * 64 + (((lane & 3) ^ ((row >> 1) & 3)) << 4), in[2 * h + d][g]);
              }
              __syncwarp();
#pragma unroll
              for (int c = 0; c < 4; ++c) {
                const uint4 v = lds128(stage + lane * 64 + ((c ^ ((lane >> 1) & 3)) << 4));
                w[16 * d + 4 * c] = v.x;
                w[16 * d + 4 * c + 1] = v.y;
                w[16 * d + 4 * c + 2] = v.z;
                w[16 * d + 4 * c + 3] = v.w;
              }
            }
            tmem_st32(lane_t + kColQ + 32 * h, w);
          }
          tmem_wait_st();
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(q_ready);
    };
    Row me{};
    const TreeRun* next = get_run(0);
    if (next) {
      uint4 in[RND][4];
      me = find_row(*next);
      load_query(*next, me, in);
      store_query(*next, me, in);
    }
    for (; next; ++unit) {
      const TreeRun& run = *next;
      const bool wide = WIDE && run.rows > kGroupThreads, live = me.live;
      const int n = wide ? 2 * run.n : run.n;  // steps; this group's: wg, wg + 2, ...
      const int b = run.b, j = run.j, t = me.t;
      const float sc = me.sc;
      uint32_t* const bad = bad_nodes + 8 * (unit & 1);
      float m_used = -INFINITY, l = 0.f;
      Place<NV> at = base;
      Place<NK> k_at = k_base;
      if (!wide) {
        at.advance(wg);
        k_at.advance(wg);
      }
      int p0 = (run.tile0 + (wide ? 0 : wg)) * kTok;
      const int seen_by_all = min(run.req.base, run.req.read) - kTok;
      auto steps = [&](auto w_) {
      constexpr bool wide = decltype(w_)::value;
      for (int u = wg; ok && u < n; u += 2) {
        const int buf = u & 3;
        // V of the tile too: the MMA warps take a P as the word that it is there
        ok = mbar_wait(&full_v[at.st], at.par, a.err) &&
             mbar_wait(&s_done[buf], parity_of(ph, u), a.err);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        if ((warp & 3) == 0 && lane == 0) {
          // This tile's K is used up (a wide unit's once both groups say so). A stage of V is free
          // after two arrivals, the commits of its P V; a small unit's tile has only one.
          mbar_arrive_n(&free_k[k_at.st], wide ? 1 : 2);
          if (!wide) mbar_arrive(&free_v[at.st]);
        }
        k_at.advance(wide ? 1 : 2);
        const int mask = page_mask[at.st];
        tc_fence_after();
        uint32_t sr[64];
        const uint32_t scol = s_col<WIDE>(buf);
        tmem_ld32(lane_t + scol, *reinterpret_cast<uint32_t(*)[32]>(&sr[0]));
        tmem_ld32(lane_t + scol + 32, *reinterpret_cast<uint32_t(*)[32]>(&sr[32]));
        tmem_wait_ld();
        const bool masked = mask != (1 << kPages) - 1 || p0 > seen_by_all;
        if (masked) {
          uint64_t seen = live ? tree_seen(a, run.req, b, t, p0) : 0ull;
#pragma unroll
          for (int p = 0; p < kPages; ++p)
            if (!((mask >> p) & 1)) seen &= ~(0xffffull << (16 * p));
#pragma unroll
          for (int k = 0; k < 64; ++k)
            if (!((seen >> k) & 1)) sr[k] = __float_as_uint(-INFINITY);
          {
            // Mend V: two threads to a row. In a wide unit both groups do (and write every row they
            // look at): each group's P V waits for its own group only.
            const int vr = r >> 1, pos = p0 + vr;
            constexpr int CH = D / 16;  // 16-byte chunks of half a row
            const uint32_t vrow = ring + S::OFF_V + at.st * S::TILE + (vr >> 4) * PAGE_MMA +
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
                const uint32_t xa = vrow + (((c0 + c) ^ (vr & 7)) << 4);
                uint4 x = lds128(xa);
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
                if (here || wide) sts128(xa, x);
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
        float mx4[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) mx4[k] = __uint_as_float(sr[k]);
#pragma unroll
        for (int k = 4; k < 60; k += 8) {
#pragma unroll
          for (int m = 0; m < 4; ++m)
            mx4[m] = max3(mx4[m], __uint_as_float(sr[k + 2 * m]), __uint_as_float(sr[k + 2 * m + 1]));
        }
        const float mx = sc * max3(max3(mx4[0], mx4[1], mx4[2]),
                                   max3(mx4[3], __uint_as_float(sr[60]), __uint_as_float(sr[61])),
                                   fmaxf(__uint_as_float(sr[62]), __uint_as_float(sr[63])));
        // s sc - m is one FMA below: m is a rounded product, the product in the FMA is not, so that a row's
        // weights are all off by one factor, which their sum shares: up to 2^0.5 for |m| <= 2^24. For
        // larger m it would soon leave f16's range and then every range: there s sc is rounded as m is.
        // (A tile that counts has its maximum near m.)
        const bool huge = fabsf(mx) > 0x1p24f && mx != -INFINITY;
        // The reference m that P and O are scaled by: from the first tile's maximum, then moved only when
        // passed by far. In a wide unit it is the thread's own. Otherwise the two groups' tiles add
        // into one O, so m goes from step to step: this group's step takes it from the other's
        // last one, sets it and says so before anything else.
        const bool first = wide ? u == wg : u == 0;
        float m_before = m_used;
        if (!wide && u > 0) {
          ok = mbar_wait(&ref_set[1 - wg], ((ph_ref >> (1 - wg)) ^ (uint32_t)((u - 1) >> 1)) & 1u,
                         a.err);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          m_before = ref[r];
        }
        // (the difference, not m_before + lazy: past 2^26 that sum would round to several times as far)
        const float m_new = first || mx - m_before > kLazyLog2<W8> + kLiftLog2<W8> ? mx - kLiftLog2<W8> : m_before;
        const bool moved = !first && m_new != m_before;
        if (!wide) {
          if (first || moved) ref[r] = m_new;
          __syncwarp();
          if (lane == 0) mbar_arrive(&ref_set[wg]);
        }
        float factor = sc;
        if (__any_sync(0xffffffffu, moved || huge)) {  // (one vote for the two: most steps have neither)
          if (__any_sync(0xffffffffu, moved)) {  // rescale this warp's rows of O (in TMEM)
            constexpr int back = wide ? 2 : 1;  // to the last step that adds into this O
            ok = mbar_wait(&pv_done[(u - back) & 3], parity_of(ph, u - back), a.err);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            tc_fence_after();
            const float alpha = moved ? exp2f(m_before - m_new) : 1.f;
            const uint32_t ocol = kColO + (wide ? 128 * wg : 0);
#pragma unroll
            for (int cb = 0; cb < D / 32; ++cb) {
              uint32_t o[32];
              tmem_ld32(lane_t + ocol + 32 * cb, o);
              tmem_wait_ld();
#pragma unroll
              for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * alpha);
              tmem_st32(lane_t + ocol + 32 * cb, o);
            }
            tmem_wait_st();
          }
          if (__any_sync(0xffffffffu, huge)) {
#pragma unroll
            for (int k = 0; k < 32; ++k) {
              float s0, s1;
              unpack2(mul2(pack2(__uint_as_float(sr[2 * k]), __uint_as_float(sr[2 * k + 1])),
                           pack2(sc, sc)),
                      s0, s1);
              sr[2 * k] = __float_as_uint(s0);
              sr[2 * k + 1] = __float_as_uint(s1);
            }
            factor = 1.f;
          }
        }
        if (m_new != m_used) {  // the group's own sum, at the maximum of its last step
          l *= exp2f(m_used - m_new);
          m_used = m_new;
        }
        // P = 2^(s - m) over the first 32 columns of the tile's S buffer
        const float m_use = m_used == -INFINITY ? 0.f : m_used;
        uint32_t pw[32];
        uint64_t sum[4] = {0, 0, 0, 0};  // (pairs of zeros)
        const uint64_t sc2 = pack2(factor, factor), m2 = pack2(-m_use, -m_use);
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
        tmem_st32(lane_t + scol, pw);
        float s0, s1;
        unpack2(add2(add2(sum[0], sum[1]), add2(sum[2], sum[3])), s0, s1);
        l += s0 + s1;
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();  // (one arrival per warp: arrivals on one barrier go one by one)
        if (lane == 0) mbar_arrive(&p_ready[buf]);
        at.advance(wide ? 1 : 2);
        p0 += wide ? kTok : 2 * kTok;
      }
      };
      if constexpr (WIDE) {
        if (wide)
          steps(BoolConst<true>{});
        else
          steps(BoolConst<false>{});
      } else {
        steps(BoolConst<false>{});
      }
      // ---- the unit's rows ----
      uint4 in[RND][4];  // the next unit's queries, on their way during the waits
      next = get_run(unit + 1);
      Row then{};
      if (next) {
        then = find_row(*next);
        load_query(*next, then, in);
      }
      // the unit's last P V (wide: the group's) is done; the other group hears of it below
      const int last = wide ? n - 2 + wg : n - 1;
      if (ok && (wide || (last & 1) == wg))
        ok = mbar_wait(&pv_done[last & 3], parity_of(ph, last), a.err);
      ok = __all_sync(0xffffffffu, ok);
      tc_fence_after();
      if (!wide) ml[exchange_slot(unit, wg, r)] = make_float2(m_used, l);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(met);
      ok = mbar_wait(met, unit & 1, a.err) && ok;
      ok = __all_sync(0xffffffffu, ok);
      tc_fence_after();
      if (threadIdx.x < 8) bad_nodes[8 * ((unit + 1) & 1) + threadIdx.x] = 0;
      // wide: the group's own rows, all dims; else group wg writes dims wg D/2 .. of every row, whose
      // sum is the two groups', each at the maximum of its last step (O is at the larger, the last)
      float M = m_used, L = l;
      if (!wide) {
        const float2 x = ml[exchange_slot(unit, 0, r)], y = ml[exchange_slot(unit, 1, r)];
        M = fmaxf(x.x, y.x);
        const float Mu = M == -INFINITY ? 0.f : M;
        L = exp2f(x.x - Mu) * x.y + exp2f(y.x - Mu) * y.y;
      }
      const float vs = me.vs;
      const float f = run.whole ? (L != 0.f ? vs / L : 0.f) : vs;
      uint32_t any_bad = 0;
#pragma unroll
      for (int k = 0; k < 8; ++k) any_bad |= bad[k];
      // 32 dims from c on of this thread's row: finished, or a partial. Rows leave PIECE bytes of each
      // at a time through shared memory, LPR lanes writing a row's.
      constexpr int LPR = S::PIECE / 16;
      const uint32_t stage = ring + S::OFF_STAGE + warp * (32 * S::PIECE);
      auto place = [&](int row, int chunk) {  // (eight lanes touch eight different banks of 16 bytes)
        return stage + row * S::PIECE + ((chunk ^ ((row / (8 / LPR)) & (LPR - 1))) << 4);
      };
      const size_t out_off = row_at(run, me);
      const int part0 = ((int)blockIdx.x * 2 + run.slot) * kTreeTcRows + me.row - lane;
      auto leave = [&](const uint32_t (&v)[16], auto&& address) {
#pragma unroll
        for (int h = 0; h < 64 / S::PIECE; ++h) {
          __syncwarp();
#pragma unroll
          for (int c4 = 0; c4 < LPR; ++c4) {
            const uint32_t* x = v + 4 * (h * LPR + c4);
            sts128(place(lane, c4), make_uint4(x[0], x[1], x[2], x[3]));
          }
          __syncwarp();
#pragma unroll
          for (int g = 0; g < LPR; ++g) {
            const int row = (32 / LPR) * g + lane / LPR;
            const uint4 x = lds128(place(row, lane % LPR));
            const size_t at = __shfl_sync(0xffffffffu, (unsigned long long)out_off, row);
            if (__shfl_sync(0xffffffffu, (int)live, row))
              *reinterpret_cast<uint4*>(address(row, at) + h * S::PIECE + 16 * (lane % LPR)) = x;
          }
        }
      };
      auto emit = [&](int c, uint32_t (&o)[32]) {
        if (any_bad && live) {  // the infinite and NaN values of the nodes this row sees
          for (int nd = 0; nd < run.req.nodes; ++nd) {
            if (!((bad[nd >> 5] >> (nd & 31)) & 1)) continue;
            const int pos = run.req.base + nd;
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
        uint32_t v[16];
        if (run.whole) {
#pragma unroll
          for (int k = 0; k < 16; ++k)
            v[k] = L != 0.f ? pack_bf16(__uint_as_float(o[2 * k]) * f, __uint_as_float(o[2 * k + 1]) * f)
                            : 0u;
          leave(v, [&](int, size_t at) { return static_cast<uint8_t*>(a.out) + 2 * (at + c); });
        } else {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int k = 0; k < 16; ++k)
              v[k] = __float_as_uint(__uint_as_float(o[16 * h + k]) * f);
            leave(v, [&](int row, size_t) {
              return reinterpret_cast<uint8_t*>(a.ws_acc + (size_t)(part0 + row) * D + c + 16 * h);
            });
          }
          if (c == 0 && live)
            *reinterpret_cast<float2*>(a.ws_ml + 2 * (size_t)(part0 + lane)) = make_float2(M, L);
        }
      };
      // the next query first, so that the next unit's scores run while this one's rows are written
      if (next) store_query(*next, then, in);
      if (ok) {
        const int c_lo = wide ? 0 : wg * (D / 2), c_hi = wide ? D : c_lo + D / 2;
        for (int c = c_lo; c < c_hi; c += 32) {
          uint32_t o[32];
          tmem_ld32(lane_t + kColO + (wide ? 128 * wg : 0) + c, o);
          tmem_wait_ld();
          emit(c, o);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(o_read);
      ph = after_steps(ph, n);
      if (!wide) ph_ref ^= (uint32_t)(((n + 1) >> 1) & 1) | (uint32_t)((n >> 1) & 1) << 1;
      base.skip(run.n);
      k_base.skip(run.n);
      me = then;
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

template <typename KV, int D, bool WIDE>
cudaError_t launch_shape(const TreeArgs& a, const CUtensorMap& tk, const CUtensorMap& tv,
                     cudaStream_t s) {
  using S = TcShape<KV, D, WIDE>;
  static std::atomic<unsigned long long> attr_done{0};  // one bit per device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !((attr_done.load() >> dev) & 1ull)) {
    e = cudaFuncSetAttribute(tree_tc_kernel<KV, D, WIDE>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             S::SMEM);
    if (e != cudaSuccess) return e;
    // the softmax warps may take no more registers than the launch brings and the others give up
    cudaFuncAttributes fa{};
    e = cudaFuncGetAttributes(&fa, tree_tc_kernel<KV, D, WIDE>);
    if (e != cudaSuccess) return e;
    if (kSoftThreads * S::SOFT_REGS + (S::THREADS - kSoftThreads) * S::REGS >
        S::THREADS * fa.numRegs)
      return cudaErrorLaunchOutOfResources;
    if (dev < 64) attr_done.fetch_or(1ull << dev);
  }
  tree_tc_kernel<KV, D, WIDE><<<a.ctas, S::THREADS, S::SMEM, s>>>(a, tk, tv);
  return cudaGetLastError();
}

template <typename KV, int D>
cudaError_t launch_t(const TreeArgs& a, const CUtensorMap& tk, const CUtensorMap& tv,
                     cudaStream_t s) {
  return (long long)a.nodes * a.group > kGroupThreads ? launch_shape<KV, D, true>(a, tk, tv, s)
                                                      : launch_shape<KV, D, false>(a, tk, tv, s);
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
