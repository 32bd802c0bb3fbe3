// Norm of each query and key head, rotary position and cache append in one pass: the write phase
// of a decode or verification step taken from the projection's output.
//
// For token n and a query or key head row x of D values:
//   y_i = x_i * rsqrt(mean(x^2) + eps) * w_i            (w absent: y = x)
//   for the first R dims, pair i = 0 .. R/2 - 1 with (a, b) = (y_i, y_{i + R/2}), or
//   (y_{2i}, y_{2i+1}) when interleaved, and c, s = cos, sin of the token's position:
//     a' = a c - b s,  b' = b c + a s;  the dims from R on pass.
// The query row goes to q_out; the key row, and the value row unchanged, to the token's cache
// slot, rounded once from fp32 (FP8 / INT8: the code of the fp32 quotient by the head's scale).
//
// The pass is bound by memory -- every row is read once and written once -- as long as the dozen
// operations a value are not many more instructions. A row is held by D / VEC lanes of a warp, and
// each lane holds both values of its pairs: for halves i and i + R/2 two 8-byte chunks R/2 apart
// (past the rotated dims, two neighbouring ones), so that the rotation needs no shuffle and the sum
// of squares is the only reduction. What does not change from token to token (a row's kind, its
// addresses, its head's scale, the weights) is worked out once per block.
//
// Measured in graphs of calls over several states: 12345 tokens of 48 heads of 128 bf16 dims: 55 us,
// 5.6 TB/s, 83 % of the copy (rows loaded into registers a token ahead instead of copied through
// shared memory: 65; copied two tokens ahead 57, three 58, five 70: more reads under way get in the
// way of the writes); 1536 tokens of 80 heads into an FP8 cache: 20 us (9 at the copy's rate). No unit
// is at its limit there: DRAM 19 % busy, 109 warp instructions a row (74 in the long prompt) issue in
// 64 % of the active cycles from six warps a scheduler, and a fifth of the time passes before the first
// and after the last; a block has seven tokens to spread its beginning over, and parts of three and two
// row groups. fp32 rows, 12345 tokens of 48 heads of 128: 95 us (90 at the copy's rate).
#include <algorithm>
#include <math.h>

#include "pkv_device.cuh"
#include "pkv_internal.h"
#include "quantize.cuh"

namespace pkv {

namespace {

constexpr int kThreads = 256;
constexpr int kWave = 152 * 3;  // blocks resident at once (three on each SM)

template <typename TIN, int D>
struct RowShape {
  static constexpr int VEC = Vec16<TIN>::N;     // values of a lane
  static constexpr int CH = VEC / 2;            // values of a chunk (8 bytes)
  static constexpr int LPR = D / VEC;           // lanes of a row
  static constexpr int ROWS = kThreads / LPR;   // rows a block takes at a time
};

__device__ __forceinline__ void widen(const uint2& v, float (&o)[4]) {
  o[0] = bf16lo(v.x);
  o[1] = bf16hi(v.x);
  o[2] = bf16lo(v.y);
  o[3] = bf16hi(v.y);
}
__device__ __forceinline__ void widen(const uint2& v, float (&o)[2]) {
  o[0] = __uint_as_float(v.x);
  o[1] = __uint_as_float(v.y);
}
__device__ __forceinline__ void vec_load(const float* p, float (&o)[4]) {  // (16-byte aligned)
  const float4 v = *reinterpret_cast<const float4*>(p);
  o[0] = v.x;
  o[1] = v.y;
  o[2] = v.z;
  o[3] = v.w;
}
__device__ __forceinline__ void vec_load(const float* p, float (&o)[2]) {
  const float2 v = *reinterpret_cast<const float2*>(p);
  o[0] = v.x;
  o[1] = v.y;
}
__device__ __forceinline__ uint2 narrow(const float (&y)[4]) {
  const __nv_bfloat162 a = __floats2bfloat162_rn(y[0], y[1]), b = __floats2bfloat162_rn(y[2], y[3]);
  return make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}
__device__ __forceinline__ uint2 narrow(const float (&y)[2]) {
  return make_uint2(__float_as_uint(y[0]), __float_as_uint(y[1]));
}

// The codes of N values. Rows that were computed in fp32 are divided as such (TDIV float: always
// the IEEE division), unchanged rows of bf16 input as the quantising append divides them.
template <typename TDIV, int CACHE, int N>
__device__ __forceinline__ uint32_t codes_of(const float (&y)[N], const KnownDivisor& d) {
  float q[N];
  const bool slow = divide_vec<TDIV, N>(y, d, q);
  uint32_t w = 0;
  if constexpr (CACHE == PKV_FP8_E4M3) {
#pragma unroll
    for (int k = 0; k < N / 2; ++k)
      w |= (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(q[2 * k], q[2 * k + 1]), __NV_SATFINITE,
                                              __NV_E4M3)
           << (16 * k);
  } else {
#pragma unroll
    for (int k = 0; k < N; ++k) {
      if (slow) q[k] = q[k] == q[k] ? q[k] : 0.f;
      w |= (int8_code_bits(q[k]) & 0xffu) << (8 * k);
    }
  }
  return w;
}

// A chunk of a K or V row into its pool row at element `at`.
template <typename TDIV, int CACHE, int N>
__device__ __forceinline__ void store_chunk(void* pool, int64_t at, const KnownDivisor& d,
                                            const float (&y)[N]) {
  if constexpr (CACHE == PKV_F32 || CACHE == PKV_BF16) {
    *reinterpret_cast<uint2*>(static_cast<uint8_t*>(pool) + at * (8 / N)) = narrow(y);
  } else {
    const uint32_t w = codes_of<TDIV, CACHE, N>(y, d);
    uint8_t* p = static_cast<uint8_t*>(pool) + at;
    if constexpr (N == 4)
      *reinterpret_cast<uint32_t*>(p) = w;
    else
      *reinterpret_cast<uint16_t*>(p) = (uint16_t)w;
  }
}

// Row groups of a token a block takes at most; a token of more is shared by `parts` blocks (block
// b always takes part b % parts). The next token's rows, cos and sin are on their way while this one's
// are worked on, the position and slot of the one after it too.
constexpr int kGroups = 3;
constexpr int kDepth = 2;  // tokens of the ring of rows

__device__ __forceinline__ void copy8(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ uint2 lds64(uint32_t at) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(at) : "memory");
  return v;
}

template <typename TIN, int CACHE, int D, bool INTER>
__global__ void __launch_bounds__(kThreads, 3) qk_norm_rope_append_kernel(const NormRopeArgs a,
                                                                          int parts, int groups) {
  using S = RowShape<TIN, D>;
  constexpr int CH = S::CH, LPR = S::LPR, ROWS = S::ROWS, VEC = S::VEC;
  const int cl = threadIdx.x % LPR, rl = threadIdx.x / LPR;
  const int h_q = a.h_q, h_kv = a.h_kv, rows = h_q + 2 * h_kv;
  const int half = a.rot_dim / 2;
  // this lane's two chunks of a row, and the first of its columns in the table's halves
  const bool turns = cl * VEC < a.rot_dim;
  const int ca = turns ? cl * CH : a.rot_dim + (cl * VEC - a.rot_dim);
  const int cb = turns ? ca + half : ca + CH;
  __shared__ alignas(16) float weights[3][D];  // of queries, of keys, ones
  for (int i = threadIdx.x; i < D; i += kThreads) {
    weights[0][i] = a.q_weight ? load_as_float(static_cast<const TIN*>(a.q_weight), i) : 1.f;
    weights[1][i] = a.k_weight ? load_as_float(static_cast<const TIN*>(a.k_weight), i) : 1.f;
    weights[2][i] = 1.f;
  }
  __syncthreads();

  // This thread's rows: kind 0 query, 1 key, 2 value, 3 none. Addresses are of chunk a; chunk b lies
  // `over` elements behind it.
  const int part = blockIdx.x % parts, row0 = part * groups * ROWS + rl;
  const int over = cb - ca;
  const int64_t step = gridDim.x / parts, n0 = blockIdx.x / parts;
  int kind[kGroups];
  const TIN* src[kGroups];
  int64_t src_step[kGroups];
  TIN* q_out[kGroups];
  int in_slot[kGroups];  // elements from the token's first cache row to this row's chunk a
  KnownDivisor scale[kGroups];
  bool norm[kGroups], rows_to_turn[kGroups];  // (the latter uniform over a warp)
#pragma unroll
  for (int g = 0; g < kGroups; ++g) {
    const int r = row0 + g * ROWS;
    kind[g] = g >= groups || r >= rows ? 3 : r >= h_q + h_kv ? 2 : r >= h_q ? 1 : 0;
    const int head = kind[g] == 0 ? r : kind[g] == 1 ? r - h_q : kind[g] == 2 ? r - h_q - h_kv : 0;
    const int64_t stride = kind[g] == 0 ? a.q_stride : kind[g] == 1 ? a.k_stride : a.v_stride;
    src[g] = static_cast<const TIN*>(kind[g] == 0 ? a.q : kind[g] == 1 ? a.k : a.v) + n0 * stride +
             head * D + ca;
    src_step[g] = step * stride;
    q_out[g] = static_cast<TIN*>(a.q_out) + n0 * a.q_out_stride + head * D + ca;
    in_slot[g] = head * kPageSize * D + ca;
    norm[g] = kind[g] == 0 ? a.q_weight != nullptr : kind[g] == 1 && a.k_weight != nullptr;
    rows_to_turn[g] = __any_sync(0xffffffffu, kind[g] < 2);
    if constexpr (CACHE == PKV_FP8_E4M3 || CACHE == PKV_INT8)
      scale[g] = known_divisor(kind[g] == 1   ? a.k_scales[head]
                               : kind[g] == 2 ? a.v_scales[head]
                                              : 1.f);
  }
  const int64_t out_step = step * a.q_out_stride;

  struct Where {
    int pos;
    int64_t slot;
  };
  struct Token {
    Where at;
    float cs[CH], sn[CH];
  };
  // Rows come into a ring in shared memory, kDepth - 1 tokens ahead; a thread reads what it copied
  // itself, so it waits for its own copies only and no barrier is needed.
  __shared__ uint2 ring[kDepth * kGroups * 2 * kThreads];
  const uint32_t ring0 = smem_u32(ring) + 8 * threadIdx.x;
  constexpr uint32_t PART = 8 * kThreads, STAGE = 2 * kGroups * PART;
  uint32_t put = 0, get = 0;  // byte offsets of the stages
  auto copy_rows = [&](bool there) {  // (called for n0, n0 + step, ... in turn)
    if (there) {
#pragma unroll
      for (int g = 0; g < kGroups; ++g) {
        if (kind[g] != 3) {
          copy8(ring0 + put + 2 * g * PART, src[g]);
          copy8(ring0 + put + (2 * g + 1) * PART, src[g] + over);
        }
        src[g] += src_step[g];
      }
      put = put == (kDepth - 1) * STAGE ? 0 : put + STAGE;
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  auto look_up = [&](int64_t n) {
    if (n >= a.num_tokens) return Where{0, -1};
    return Where{a.rot_dim > 0 ? a.positions[n] : 0, a.slots[n]};
  };
  auto load_turn = [&](Token& t) {
    if (!turns || (unsigned)t.at.pos >= (unsigned)a.max_positions) return;
    const float* row = a.cos_sin + (int64_t)t.at.pos * a.rot_dim;
    if constexpr (INTER) {  // the pairs of chunk a, then of chunk b
#pragma unroll
      for (int e = 0; e < CH / 2; ++e) {
        t.cs[e] = row[ca / 2 + e];
        t.sn[e] = row[half + ca / 2 + e];
        t.cs[CH / 2 + e] = row[cb / 2 + e];
        t.sn[CH / 2 + e] = row[half + cb / 2 + e];
      }
    } else {
      vec_load(row + ca, t.cs);
      vec_load(row + half + ca, t.sn);
    }
  };
  auto work = [&](Token& t) {  // (likewise)
    const bool left_out = a.rot_dim > 0 && (unsigned)t.at.pos >= (unsigned)a.max_positions;
    bool stored = t.at.slot >= 0;
    if (left_out) {  // the whole token
      if (threadIdx.x == 0 && part == 0) atomicOr(a.err, PKV_DEVERR_BAD_POSITION);
    } else if (t.at.slot >= a.num_slots) {
      if (threadIdx.x == 0 && part == 0) atomicOr(a.err, PKV_DEVERR_BAD_SLOT);
      stored = false;
    }
    const uint64_t slot = (uint64_t)t.at.slot;
    const int64_t row0 = (int64_t)(((slot >> 4) * h_kv * kPageSize + (slot & 15)) * D);
    static_assert(kPageSize == 16, "slot arithmetic");
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
      if (left_out || g >= groups) break;  // (uniform over the block)
      float xa[CH], xb[CH];
      const uint2 ra = lds64(ring0 + get + 2 * g * PART);
      const uint2 rb = lds64(ring0 + get + (2 * g + 1) * PART);
      widen(ra, xa);
      widen(rb, xb);
      const int64_t at = row0 + in_slot[g];
      if (kind[g] == 2 && stored) {
        if constexpr (CACHE == PKV_F32 || CACHE == PKV_BF16) {  // the bits as they came (a NaN's too)
          TIN* v = static_cast<TIN*>(a.v_cache) + at;
          *reinterpret_cast<uint2*>(v) = ra;
          *reinterpret_cast<uint2*>(v + over) = rb;
        } else {
          store_chunk<TIN, CACHE, CH>(a.v_cache, at, scale[g], xa);
          store_chunk<TIN, CACHE, CH>(a.v_cache, at + over, scale[g], xb);
        }
      }
      if (!rows_to_turn[g]) continue;
      float ss = 0.f;
#pragma unroll
      for (int e = 0; e < CH; ++e) ss = fmaf(xa[e], xa[e], fmaf(xb[e], xb[e], ss));
#pragma unroll
      for (int o = LPR / 2; o >= 1; o /= 2) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      const float rstd = norm[g] ? rsqrtf(fmaf(ss, 1.f / D, a.eps)) : 1.f;
      const float* w = weights[kind[g] < 2 ? kind[g] : 2];
      float wa[CH], wb[CH];
      vec_load(w + ca, wa);
      vec_load(w + cb, wb);
#pragma unroll
      for (int e = 0; e < CH; ++e) {
        xa[e] *= rstd * wa[e];
        xb[e] *= rstd * wb[e];
      }
      if (turns) {
        if constexpr (INTER) {
#pragma unroll
          for (int e = 0; e < CH; e += 2) {
            const float a0 = xa[e], a1 = xa[e + 1], b0 = xb[e], b1 = xb[e + 1];
            const float ac = t.cs[e / 2], as = t.sn[e / 2];
            const float bc = t.cs[CH / 2 + e / 2], bs = t.sn[CH / 2 + e / 2];
            xa[e] = fmaf(a0, ac, -(a1 * as));
            xa[e + 1] = fmaf(a1, ac, a0 * as);
            xb[e] = fmaf(b0, bc, -(b1 * bs));
            xb[e + 1] = fmaf(b1, bc, b0 * bs);
          }
        } else {
#pragma unroll
          for (int e = 0; e < CH; ++e) {
            const float f = xa[e], s = xb[e];
            xa[e] = fmaf(f, t.cs[e], -(s * t.sn[e]));
            xb[e] = fmaf(s, t.cs[e], f * t.sn[e]);
          }
        }
      }
      if (kind[g] == 0) {
        *reinterpret_cast<uint2*>(q_out[g]) = narrow(xa);
        *reinterpret_cast<uint2*>(q_out[g] + over) = narrow(xb);
      } else if (kind[g] == 1 && stored) {
        store_chunk<float, CACHE, CH>(a.k_cache, at, scale[g], xa);
        store_chunk<float, CACHE, CH>(a.k_cache, at + over, scale[g], xb);
      }
    }
#pragma unroll
    for (int g = 0; g < kGroups; ++g) q_out[g] += out_step;
    get = get == (kDepth - 1) * STAGE ? 0 : get + STAGE;
  };

  Token even{}, odd{};
  even.at = look_up(n0);
  odd.at = look_up(n0 + step);
  for (int i = 0; i < kDepth - 1; ++i) copy_rows(n0 + i * step < a.num_tokens);
  load_turn(even);
  for (int64_t n = n0;;) {
    copy_rows(n + (kDepth - 1) * step < a.num_tokens);
    const bool second = n + step < a.num_tokens;
    if (second) load_turn(odd);
    asm volatile("cp.async.wait_group %0;" ::"n"(kDepth - 1) : "memory");
    const Where w2 = look_up(n + 2 * step);
    work(even);
    even.at = w2;
    if (!second) break;
    n += step;
    copy_rows(n + (kDepth - 1) * step < a.num_tokens);
    const bool third = n + step < a.num_tokens;
    if (third) load_turn(even);
    asm volatile("cp.async.wait_group %0;" ::"n"(kDepth - 1) : "memory");
    const Where w3 = look_up(n + 2 * step);
    work(odd);
    odd.at = w3;
    if (!third) break;
    n += step;
  }
}

template <typename TIN, int CACHE, int D>
cudaError_t launch_d(const NormRopeArgs& a, cudaStream_t s) {
  constexpr int R = RowShape<TIN, D>::ROWS;
  const int all = (a.h_q + 2 * a.h_kv + R - 1) / R;  // row groups of a token
  // few tokens: a block for every group; otherwise the fewest near-equal parts of <= kGroups
  int parts = (int64_t)a.num_tokens * all <= kWave ? all : (all + kGroups - 1) / kGroups;
  const int groups = (all + parts - 1) / parts;
  parts = (all + groups - 1) / groups;
  const int64_t tokens = std::min<int64_t>(a.num_tokens, std::max(1, kWave / parts));
  const int grid = (int)(tokens * parts);
  if (a.interleaved)
    qk_norm_rope_append_kernel<TIN, CACHE, D, true><<<grid, kThreads, 0, s>>>(a, parts, groups);
  else
    qk_norm_rope_append_kernel<TIN, CACHE, D, false><<<grid, kThreads, 0, s>>>(a, parts, groups);
  return cudaGetLastError();
}

template <typename TIN, int CACHE>
cudaError_t launch_t(const NormRopeArgs& a, cudaStream_t s) {
  return a.head_dim == 64 ? launch_d<TIN, CACHE, 64>(a, s) : launch_d<TIN, CACHE, 128>(a, s);
}

}  // namespace

cudaError_t launch_qk_norm_rope_append(const NormRopeArgs& a, int io_dtype, int cache_dtype,
                                       cudaStream_t s) {
  if (io_dtype == PKV_BF16) {
    if (cache_dtype == PKV_BF16) return launch_t<__nv_bfloat16, PKV_BF16>(a, s);
    if (cache_dtype == PKV_FP8_E4M3) return launch_t<__nv_bfloat16, PKV_FP8_E4M3>(a, s);
    return launch_t<__nv_bfloat16, PKV_INT8>(a, s);
  }
  if (cache_dtype == PKV_F32) return launch_t<float, PKV_F32>(a, s);
  if (cache_dtype == PKV_FP8_E4M3) return launch_t<float, PKV_FP8_E4M3>(a, s);
  return launch_t<float, PKV_INT8>(a, s);
}

}  // namespace pkv
