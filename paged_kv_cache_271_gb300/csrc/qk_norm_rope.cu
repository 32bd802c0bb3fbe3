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
// The pass is bound by memory: every row is read once and written once, about ten operations a
// value. A row is held by LPR lanes of a warp, 16 bytes each, so its sum of squares is a shuffle
// reduction inside the row's lanes and the rotation's partner values come by one shuffle (R/2
// dims is a whole number of lanes) or sit in the same lane (interleaved).
#include <algorithm>
#include <math.h>

#include "pkv_device.cuh"
#include "pkv_internal.h"
#include "quantize.cuh"

namespace pkv {

namespace {

constexpr int kThreads = 256;

template <typename TIN, int D>
struct RowShape {
  static constexpr int VEC = Vec16<TIN>::N;
  static constexpr int LPR = D / VEC;           // lanes of a row
  static constexpr int ROWS = kThreads / LPR;   // rows a block takes at a time
};

__device__ __forceinline__ uint4 pack_vec(const float (&y)[8]) {
  uint4 v;
  uint32_t* w = &v.x;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(y[2 * k], y[2 * k + 1]);
    w[k] = *reinterpret_cast<const uint32_t*>(&p);
  }
  return v;
}
__device__ __forceinline__ uint4 pack_vec(const float (&y)[4]) {
  return make_uint4(__float_as_uint(y[0]), __float_as_uint(y[1]), __float_as_uint(y[2]),
                    __float_as_uint(y[3]));
}

// One 16-byte vector (column cl of a row) of a K or V row into its pool row. Rows that were
// computed in fp32 are divided as such (float: always the IEEE division); unchanged rows of bf16
// input as the quantising append divides them.
template <typename TDIV, int CACHE, int VEC>
__device__ __forceinline__ void store_cache(void* pool, int64_t row, int D, int cl, float scale,
                                            const float (&y)[VEC]) {
  const int64_t at = row * D + cl * VEC;
  if constexpr (CACHE == PKV_FP8_E4M3) {
    quantize_store<TDIV, VEC>(y, known_divisor(scale), static_cast<uint8_t*>(pool) + at);
  } else if constexpr (CACHE == PKV_INT8) {
    quantize_store_int8<TDIV, VEC>(y, known_divisor(scale), static_cast<uint8_t*>(pool) + at);
  } else {
    constexpr int EB = CACHE == PKV_F32 ? 4 : 2;
    *reinterpret_cast<uint4*>(static_cast<uint8_t*>(pool) + at * EB) = pack_vec(y);
  }
}

// A block takes one token and the row groups blockIdx.y, blockIdx.y + gridDim.y, ... of its
// h_q + 2 h_kv rows (queries, keys, values), ROWS rows at a time. A lane keeps its columns, so
// the token's cos and sin of those columns are read once.
template <typename TIN, int CACHE, int D>
__global__ void __launch_bounds__(kThreads) qk_norm_rope_append_kernel(const NormRopeArgs a) {
  using S = RowShape<TIN, D>;
  constexpr int VEC = S::VEC, LPR = S::LPR, ROWS = S::ROWS;
  const int64_t n = blockIdx.x;
  const int lane = threadIdx.x & 31, cl = threadIdx.x % LPR, rl = threadIdx.x / LPR;
  const int col = cl * VEC;
  const int pos = a.rot_dim > 0 ? a.positions[n] : 0;
  if (a.rot_dim > 0 && (pos < 0 || pos >= a.max_positions)) {  // the whole token is left out
    if (threadIdx.x == 0 && blockIdx.y == 0) atomicOr(a.err, PKV_DEVERR_BAD_POSITION);
    return;
  }
  int64_t slot = a.slots[n];
  if (slot >= a.num_slots) {
    if (threadIdx.x == 0 && blockIdx.y == 0) atomicOr(a.err, PKV_DEVERR_BAD_SLOT);
    slot = -1;
  }
  const int64_t crow0 = (slot / kPageSize) * a.h_kv * kPageSize + slot % kPageSize;

  // cos and sin of this lane's values; a value's partner is `far` lanes away (0: in this lane)
  float cs[VEC], sn[VEC];
  const int half = a.rot_dim / 2;
  const bool turns = col < a.rot_dim;
  int partner = lane;
  if (turns) {
    const float* row = a.cos_sin + (int64_t)pos * a.rot_dim;
    if (a.interleaved) {
#pragma unroll
      for (int k = 0; k < VEC; ++k) {
        cs[k] = row[(col + k) / 2];
        sn[k] = row[half + (col + k) / 2];
        if ((k & 1) == 0) sn[k] = -sn[k];
      }
    } else {
      const bool upper = col >= half;
      const int c0 = upper ? col - half : col;
      partner = upper ? lane - half / VEC : lane + half / VEC;
#pragma unroll
      for (int k = 0; k < VEC; k += 4) {
        const float4 c4 = *reinterpret_cast<const float4*>(row + c0 + k);
        const float4 s4 = *reinterpret_cast<const float4*>(row + half + c0 + k);
        cs[k] = c4.x; cs[k + 1] = c4.y; cs[k + 2] = c4.z; cs[k + 3] = c4.w;
        sn[k] = upper ? s4.x : -s4.x;
        sn[k + 1] = upper ? s4.y : -s4.y;
        sn[k + 2] = upper ? s4.z : -s4.z;
        sn[k + 3] = upper ? s4.w : -s4.w;
      }
    }
  } else {
#pragma unroll
    for (int k = 0; k < VEC; ++k) {
      cs[k] = 1.f;
      sn[k] = 0.f;
    }
  }

  const int h_q = a.h_q, h_kv = a.h_kv, rows = h_q + 2 * h_kv;
  for (int r0 = blockIdx.y * ROWS; r0 < rows; r0 += gridDim.y * ROWS) {
    const int r = r0 + rl;
    // 0 query, 1 key, 2 value, 3 nothing to do
    const int kind = r >= rows ? 3 : r >= h_q + h_kv ? 2 : r >= h_q ? 1 : 0;
    const bool live = kind == 0 || (kind < 3 && slot >= 0);
    const int h = kind == 0 ? r : kind == 1 ? r - h_q : r - h_q - h_kv;
    const TIN* src = kind == 0 ? static_cast<const TIN*>(a.q) + n * a.q_stride
                   : kind == 1 ? static_cast<const TIN*>(a.k) + n * a.k_stride
                               : static_cast<const TIN*>(a.v) + n * a.v_stride;
    uint4 raw = make_uint4(0, 0, 0, 0);
    if (live) raw = __ldcs(reinterpret_cast<const uint4*>(src + (int64_t)h * D + col));
    float x[VEC];
    Vec16<TIN>::load(&raw, x);
    if (kind == 2) {
      if (live)
        store_cache<TIN, CACHE, VEC>(a.v_cache, crow0 + (int64_t)h * kPageSize, D, cl,
                                     a.v_scales ? a.v_scales[h] : 1.f, x);
    }
    const TIN* w = static_cast<const TIN*>(kind == 0 ? a.q_weight : kind == 1 ? a.k_weight : nullptr);
    float ss = 0.f;
#pragma unroll
    for (int k = 0; k < VEC; ++k) ss = fmaf(x[k], x[k], ss);
#pragma unroll
    for (int o = LPR / 2; o >= 1; o /= 2) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    if (w) {
      const float rstd = rsqrtf(fmaf(ss, 1.f / D, a.eps));
      float wv[VEC];
      Vec16<TIN>::load(w + col, wv);
#pragma unroll
      for (int k = 0; k < VEC; ++k) x[k] = x[k] * rstd * wv[k];
    }
    float y[VEC];
    if (a.interleaved) {
#pragma unroll
      for (int k = 0; k < VEC; ++k) y[k] = fmaf(x[k], cs[k], x[k ^ 1] * sn[k]);
    } else {
#pragma unroll
      for (int k = 0; k < VEC; ++k) {
        const float o = __shfl_sync(0xffffffffu, x[k], partner);
        y[k] = fmaf(x[k], cs[k], o * sn[k]);
      }
    }
    if (!turns) {  // (not x * 1 + o * 0: o may be infinite)
#pragma unroll
      for (int k = 0; k < VEC; ++k) y[k] = x[k];
    }
    if (kind == 0)
      *reinterpret_cast<uint4*>(static_cast<TIN*>(a.q_out) + n * a.q_out_stride + (int64_t)h * D +
                                col) = pack_vec(y);
    else if (kind == 1 && live)
      store_cache<float, CACHE, VEC>(a.k_cache, crow0 + (int64_t)h * kPageSize, D, cl,
                                     a.k_scales ? a.k_scales[h] : 1.f, y);
  }
}

template <typename TIN, int CACHE>
cudaError_t launch_t(const NormRopeArgs& a, cudaStream_t s) {
  const int rows = a.h_q + 2 * a.h_kv;
  auto go = [&](auto kern, int rows_per_pass) {
    const int passes = (rows + rows_per_pass - 1) / rows_per_pass;
    // few tokens: a block for every pass of a token; many: a block for every token
    const int split = std::min<int64_t>(passes, std::max<int64_t>(1, 152 * 8 / a.num_tokens));
    kern<<<dim3(a.num_tokens, split), kThreads, 0, s>>>(a);
  };
  if (a.head_dim == 64)
    go(qk_norm_rope_append_kernel<TIN, CACHE, 64>, RowShape<TIN, 64>::ROWS);
  else
    go(qk_norm_rope_append_kernel<TIN, CACHE, 128>, RowShape<TIN, 128>::ROWS);
  return cudaGetLastError();
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
