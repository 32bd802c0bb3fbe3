// Rounding of cache rows: 16-byte input vectors widened to float, and their FP8 E4M3 or INT8
// codes. Shared by the quantising append and the fused norm + rotation + append.
#pragma once

#include <math.h>

#include "pkv_device.cuh"

namespace pkv {

template <typename TIN>
struct Vec16;  // one 16-byte vector of input elements, widened to float
template <>
struct Vec16<float> {
  static constexpr int N = 4;
  __device__ __forceinline__ static void load(const void* p, float (&o)[4]) {
    float4 v = *reinterpret_cast<const float4*>(p);
    o[0] = v.x;
    o[1] = v.y;
    o[2] = v.z;
    o[3] = v.w;
  }
};
template <>
struct Vec16<__nv_bfloat16> {
  static constexpr int N = 8;
  __device__ __forceinline__ static void load(const void* p, float (&o)[8]) {
    uint4 v = *reinterpret_cast<const uint4*>(p);
    o[0] = bf16lo(v.x);
    o[1] = bf16hi(v.x);
    o[2] = bf16lo(v.y);
    o[3] = bf16hi(v.y);
    o[4] = bf16lo(v.z);
    o[5] = bf16hi(v.z);
    o[6] = bf16lo(v.w);
    o[7] = bf16hi(v.w);
  }
};

// x / s, correctly rounded to fp32, for a divisor known in advance (the head's scale): with
// r = RN(1/s) computed once, q0 = RN(x r) and one FMA correction q = RN(q0 - r RN(q0 s - x))
// (Markstein's correction step; Brisebarre, Muller and Raina, "Accelerating correctly rounded
// floating-point division when the divisor is known in advance", IEEE Trans. Computers 53(8),
// 2004, study exactly this case). For x with at most 8 significant bits -- every bf16 value --
// and any fp32 s, q equals the IEEE quotient: checked exhaustively over the 2^7 bf16
// significands and the 2^23 fp32 significands of s, which covers every exponent as long as
// no intermediate is subnormal or overflows. That holds for s in [2^-80, 2^80] whenever the
// quotient matters (|q| >= 2^-13; smaller quotients give the code 0 either way). The remainder
// is taken as q0 s - x and subtracted, which equals adding x - q0 s exactly (rounding to
// nearest is symmetric) and keeps the sign of a zero quotient: -0 / s gives -0. Anything else
// -- s outside that range, an infinite or NaN x or an overflow, which all leave a NaN in q --
// takes the IEEE division for the whole vector.
// fp32 inputs (24-bit significands) always take the IEEE division.
struct KnownDivisor {
  float s, r;
  bool fast;
};

__device__ __forceinline__ KnownDivisor known_divisor(float scale) {
  KnownDivisor d;
  d.s = scale;
  d.r = __fdiv_rn(1.f, scale);
  d.fast = scale >= 0x1p-80f && scale <= 0x1p80f;  // (false for NaN)
  return d;
}

// Returns true where the vector took the IEEE division (NaN quotients stay NaN there).
template <typename TIN, int N>
__device__ __forceinline__ bool divide_vec(const float (&x)[N], const KnownDivisor& d,
                                           float (&q)[N]) {
  bool slow = sizeof(TIN) == 4 || !d.fast;
  if (!slow) {
    float sum = 0.f;
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const float q0 = __fmul_rn(x[k], d.r);
      q[k] = __fmaf_rn(-__fmaf_rn(q0, d.s, -x[k]), d.r, q0);
      sum = __fadd_rn(sum, q[k]);
    }
    // a NaN quotient makes the sum NaN; so can two infinite ones of opposite signs, which the
    // IEEE division then gives again
    slow = sum != sum;
  }
  if (slow) {
#pragma unroll
    for (int k = 0; k < N; ++k) q[k] = __fdiv_rn(x[k], d.s);
  }
  return slow;
}

template <typename TIN, int N>
__device__ __forceinline__ void quantize_store(const float (&x)[N], const KnownDivisor& d,
                                               uint8_t* dst) {
  float y[N];
  divide_vec<TIN, N>(x, d, y);
  uint16_t codes[N / 2];
#pragma unroll
  for (int k = 0; k < N / 2; ++k)
    codes[k] = static_cast<uint16_t>(__nv_cvt_float2_to_fp8x2(make_float2(y[2 * k], y[2 * k + 1]),
                                                              __NV_SATFINITE, __NV_E4M3));
  if constexpr (N == 8) {
    uint2 w;
    w.x = (uint32_t)codes[0] | ((uint32_t)codes[1] << 16);
    w.y = (uint32_t)codes[2] | ((uint32_t)codes[3] << 16);
    __stcs(reinterpret_cast<uint2*>(dst), w);
  } else {
    __stcs(reinterpret_cast<uint32_t*>(dst), (uint32_t)codes[0] | ((uint32_t)codes[1] << 16));
  }
}

// The INT8 code of y -- y rounded to the nearest integer, ties to even, and clamped to
// [-127, 127] -- in the low byte of the result. Clamping first changes nothing (the bounds are
// integers); adding 1.5 * 2^23 to a value in [-127, 127] gives a sum in [2^23, 2^24), whose
// last significand bit has weight 1, so the addition itself rounds to the nearest integer
// (ties to even: 1.5 * 2^23 is even) and the sum's representation is that of 1.5 * 2^23 plus
// the integer, two's complement in the low bits.
__device__ __forceinline__ uint32_t int8_code_bits(float y) {
  return __float_as_uint(__fadd_rn(fminf(fmaxf(y, -127.f), 127.f), 12582912.f));
}

// INT8 codes of N values: fp32(x / s) rounded to nearest even, clamped to [-127, 127]
// (a NaN quotient gives the code 0).
template <typename TIN, int N>
__device__ __forceinline__ void quantize_store_int8(const float (&x)[N], const KnownDivisor& d,
                                                    uint8_t* dst) {
  float y[N];
  if (divide_vec<TIN, N>(x, d, y)) {
#pragma unroll
    for (int k = 0; k < N; ++k) y[k] = y[k] == y[k] ? y[k] : 0.f;
  }
  uint32_t w[N / 4];
#pragma unroll
  for (int k = 0; k < N / 4; ++k) {
    // low bytes of four codes into one word: (c0, c1) and (c2, c3), then the two pairs
    const uint32_t c01 = __byte_perm(int8_code_bits(y[4 * k]), int8_code_bits(y[4 * k + 1]),
                                     0x0040);
    const uint32_t c23 = __byte_perm(int8_code_bits(y[4 * k + 2]), int8_code_bits(y[4 * k + 3]),
                                     0x0040);
    w[k] = __byte_perm(c01, c23, 0x5410);
  }
  if constexpr (N == 8) {
    __stcs(reinterpret_cast<uint2*>(dst), make_uint2(w[0], w[1]));
  } else {
    __stcs(reinterpret_cast<uint32_t*>(dst), w[0]);
  }
}

}  // namespace pkv
