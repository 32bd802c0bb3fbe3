// Pieces shared by the tcgen05 kernels on chunks of new tokens: places in rings of shared memory, the
// registers' split between warps, queries for an 8-bit cache, the cap's tanh.
#pragma once

#include <stdint.h>

#include "chunk_score.cuh"
#include "paged_decode_mma.cuh"
#include "pkv_device.cuh"
#include "tcgen05.cuh"

namespace pkv {

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

// Whether the phase with the given parity is over, without waiting for it.
__device__ __forceinline__ bool mbar_test(uint64_t* bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n.reg .pred p;\nmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n"
      "selp.u32 %0, 1, 0, p;\n}"
      : "=r"(done)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return done != 0;
}

template <int N>
__device__ __forceinline__ void regs_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// A row of queries for an 8-bit cache: bf16 to f16, scaled by 2^e that puts the row's largest value in
// f16's top binade. Four lanes hold a row, chunk lane % 4 of each 64-byte round in in[d]. sc is the score
// factor of the KV head (log2 domain); the row's own, with 2^-e, is returned. It stays positive, and at
// least the smallest normal number (an unseen score of -inf must stay one): a K scale's sign, or a NaN
// one, goes into the queries.
template <int RND>
__device__ __forceinline__ float query_to_f16(uint4 (&in)[RND], const float sc) {
  uint32_t lo = 0, hi = 0;  // largest |q| as bits (bf16 magnitudes order like integers)
#pragma unroll
  for (int d = 0; d < RND; ++d) {
    const uint32_t* w = &in[d].x;
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
  const float two_e = __int_as_float((127 + e) << 23);
  const float up = sc < 0.f ? -two_e : sc == sc ? two_e : sc;
#pragma unroll
  for (int d = 0; d < RND; ++d) {
    uint32_t* w = &in[d].x;
#pragma unroll
    for (int k = 0; k < 4; ++k) w[k] = pack_f16(bf16lo(w[k]) * up, bf16hi(w[k]) * up);
  }
  return fmaxf(fabsf(sc) * __int_as_float((127 - e) << 23), 0x1p-126f);
}

// 3-D tiled TMA load of one box into shared memory, completing on `bar` (x a multiple of 8 elements).
__device__ __forceinline__ void tma_load_box(uint32_t smem_dst, const CUtensorMap* map, int x, int y,
                                             int z, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
      : "memory");
}

// 16 consecutive columns of this thread's lane of tensor memory.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, "
      "[%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]),
        "=r"(r[15])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

// 16 rows x 32 fp32 columns of tensor memory: r[4 n + 2 b + m] is column 8 n + 2 (lane % 4) + m of row
// lane / 4 + 8 b.
__device__ __forceinline__ void tmem_ld_16x256(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, "
      "[%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]),
        "=r"(r[15])
      : "r"(taddr));
}

// Of four lanes with four words each: lane q4 gets word q4 of every lane, in lane order.
__device__ __forceinline__ void quad_transpose(uint32_t (&x)[4], int q4) {
  const bool odd = q4 & 1, high = q4 & 2;
#pragma unroll
  for (int k = 0; k < 4; k += 2) {
    const uint32_t y = __shfl_xor_sync(0xffffffffu, odd ? x[k] : x[k + 1], 1);
    (odd ? x[k] : x[k + 1]) = y;
  }
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const uint32_t y = __shfl_xor_sync(0xffffffffu, high ? x[k] : x[k + 2], 2);
    (high ? x[k] : x[k + 2]) = y;
  }
}

// Two scores side by side.
__device__ __forceinline__ uint64_t get2(const uint32_t* s) {
  return pack2(__uint_as_float(s[0]), __uint_as_float(s[1]));
}
__device__ __forceinline__ void put2(uint32_t* s, uint64_t v) {
  float x, y;
  unpack2(v, x, y);
  s[0] = __float_as_uint(x);
  s[1] = __float_as_uint(y);
}

// N scores of each lane capped: s <- top tanh(in s). Where all of a warp's are at most 0.7 times the cap,
// as scores mostly are, tanh x = x P(x^2) with a polynomial of degree 5 that interpolates tanh(x) / x at
// the Chebyshev nodes of x^2 in [0, 0.49] (off by at most 8e-9, in fp32 7e-8), in paired FMAs; otherwise
// tanh x = 1 - 2 / (1 + e^{2x}), whose exponential and reciprocal take the special-function unit
// three times as long as the weights' own exponentials (off by some 2^-22, with the exact limits at
// infinities).
template <int N>
__device__ __forceinline__ void cap_scores(uint32_t* s, float in, float top) {
  float most = 0.f;
#pragma unroll
  for (int k = 0; k < N; k += 2)
    most = max3(most, fabsf(__uint_as_float(s[k])), fabsf(__uint_as_float(s[k + 1])));
  const uint64_t in2 = pack2(in, in);
  if (__all_sync(0xffffffffu, most * fabsf(in) <= 0.7f)) {  // (NaNs, which max3 passes over, stay NaN)
    constexpr float C[6] = {-0.005084393545985222f, 0.02001960761845112f, -0.053523916751146317f,
                            0.13328377902507782f,   -0.33333128690719604f, 1.f};
    uint64_t c[6];
#pragma unroll
    for (int i = 0; i < 6; ++i) c[i] = pack2(C[i] * top, C[i] * top);
#pragma unroll
    for (int k = 0; k < N; k += 2) {
      const uint64_t x = mul2(get2(&s[k]), in2), u = mul2(x, x);
      uint64_t p = c[0];
#pragma unroll
      for (int i = 1; i < 6; ++i) p = fma2(p, u, c[i]);
      put2(&s[k], mul2(x, p));
    }
  } else {
#pragma unroll
    for (int k = 0; k < N; ++k) {
      float r;
      asm("rcp.approx.ftz.f32 %0, %1;"
          : "=f"(r)
          : "f"(1.f + ex2_approx(2.f * kLog2e * in * __uint_as_float(s[k]))));
      s[k] = __float_as_uint(fmaf(-2.f * top, r, top));
    }
  }
}

}  // namespace pkv
