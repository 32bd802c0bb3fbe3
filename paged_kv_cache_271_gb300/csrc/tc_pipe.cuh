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

template <int N>
__device__ __forceinline__ void regs_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// Queries of 32 rows for an 8-bit cache: bf16 to f16, scaled by a row's 2^e that puts its largest value
// in f16's top binade. in[d][g]: chunk lane % 4 of 64-byte round d of row 8 g + lane / 4 (the four lanes
// that hold a row agree). sc is the score factor of the KV head (log2 domain); mine receives that of this
// lane's row with its 2^-e. It stays positive, and at least the smallest normal number (an unseen
// score of -inf must stay one): a K scale's sign, or a NaN one, goes into the queries.
template <int RND>
__device__ __forceinline__ void query_to_f16(uint4 (&in)[RND][4], const float sc, float& mine) {
  const int lane = threadIdx.x & 31;
  float own = 0.f;
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
    const float two_e = __int_as_float((127 + e) << 23);
    const float up = sc < 0.f ? -two_e : sc == sc ? two_e : sc;
    const float of = fmaxf(fabsf(sc) * __int_as_float((127 - e) << 23), 0x1p-126f);
    const float theirs = __shfl_sync(0xffffffffu, of, 4 * (lane & 7));
    if ((lane >> 3) == g) own = theirs;
#pragma unroll
    for (int d = 0; d < RND; ++d) {
      uint32_t* w = &in[d][g].x;
#pragma unroll
      for (int k = 0; k < 4; ++k) w[k] = pack_f16(bf16lo(w[k]) * up, bf16hi(w[k]) * up);
    }
  }
  mine = own;
}

// tanh x = 1 - 2 / (1 + e^{2x}): off by at most some 2^-22, with the exact limits at infinities.
__device__ __forceinline__ float tanh_of(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + ex2_approx(2.f * kLog2e * x)));
  return fmaf(-2.f, r, 1.f);
}

}  // namespace pkv
