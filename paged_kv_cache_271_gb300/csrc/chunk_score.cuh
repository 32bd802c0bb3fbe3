// Scores of the chunk operators on CUDA cores: their form and their loads.
#pragma once

#include <math.h>

#include "pkv_device.cuh"
#include "pkv_internal.h"

namespace pkv {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// A score in the log2 domain, from the product of a query and a key.
struct ScoreForm {
  float scale, cap_in, cap;  // without a cap: scale log2(e); with one: cap tanh(cap_in x), log2 domain
  __device__ __forceinline__ ScoreForm(const ChunkArgs& a, float k_scale) {
    scale = a.scale * k_scale * kLog2e;
    cap = a.softcap * kLog2e;
    cap_in = a.softcap > 0.f ? a.scale * k_scale / a.softcap : 0.f;
  }
  __device__ __forceinline__ float operator()(float x, float slope_log2, int distance) const {
    const float s = cap > 0.f ? cap * tanhf(x * cap_in) : x * scale;
    return slope_log2 != 0.f ? fmaf(-slope_log2, (float)distance, s) : s;
  }
};

// Four elements of a row as fp32.
__device__ __forceinline__ float4 load4(const float* p) {
  return *reinterpret_cast<const float4*>(p);
}
__device__ __forceinline__ float4 load4(const __nv_bfloat16* p) {
  const uint2 w = *reinterpret_cast<const uint2*>(p);
  return make_float4(bf16lo(w.x), bf16hi(w.x), bf16lo(w.y), bf16hi(w.y));
}

}  // namespace pkv
