// What the translation units of the C ABI share: descriptor checks, the device error word,
// tensor maps of the pools and launch tracing (all defined in capi.cu).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <atomic>

#include "pkv.h"
#include "pkv_host.h"

namespace pkv {

int check_desc(const pkv_cache_desc* d, const char* who);
int cuda_status(cudaError_t e, const char* what);
// Device address of the current device's error word (looked up once per device).
int error_word(int** out);

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline size_t align256(size_t x) { return (x + 255) & ~size_t(255); }
inline int dtype_bytes(int dtype) { return dtype == PKV_F32 ? 4 : dtype == PKV_BF16 ? 2 : 1; }
inline bool is_coded(int dtype) { return dtype == PKV_FP8_E4M3 || dtype == PKV_INT8; }

// The TMA view of a pool, encoded once per (device, pool, shape). A row of 128 bytes (FP8,
// INT8 at head_dim 128) is a 2-D tensor [num_pages * h_kv * 16 rows][128 bytes], one
// (page, KV head) tile per box of 16 rows. A bf16 row of 256 bytes is a 3-D tensor
// [2 halves][rows][64 elements] (halves 128 bytes apart, rows 256 bytes apart), so that one box
// of 2 x 16 x 64 moves a whole (page, KV head) tile into shared memory as two 128-byte-swizzled
// blocks of 16 rows, the first half of every row before the second (the layout the kernels
// read); *rank receives 2 or 3. force_2d asks for the 2-D view of a bf16 pool too (two boxes
// of 16 rows x 64 elements per tile).
int pool_tensor_map(const void* base, const pkv_cache_desc* d, CUtensorMap* out, int* rank,
                    bool force_2d = false);

// Launch tracing: while it is on, a launch is bracketed by two events recorded under `name`.
extern std::atomic<bool> g_trace_on;
cudaError_t trace_begin(cudaEvent_t (&ev)[2], cudaStream_t s);
void trace_end(const char* name, const cudaEvent_t (&ev)[2], cudaStream_t s);

template <class F>
cudaError_t traced(const char* name, cudaStream_t s, F&& launch) {
  if (!g_trace_on.load(std::memory_order_relaxed)) return launch();
  cudaEvent_t ev[2] = {nullptr, nullptr};
  cudaError_t e = trace_begin(ev, s);
  if (e != cudaSuccess) return e;
  e = launch();
  trace_end(name, ev, s);
  return e;
}

}  // namespace pkv
