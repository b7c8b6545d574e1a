// Device helpers of the optimiser and quantised-linear kernels: element types and wave sums.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "bcjr.h"

namespace bcjr {
namespace {

struct F32 {
  using T = float;
  static __device__ float load(const float* p) { return *p; }
  static __device__ void store(float* p, float v) { *p = v; }
};
struct F16 {
  using T = _Float16;
  static __device__ float load(const _Float16* p) { return (float)*p; }
  static __device__ void store(_Float16* p, float v) { *p = (_Float16)v; }
};
struct BF16 {
  using T = __bf16;
  static __device__ float load(const __bf16* p) { return (float)*p; }
  static __device__ void store(__bf16* p, float v) { *p = (__bf16)v; }  // to nearest, ties to even
};

// Sum over the 64 lanes, the same in every lane.
__device__ inline float wave_sum(float v) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) v += __shfl_xor(v, d, 64);
  return v;
}

}  // namespace

// Calls f with the element type of a dtype code (checked by the host layer).
template <class Fn>
inline int with_type(int dtype, Fn f) {
  return dtype == BCJR_F32 ? f(F32{}) : dtype == BCJR_F16 ? f(F16{}) : f(BF16{});
}

// Groups of a one-dimensional launch, at most 2^20: kernels stride over what is left.
inline unsigned grid_of(int64_t groups) {
  return (unsigned)(groups < (1 << 20) ? groups : (1 << 20));
}

}  // namespace bcjr
