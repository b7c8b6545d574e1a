// Internal declarations shared by the optimiser and quantised-linear operators: their host layer
// (host_ops.cpp) and kernels (optim_kernels.hip, int4_kernels.hip, linear_kernels.hip).
#pragma once
#include <stddef.h>
#include <stdint.h>

#include "bcjr.h"

namespace bcjr {

// x [tokens, cols] and y [tokens, rows] of a product with quantised weights.
struct MatvecIO {
  const void* x;
  void* y;
  int64_t tokens, x_stride, y_stride;
  int dtype;
};

int launch_code_matvec(int n, int k, const uint32_t* code, int64_t rows, int64_t cols, int64_t L,
                       const float* codebook, const float* scales, const MatvecIO& io, void* stream);

// The tiled products with trellis-coded weights, one type each (code_tiles.hip, built once for each).
struct CodeArgs;
int launch_code_tiles_f32(const CodeArgs& a, int k, void* stream);
int launch_code_tiles_f16(const CodeArgs& a, int k, void* stream);
int launch_code_tiles_bf16(const CodeArgs& a, int k, void* stream);

int launch_int4_quantize(const void* w, int dtype, int64_t rows, int64_t cols, int64_t group,
                         uint32_t* q, float* scales, uint8_t* zeros, void* stream);
int launch_int4_dequantize(const uint32_t* q, const float* scales, const uint8_t* zeros,
                           int64_t rows, int64_t cols, int64_t group, float* w, void* stream);
int launch_int4_matvec(const uint32_t* q, const float* scales, const uint8_t* zeros, int64_t rows,
                       int64_t cols, int64_t group, const MatvecIO& io, void* stream);

// Moments lie in blocks of 32 elements; a tensor begins at a block.
constexpr int kMomentBlock = 32;
inline int64_t moment_numel(int64_t numel) { return (numel + kMomentBlock - 1) / kMomentBlock * kMomentBlock; }

struct AdamwState {
  void *avg, *sq;
  uint8_t *avg_scale, *sq_scale;
  int bits;
};

int launch_adamw(const bcjr_adamw_tensor* tensors, int64_t count, int param_type, int grad_type,
                 const bcjr_adamw& hyper, const AdamwState& state, void* stream);

}  // namespace bcjr
