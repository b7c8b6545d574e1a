// Host layer of the optimiser and quantised-linear entry points (include/bcjr.h): argument checks and
// dispatch. Every check runs before anything touches the HIP runtime.
#include <math.h>
#include <stdlib.h>

#include "bcjr.h"
#include "internal.h"
#include "ops.h"

using namespace bcjr;

namespace {

constexpr int64_t kMaxElements = (int64_t)1 << 40;
constexpr int64_t kInt4Columns = (int64_t)1 << 24;  // the kernels hold columns in 32 bits (tiles.h)

bool dtype_ok(int t) { return t == BCJR_F32 || t == BCJR_F16 || t == BCJR_BF16; }
int dtype_size(int t) { return t == BCJR_F32 ? 4 : 2; }
bool aligned(const void* p, int n) { return ((uintptr_t)p & (n - 1)) == 0; }
bcjr_status from_hip(int e) { return e == 0 ? BCJR_OK : BCJR_E_DEVICE; }
// a * b <= kMaxElements for a, b >= 0
bool fits(int64_t a, int64_t b) { return a == 0 || b <= kMaxElements / a; }

bool product_shapes_ok(int64_t rows, int64_t cols, const MatvecIO& io) {
  return rows >= 0 && cols >= 1 && io.tokens >= 0 && io.x_stride >= cols && io.y_stride >= rows &&
         fits(rows, cols) && rows <= kMaxElements && cols <= kMaxElements &&
         fits(io.tokens, io.x_stride) && fits(io.tokens, io.y_stride) && io.tokens <= kMaxElements;
}

bool product_pointers_ok(const MatvecIO& io) {
  const int b = dtype_size(io.dtype);
  return io.x != nullptr && io.y != nullptr && aligned(io.x, b) && aligned(io.y, b);
}

bool int4_shapes_ok(int64_t rows, int64_t cols, int64_t group) {
  return rows >= 0 && cols >= 1 && rows <= kMaxElements && cols <= kInt4Columns && fits(rows, cols) &&
         group >= 32 && group % 32 == 0 && group <= kMaxElements;
}

int by_address(const void* a, const void* b) {
  const bcjr_adamw_tensor* x = *(const bcjr_adamw_tensor* const*)a;
  const bcjr_adamw_tensor* y = *(const bcjr_adamw_tensor* const*)b;
  return x->param < y->param ? -1 : x->param > y->param ? 1 : 0;
}

// No two params share memory: sorted by address, each ends before the next begins.
bool apart(const bcjr_adamw_tensor* t, int64_t count, int size, bool* no_memory) {
  *no_memory = false;
  if (count < 2) return true;
  const bcjr_adamw_tensor** order =
      (const bcjr_adamw_tensor**)malloc((size_t)count * sizeof(bcjr_adamw_tensor*));
  if (order == nullptr) {
    *no_memory = true;
    return false;
  }
  int64_t m = 0;
  for (int64_t i = 0; i < count; ++i)
    if (t[i].numel > 0) order[m++] = &t[i];
  bool sorted = true;
  for (int64_t i = 1; i < m && sorted; ++i) sorted = order[i - 1]->param <= order[i]->param;
  if (!sorted) qsort(order, (size_t)m, sizeof(order[0]), by_address);
  bool ok = true;
  for (int64_t i = 1; i < m && ok; ++i)
    ok = (uintptr_t)order[i - 1]->param + (uintptr_t)(order[i - 1]->numel * size) <=
         (uintptr_t)order[i]->param;
  free(order);
  return ok;
}

}  // namespace

extern "C" {

bcjr_status bcjr_code_matvec(const bcjr_trellis* tr, const uint32_t* code, int64_t rows,
                             int64_t cols, int64_t L, const float* scales, const void* x,
                             int64_t tokens, int64_t x_stride, bcjr_dtype dtype, void* y,
                             int64_t y_stride, bcjr_stream_t stream) {
  if (tr == nullptr || !dtype_ok(dtype)) return BCJR_E_ARG;
  const MatvecIO io{x, y, tokens, x_stride, y_stride, dtype};
  const int n = tr->state_bits, k = tr->bits_per_step;
  if (n < 1 || n > 16 || k < 1 || k > n || !product_shapes_ok(rows, cols, io) || L < 1 || cols % L)
    return BCJR_E_SHAPE;
  if (tr->weights_per_step != 1) return BCJR_E_UNSUPPORTED;
  if (rows == 0 || tokens == 0) return BCJR_OK;
  if (!code || !tr->codebook || !product_pointers_ok(io)) return BCJR_E_ARG;
  return from_hip(launch_code_matvec(n, k, code, rows, cols, L, tr->codebook, scales, io, stream));
}

int64_t bcjr_int4_words(int64_t cols) {
  return cols < 1 || cols > kInt4Columns ? 0 : (cols + 127) / 128 * 16;
}

bcjr_status bcjr_int4_quantize(const void* w, bcjr_dtype dtype, int64_t rows, int64_t cols,
                               int64_t group, uint32_t* q, float* scales, uint8_t* zeros,
                               bcjr_stream_t stream) {
  if (!dtype_ok(dtype)) return BCJR_E_ARG;
  if (!int4_shapes_ok(rows, cols, group)) return BCJR_E_SHAPE;
  if (rows == 0) return BCJR_OK;
  if (!w || !q || !scales || !aligned(w, dtype_size(dtype)) || !aligned(q, 16)) return BCJR_E_ARG;
  return from_hip(launch_int4_quantize(w, dtype, rows, cols, group, q, scales, zeros, stream));
}

bcjr_status bcjr_int4_dequantize(const uint32_t* q, const float* scales, const uint8_t* zeros,
                                 int64_t rows, int64_t cols, int64_t group, float* w,
                                 bcjr_stream_t stream) {
  if (!int4_shapes_ok(rows, cols, group)) return BCJR_E_SHAPE;
  if (rows == 0) return BCJR_OK;
  if (!q || !scales || !w || !aligned(q, 16)) return BCJR_E_ARG;
  return from_hip(launch_int4_dequantize(q, scales, zeros, rows, cols, group, w, stream));
}

bcjr_status bcjr_int4_matvec(const uint32_t* q, const float* scales, const uint8_t* zeros,
                             int64_t rows, int64_t cols, int64_t group, const void* x,
                             int64_t tokens, int64_t x_stride, bcjr_dtype dtype, void* y,
                             int64_t y_stride, bcjr_stream_t stream) {
  if (!dtype_ok(dtype)) return BCJR_E_ARG;
  const MatvecIO io{x, y, tokens, x_stride, y_stride, dtype};
  if (!int4_shapes_ok(rows, cols, group) || !product_shapes_ok(rows, cols, io)) return BCJR_E_SHAPE;
  if (rows == 0 || tokens == 0) return BCJR_OK;
  if (!q || !scales || !aligned(q, 16) || !product_pointers_ok(io)) return BCJR_E_ARG;
  return from_hip(launch_int4_matvec(q, scales, zeros, rows, cols, group, io, stream));
}

int64_t bcjr_adamw_state_numel(const bcjr_adamw_tensor* tensors, int64_t count) {
  if (count < 1 || tensors == nullptr) return 0;
  int64_t total = 0;
  for (int64_t i = 0; i < count; ++i) {
    if (tensors[i].numel < 0 || tensors[i].numel > kMaxElements) return 0;
    total += moment_numel(tensors[i].numel);
    if (total > kMaxElements) return 0;
  }
  return total;
}

bcjr_status bcjr_adamw_step(const bcjr_adamw_tensor* tensors, int64_t count, bcjr_dtype param_type,
                            bcjr_dtype grad_type, int state_bits, const bcjr_adamw* hyper,
                            void* exp_avg, void* exp_avg_sq, uint8_t* avg_scale,
                            uint8_t* avg_sq_scale, bcjr_stream_t stream) {
  if (!dtype_ok(param_type) || !dtype_ok(grad_type) || hyper == nullptr) return BCJR_E_ARG;
  const bcjr_adamw& h = *hyper;
  // written so that a NaN fails
  if (!(h.lr >= 0 && h.eps >= 0 && h.weight_decay >= 0 && h.beta1 >= 0 && h.beta1 < 1 &&
        h.beta2 >= 0 && h.beta2 < 1) ||
      isinf(h.lr) || isinf(h.eps) || isinf(h.weight_decay) || h.step < 1)
    return BCJR_E_ARG;
  if (state_bits != 8 && state_bits != 32) return BCJR_E_UNSUPPORTED;
  if (count < 0) return BCJR_E_SHAPE;
  if (count == 0) return BCJR_OK;
  if (tensors == nullptr) return BCJR_E_ARG;
  int64_t total = 0;
  const int ps = dtype_size(param_type), gs = dtype_size(grad_type);
  for (int64_t i = 0; i < count; ++i) {
    const bcjr_adamw_tensor& t = tensors[i];
    if (t.numel < 0 || t.numel > kMaxElements) return BCJR_E_SHAPE;
    total += moment_numel(t.numel);
    if (total > kMaxElements) return BCJR_E_SHAPE;
    if (t.numel > 0 && (!t.param || !t.grad || !aligned(t.param, ps) || !aligned(t.grad, gs)))
      return BCJR_E_ARG;
  }
  if (total == 0) return BCJR_OK;
  if (!exp_avg || !exp_avg_sq || !aligned(exp_avg, 16) || !aligned(exp_avg_sq, 16)) return BCJR_E_ARG;
  if (state_bits == 8 && (!avg_scale || !avg_sq_scale)) return BCJR_E_ARG;
  bool no_memory;
  if (!apart(tensors, count, ps, &no_memory)) return no_memory ? BCJR_E_DEVICE : BCJR_E_ARG;
  const AdamwState state{exp_avg, exp_avg_sq, avg_scale, avg_sq_scale, state_bits};
  return from_hip(launch_adamw(tensors, count, param_type, grad_type, h, state, stream));
}

}  // extern "C"
