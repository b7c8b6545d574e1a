// Products of a few tokens with trellis-coded weights (the packed hard code of the bitshift trellis).
// Every state is the n-bit window of its chain's code at bit k t, so a weight is two shifts and one
// table read away from the code and no chain is walked: y[m, r] = sum_q scales[r, q] sum_t
// c(s_t) x[m, q L + t].
#include <hip/hip_runtime.h>

#include "internal.h"
#include "ops.h"
#include "ops_device.h"
#include "tiles.h"

namespace bcjr {
namespace {

// Any shape: one wave for a row and TB tokens, a lane for a column. For what the tiles do not take; bound by its 64-bit
// addresses and one table read a weight (2048 x 8192 with k = 8 and one token 103 us).
template <class E, int TB>
__global__ void __launch_bounds__(256)
k_code_matvec(const unsigned* __restrict__ code, long long rows, long long cols, long long L, int n,
              int k, long long W, const float* __restrict__ cb, const float* __restrict__ scales,
              const typename E::T* __restrict__ x, long long tokens, long long xs,
              typename E::T* __restrict__ y, long long ys) {
  const int lane = threadIdx.x & 63;
  const long long waves = (long long)gridDim.x * 4;
  const unsigned mask = (1u << n) - 1u;
  for (long long m0 = (long long)blockIdx.y * TB; m0 < tokens; m0 += (long long)gridDim.y * TB) {
    for (long long r = (long long)blockIdx.x * 4 + (threadIdx.x >> 6); r < rows; r += waves) {
      float acc[TB] = {};
      const long long q0 = r * (cols / L);
      for (long long c = lane; c < cols; c += 64) {
        const long long q = q0 + c / L, p = k * (c % L);
        const unsigned* __restrict__ cw = code + q * W + (p >> 5);
        const int off = (int)(p & 31);
        const unsigned long long lo = off + n > 32 ? cw[1] : 0u;
        const unsigned s = (unsigned)((((unsigned long long)cw[0] << 32) | lo) >> (64 - off - n)) & mask;
        const float w = scales != nullptr ? scales[q] * cb[s] : cb[s];
#pragma unroll
        for (int i = 0; i < TB; ++i)
          if (m0 + i < tokens) acc[i] = fmaf(w, E::load(x + (m0 + i) * xs + c), acc[i]);
      }
#pragma unroll
      for (int i = 0; i < TB; ++i) {
        const float s = wave_sum(acc[i]);
        if (lane == 0 && m0 + i < tokens) E::store(y + (m0 + i) * ys + r, s);
      }
    }
  }
}

}  // namespace

int launch_code_matvec(int n, int k, const uint32_t* code, int64_t rows, int64_t cols, int64_t L,
                       const float* codebook, const float* scales, const MatvecIO& io, void* stream) {
  // On the matrix cores. Whole blocks of 128 columns in a chain and a table of at most 128 KiB, which leaves 8 waves
  // the LDS they need (a codeword takes 4 bytes, 8 for fp32), are decoded faster than other chains of at least 8.
  const int64_t words = code_words(n, k, L);
  const bool blocks = L % 128 == 0 && n <= (io.dtype == BCJR_F32 ? 14 : 15) && cols <= kTileColumns;
  if (k <= 4 && (blocks || (L >= 8 && cols <= ((int64_t)1 << 20)))) {
    CodeArgs a;
    a.code = code;
    a.codebook = codebook;
    a.scales = scales;
    a.n = n;
    a.k = k;
    a.chains = (int)(cols / L);
    a.words = (int)words;
    a.per_chain = blocks ? (int)(L / 128) : 0;
    a.L = blocks ? 0 : (int)L;
    a.reciprocal = 1.0f / (float)(blocks ? a.per_chain : a.L);
    return in_pieces(io, io.dtype == BCJR_F32 ? 4 : 2, [&](const MatvecIO& piece) {
      a.tile = tile_args(piece, rows, cols);
      return io.dtype == BCJR_F32   ? launch_code_tiles_f32(a, k, stream)
             : io.dtype == BCJR_F16 ? launch_code_tiles_f16(a, k, stream)
                                    : launch_code_tiles_bf16(a, k, stream);
    });
  }
  return with_type(io.dtype, [&](auto e) {
    using E = decltype(e);
    const int64_t blocks = (io.tokens + 3) / 4;
    const dim3 grid(grid_of((rows + 3) / 4), (unsigned)(blocks < 32768 ? blocks : 32768));
    hipLaunchKernelGGL((k_code_matvec<E, 4>), grid, dim3(256), 0, static_cast<hipStream_t>(stream),
                       code, (long long)rows, (long long)cols, (long long)L, n, k,
                       (long long)words, codebook, scales,
                       static_cast<const typename E::T*>(io.x), (long long)io.tokens,
                       (long long)io.x_stride, static_cast<typename E::T*>(io.y),
                       (long long)io.y_stride);
    return (int)hipGetLastError();
  });
}

}  // namespace bcjr
