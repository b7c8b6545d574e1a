// Products of a few tokens with trellis-coded weights (the packed hard code of the bitshift trellis).
// Every state is the n-bit window of its chain's code at bit k t, so a weight is two shifts and one
// table read away from the code and no chain is walked: y[m, r] = sum_q scales[r, q] sum_t
// c(s_t) x[m, q L + t].
#include <hip/hip_runtime.h>

#include "code_mfma.h"
#include "internal.h"
#include "ops.h"
#include "ops_device.h"

namespace bcjr {
namespace {

// Any shape: one wave for a row and TB tokens, a lane for a column.
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

template <class E, int F, int RT, int NT, int K>
int launch_tiles(CodeArgs a, hipStream_t stream) {
  constexpr int kRowsOfWave = RT * 16 / F;
  const int steps = (a.tile.cols / 128 + F - 1) / F;
  const int64_t units = (a.tile.rows + kRowsOfWave - 1) / kRowsOfWave;
  // Every block makes a table: 8 waves share it, or as many as LDS leaves room for beside it (4 at 2^15
  // states), and no more blocks than fit the chip are started.
  auto lds_of = [&](int waves) { return ((size_t)1 << a.n) * sizeof(float) + (size_t)waves * NT * kXBytes; };
  int waves = kMaxWaves;
  while (lds_of(waves) > kLds) waves /= 2;
  const size_t lds = lds_of(waves);
  const int along = waves_along(steps, units), kw = along < waves ? along : waves;
  a.tile.kw = kw;
  const int64_t rw = waves / kw, blocks = (units + rw - 1) / rw;
  const int64_t tokens = (a.tile.tokens + NT * tile_tokens<E, F>() - 1) / (NT * tile_tokens<E, F>());
  const void* kernel = reinterpret_cast<const void*>(k_code_tiles<E, F, RT, NT, K>);
  if (lds > 65536) {
    const hipError_t e = hipFuncSetAttribute(kernel, hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
    if (e != hipSuccess) return (int)e;
  }
  const int64_t room = 256 * (lds > kLds / 2 ? 1 : 2);
  hipLaunchKernelGGL((k_code_tiles<E, F, RT, NT, K>), dim3((unsigned)(blocks < room ? blocks : room), (unsigned)tokens),
                     dim3(64 * waves), lds, stream, a);
  return (int)hipGetLastError();
}

template <class E, int F, int RT, int NT>
int launch_tiles_bits(const CodeArgs& a, int k, hipStream_t stream) {
  return k == 1   ? launch_tiles<E, F, RT, NT, 1>(a, stream)
         : k == 2 ? launch_tiles<E, F, RT, NT, 2>(a, stream)
         : k == 3 ? launch_tiles<E, F, RT, NT, 3>(a, stream)
                  : launch_tiles<E, F, RT, NT, 4>(a, stream);
}

// The largest fold that the tokens leave room for and the columns fill.
template <class E>
int launch_tiles_any(const CodeArgs& a, int k, hipStream_t stream) {
  const int blocks = a.tile.cols / 128;
  if constexpr (TileOf<E>::T::kParts == 1) {
    if (a.tile.tokens == 1 && blocks > 8) return launch_tiles_bits<E, 16, 2, 1>(a, k, stream);
    if (a.tile.tokens <= 2 && blocks > 4) return launch_tiles_bits<E, 8, 2, 1>(a, k, stream);
  }
  if (a.tile.tokens <= tile_tokens<E, 4>() && blocks > 2) return launch_tiles_bits<E, 4, 2, 1>(a, k, stream);
  if (a.tile.tokens <= tile_tokens<E, 2>() && blocks > 1) return launch_tiles_bits<E, 2, 1, 1>(a, k, stream);
  // beside 2^15 codewords there is no room for the x of two tiles of tokens
  if (a.tile.tokens <= tile_tokens<E, 1>() || a.n == 15) return launch_tiles_bits<E, 1, 1, 1>(a, k, stream);
  return launch_tiles_bits<E, 1, 1, 2>(a, k, stream);
}

}  // namespace

int launch_code_matvec(int n, int k, const uint32_t* code, int64_t rows, int64_t cols, int64_t L,
                       const float* codebook, const float* scales, const MatvecIO& io, void* stream) {
  // The matrix-core form: whole blocks of 128 columns in a chain and a table that fits LDS.
  const int64_t words = code_words(n, k, L);
  if (L % 128 == 0 && n <= 15 && k <= 4 && cols <= kTileColumns) {
    CodeArgs a;
    a.code = code;
    a.codebook = codebook;
    a.scales = scales;
    a.n = n;
    a.chains = (int)(cols / L);
    a.words = (int)words;
    a.per_chain = (int)(L / 128);
    a.reciprocal = 1.0f / (float)a.per_chain;
    return in_pieces(io, io.dtype == BCJR_F32 ? 4 : 2, [&](const MatvecIO& piece) {
      a.tile = tile_args(piece, rows, cols);
      return with_type(io.dtype, [&](auto e) {
        return launch_tiles_any<decltype(e)>(a, k, static_cast<hipStream_t>(stream));
      });
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
