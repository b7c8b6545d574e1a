// 4-bit weights with a scale (and optionally a zero point) for each group of columns: rounding to
// them, the values they stand for, and the products of a few tokens with them. The layout of the
// codes is in include/bcjr.h.
#include <hip/hip_runtime.h>

#include "int4_mfma.h"
#include "internal.h"
#include "ops.h"
#include "ops_device.h"

namespace bcjr {
namespace {

// The word of a row that holds columns 8 u .. 8 u + 7.
__device__ inline long long word_of(long long u) {
  return (u & ~15ll) + 4 * (u & 3) + ((u >> 2) & 3);
}
// The low bit of column c (0 .. 7) of a word.
__device__ inline int nibble_shift(int c) { return 4 * ((c >> 1) + 4 * (c & 1)); }

// rint(w / s) for s > 0 as exact division gives it: the rounded quotient is at most one off, and the
// sign of w - (q +- 1/2) s, which a fused multiply-add keeps, says so; a tie goes to the even code.
__device__ inline float rint_quotient(float w, float s) {
  float q = rintf(w / s);
  const float up = fmaf(-(q + 0.5f), s, w), down = fmaf(-(q - 0.5f), s, w);
  const bool odd = ((int)q) & 1;
  if (up > 0.0f || (up == 0.0f && odd)) q += 1.0f;
  if (down < 0.0f || (down == 0.0f && odd)) q -= 1.0f;
  return q;
}

// LG lanes for a group, a lane for 8 columns at a time: a pass for the range, a pass for the codes
// (the second read of a group is served by the caches).
template <class E>
__global__ void __launch_bounds__(256)
k_int4_quantize(const typename E::T* __restrict__ w, long long rows, long long cols, long long group,
                long long groups, long long words, int lg, unsigned* __restrict__ q,
                float* __restrict__ scales, uint8_t* __restrict__ zeros) {
  const int sub = threadIdx.x % lg;
  const long long per = 256 / lg, total = rows * groups;
  for (long long i0 = (long long)blockIdx.x * per; i0 < total; i0 += (long long)gridDim.x * per) {
    const long long i = i0 + threadIdx.x / lg;
    const bool live = i < total;
    const long long r = live ? i / groups : 0, g = live ? i - r * groups : 0;
    const long long c0 = g * group, end = c0 + group < cols ? c0 + group : cols;
    const typename E::T* __restrict__ row = w + r * cols;
    float hi = 0.0f, lo = 0.0f;
    bool odd = false;  // a NaN or Inf
    if (live)
      for (long long c = c0 + 8 * sub; c < end; c += 8 * lg)
        for (int j = 0; j < 8; ++j)
          if (c + j < end) {
            const float v = E::load(row + c + j);
            odd |= !(fabsf(v) < INFINITY);
            hi = fmaxf(hi, v);
            lo = fminf(lo, v);
          }
    int bad = odd;
    for (int d = 1; d < lg; d <<= 1) {
      hi = fmaxf(hi, __shfl_xor(hi, d, 64));
      lo = fminf(lo, __shfl_xor(lo, d, 64));
      bad |= __shfl_xor(bad, d, 64);
    }
    float s = zeros != nullptr ? (float)(((double)hi - (double)lo) / 15.0) : fmaxf(hi, -lo) / 7.0f;
    float z = 8.0f;
    if (zeros != nullptr) z = !bad && s > 0.0f ? fminf(rint_quotient(-lo, s), 15.0f) : 0.0f;
    if (bad) s = NAN;
    if (!live) continue;
    if (sub == 0) {
      scales[i] = s;
      if (zeros != nullptr) zeros[i] = (uint8_t)z;
    }
    // the last group of a row also writes the zero nibbles behind it
    const long long stop = g == groups - 1 ? 8 * words : c0 + group;
    for (long long c = c0 + 8 * sub; c < stop; c += 8 * lg) {
      unsigned word = 0;
      for (int j = 0; j < 8; ++j)
        if (c + j < end) {
          float code = z;
          if (!bad && s > 0.0f) code += rint_quotient(E::load(row + c + j), s);
          code = fminf(fmaxf(code, 0.0f), 15.0f);
          word |= (unsigned)code << nibble_shift(j);
        }
      q[r * words + word_of(c / 8)] = word;
    }
  }
}

__global__ void __launch_bounds__(256)
k_int4_dequantize(const unsigned* __restrict__ q, const float* __restrict__ scales,
                  const uint8_t* __restrict__ zeros, long long rows, long long cols, long long group,
                  long long groups, long long words, float* __restrict__ w) {
  const long long units = (cols + 7) / 8, total = rows * units;
  for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < total; i += (long long)gridDim.x * 256) {
    const long long r = i / units, u = i - r * units, g = r * groups + 8 * u / group;
    const unsigned word = q[r * words + word_of(u)];
    const float s = scales[g], z = zeros != nullptr ? (float)zeros[g] : 8.0f;
    for (int j = 0; j < 8; ++j)
      if (8 * u + j < cols) w[r * cols + 8 * u + j] = ((float)((word >> nibble_shift(j)) & 15u) - z) * s;
  }
}

// Any shape: one wave for a row and TB tokens, a lane for 8 columns.
template <class E, int TB>
__global__ void __launch_bounds__(256)
k_int4_matvec(const unsigned* __restrict__ q, const float* __restrict__ scales,
              const uint8_t* __restrict__ zeros, long long rows, long long cols, long long group,
              long long groups, long long words, const typename E::T* __restrict__ x,
              long long tokens, long long xs, typename E::T* __restrict__ y, long long ys) {
  const int lane = threadIdx.x & 63;
  const long long waves = (long long)gridDim.x * 4;
  for (long long m0 = (long long)blockIdx.y * TB; m0 < tokens; m0 += (long long)gridDim.y * TB) {
    for (long long r = (long long)blockIdx.x * 4 + (threadIdx.x >> 6); r < rows; r += waves) {
      float acc[TB] = {};
      for (long long c = 8 * lane; c < cols; c += 512) {
        const unsigned word = q[r * words + word_of(c / 8)];
        const long long g = r * groups + c / group;
        const float s = scales[g], z = zeros != nullptr ? (float)zeros[g] : 8.0f;
        for (int j = 0; j < 8; ++j) {
          if (c + j >= cols) break;
          const float v = ((float)((word >> nibble_shift(j)) & 15u) - z) * s;
#pragma unroll
          for (int i = 0; i < TB; ++i)
            if (m0 + i < tokens) acc[i] = fmaf(v, E::load(x + (m0 + i) * xs + c + j), acc[i]);
        }
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

int launch_int4_quantize(const void* w, int dtype, int64_t rows, int64_t cols, int64_t group,
                         uint32_t* q, float* scales, uint8_t* zeros, void* stream) {
  const int64_t groups = (cols + group - 1) / group;
  int lg = 1;
  while (lg < 64 && 8 * lg < group && 8 * lg < cols) lg *= 2;
  return with_type(dtype, [&](auto e) {
    using E = decltype(e);
    const int64_t per = 256 / lg;
    hipLaunchKernelGGL((k_int4_quantize<E>), dim3(grid_of((rows * groups + per - 1) / per)), dim3(256), 0,
                       static_cast<hipStream_t>(stream), static_cast<const typename E::T*>(w),
                       (long long)rows, (long long)cols, (long long)group, (long long)groups,
                       (long long)bcjr_int4_words(cols), lg, q, scales, zeros);
    return (int)hipGetLastError();
  });
}

int launch_int4_dequantize(const uint32_t* q, const float* scales, const uint8_t* zeros,
                           int64_t rows, int64_t cols, int64_t group, float* w, void* stream) {
  const int64_t groups = (cols + group - 1) / group, units = (cols + 7) / 8;
  hipLaunchKernelGGL(k_int4_dequantize, dim3(grid_of((rows * units + 255) / 256)), dim3(256), 0,
                     static_cast<hipStream_t>(stream), q, scales, zeros, (long long)rows,
                     (long long)cols, (long long)group, (long long)groups,
                     (long long)bcjr_int4_words(cols), w);
  return (int)hipGetLastError();
}

namespace {

template <class E, int F, int RT, int NT, int GS>
int launch_tiles(Int4Args a, hipStream_t stream) {
  constexpr int kRowsOfWave = RT * 16 / F;
  const int steps = ((a.tile.cols + 127) / 128 + F - 1) / F;
  const int64_t units = (a.tile.rows + kRowsOfWave - 1) / kRowsOfWave;
  const int kw = waves_along(steps, units), waves = kw < 4 ? 4 : kw;
  a.tile.kw = kw;
  const int64_t rw = waves / kw, blocks = (units + rw - 1) / rw;
  const int64_t tokens = (a.tile.tokens + NT * tile_tokens<E, F>() - 1) / (NT * tile_tokens<E, F>());
  const size_t lds = (size_t)waves * RT * (16 / F) * NT * (16 / F) * sizeof(float);
  hipLaunchKernelGGL((k_int4_tiles<E, F, RT, NT, GS>), dim3(grid_of(blocks), (unsigned)tokens), dim3(64 * waves), lds,
                     stream, a);
  return (int)hipGetLastError();
}

template <class E, int F, int RT, int NT>
int launch_tiles_group(const Int4Args& a, hipStream_t stream) {
  return a.per_group % 4 == 0   ? launch_tiles<E, F, RT, NT, 4>(a, stream)
         : a.per_group % 2 == 0 ? launch_tiles<E, F, RT, NT, 2>(a, stream)
                                : launch_tiles<E, F, RT, NT, 1>(a, stream);
}

// The largest fold that the tokens leave room for and the columns fill.
template <class E>
int launch_tiles_any(const Int4Args& a, hipStream_t stream) {
  const int blocks = (a.tile.cols + 127) / 128;
  if constexpr (TileOf<E>::T::kParts == 1) {
    if (a.tile.tokens == 1 && blocks > 8) return launch_tiles_group<E, 16, 4, 1>(a, stream);
    if (a.tile.tokens <= 2 && blocks > 4) return launch_tiles_group<E, 8, 4, 1>(a, stream);
  }
  if (a.tile.tokens <= tile_tokens<E, 4>() && blocks > 2) return launch_tiles_group<E, 4, 2, 1>(a, stream);
  if (a.tile.tokens <= tile_tokens<E, 2>() && blocks > 1) return launch_tiles_group<E, 2, 2, 1>(a, stream);
  if (a.tile.tokens <= tile_tokens<E, 1>()) return launch_tiles_group<E, 1, 1, 1>(a, stream);
  return launch_tiles_group<E, 1, 2, 2>(a, stream);
}

}  // namespace

int launch_int4_matvec(const uint32_t* q, const float* scales, const uint8_t* zeros, int64_t rows,
                       int64_t cols, int64_t group, const MatvecIO& io, void* stream) {
  const int64_t groups = (cols + group - 1) / group;
  // The matrix-core form holds columns in 32 bits and divides a column by the group's length with one
  // high product, exact while (cols / 32 + 4 * 16) * group / 32 < 2^32 (a step may reach 16 blocks over).
  const int64_t per_group = group / 32, units = (cols + 31) / 32 + 64;
  if (cols <= ((int64_t)1 << 24) && per_group <= ((int64_t)1 << 30) / units && io.tokens <= 65535) {
    Int4Args a;
    a.q = q;
    a.scales = scales;
    a.zeros = zeros;
    a.tile = tile_args(io, rows, cols);
    a.groups = (int)groups;
    a.words = (int)bcjr_int4_words(cols);
    a.per_group = (unsigned)per_group;
    a.magic = (unsigned)((((int64_t)1 << 32) + per_group - 1) / per_group);
    return with_type(io.dtype, [&](auto e) {
      return launch_tiles_any<decltype(e)>(a, static_cast<hipStream_t>(stream));
    });
  }
  return with_type(io.dtype, [&](auto e) {
    using E = decltype(e);
    const int64_t blocks = (io.tokens + 3) / 4;
    const dim3 grid(grid_of((rows + 3) / 4), (unsigned)(blocks < 32768 ? blocks : 32768));
    hipLaunchKernelGGL((k_int4_matvec<E, 4>), grid, dim3(256), 0, static_cast<hipStream_t>(stream), q,
                       scales, zeros, (long long)rows, (long long)cols, (long long)group,
                       (long long)groups, (long long)bcjr_int4_words(cols),
                       static_cast<const typename E::T*>(io.x), (long long)io.tokens,
                       (long long)io.x_stride, static_cast<typename E::T*>(io.y),
                       (long long)io.y_stride);
    return (int)hipGetLastError();
  });
}

}  // namespace bcjr
