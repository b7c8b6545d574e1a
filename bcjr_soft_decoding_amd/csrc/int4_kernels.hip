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

// rint(w / s) for s > 0 as exact division gives it, by = 1 / s to an ulp: the product is at most one off,
// and the sign of w - (q +- 1/2) s, which a fused multiply-add keeps, says so; a tie goes to the even code.
__device__ inline float rint_quotient(float w, float s, float by) {
  const float q = rintf(w * by), half = fmaf(-q, s, w) < 0.0f ? -0.5f : 0.5f;
  const float over = fmaf(-(q + half), s, w) * half;  // > 0: w is nearer to the next code on its side
  const bool odd = (int)q & 1;
  return over > 0.0f || (over == 0.0f && odd) ? q + 2.0f * half : q;
}

// The same for eight weights. The product is off the exact quotient, at most 16, by less than 2^-18: only
// within 2^-17 of a border does it have to be looked at again, in one wave of a hundred.
__device__ inline void rint_quotients(const float (&w)[8], float s, float by, float (&q)[8]) {
  float nearest = 1.0f;  // to a border
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float t = w[j] * by;
    q[j] = rintf(t);
    nearest = fminf(nearest, fabsf(fabsf(t - q[j]) - 0.5f));
  }
  if (nearest < 0x1p-17f) {
#pragma unroll
    for (int j = 0; j < 8; ++j) q[j] = rint_quotient(w[j], s, by);
  }
}

// Maximum over lg lanes (a power of two): within fours, eights and rows of 16 by crossed lanes (what the halves
// hold is uniform by then, so mirroring brings the other half), beyond by shuffles.
template <class I>
__device__ inline I max_over(I v, int lg) {
  if (lg >= 2) v = max(v, (I)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xf, 0xf, true));    // quad_perm 1 0 3 2
  if (lg >= 4) v = max(v, (I)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xf, 0xf, true));    // quad_perm 2 3 0 1
  if (lg >= 8) v = max(v, (I)__builtin_amdgcn_update_dpp(0, (int)v, 0x141, 0xf, 0xf, true));   // row_half_mirror
  if (lg >= 16) v = max(v, (I)__builtin_amdgcn_update_dpp(0, (int)v, 0x140, 0xf, 0xf, true));  // row_mirror
  if (lg >= 32) v = max(v, (I)__shfl_xor((int)v, 16, 64));
  if (lg >= 64) v = max(v, (I)__shfl_xor((int)v, 32, 64));
  return v;
}

// Eight columns of a row, zeros from end on.
template <class E>
__device__ inline void load_w8(const typename E::T* row, long long c, long long end, float out[8]) {
  using X = typename E::T;
  if (c + 8 <= end) {
#pragma unroll
    for (int h = 0; h < 8; h += 4) {
      const auto v = *reinterpret_cast<const typename Loose<X, 4>::V*>(row + c + h);
#pragma unroll
      for (int i = 0; i < 4; ++i) out[h + i] = (float)v[i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) out[i] = c + i < end ? E::load(row + c + i) : 0.0f;
  }
}

// LG lanes for a group, a lane for 8 columns: loaded once where the group has no more (ONCE), else
// once for the range and once for the codes. Bound by memory: 2048 x 8192 fp32 weights are read and
// their codes written in 21 us, at 3.5 TB/s; a small matrix by its loads' and reductions' latency (1000 x 4100 bf16 9 us).
template <class E, bool ONCE, bool ZEROS>
__global__ void __launch_bounds__(256)
k_int4_quantize(const typename E::T* __restrict__ w, long long rows, int cols, int group, int groups, int words, int lg,
                long long dr, int dg, unsigned* __restrict__ q, float* __restrict__ scales, uint8_t* __restrict__ zeros) {
  const int sub = threadIdx.x & (lg - 1), sh = 31 - __clz(lg), per = 256 >> sh;
  const long long total = rows * groups, stride = (long long)gridDim.x * per;
  // the blocks' first groups are few: 32 bits divide them
  const unsigned first = blockIdx.x * per + (threadIdx.x >> sh);
  long long i = first;
  // a group's row and place in it, carried along without another division: a round is dr rows and dg groups on
  long long r = first / (unsigned)groups;
  int g = (int)(first - (unsigned)r * groups);
  for (; i - (threadIdx.x >> sh) < total; i += stride) {
    const bool live = i < total;
    const int c0 = g * group, end = min(c0 + group, cols);
    const typename E::T* __restrict__ row = w + (live ? r : 0) * cols;
    // The range as bits. Those of a positive number order like it as signed integers, those of a negative one
    // against it as unsigned ones, and NaN and Inf lie beyond all others.
    int top = 0;                       // of the positive ones, or (no zero points) of all magnitudes
    unsigned bottom = 0x80000000u;     // of the negative ones
    float v[8];
    if (live)
      for (int c = c0 + 8 * sub; c < end; c += 8 * lg) {
        load_w8<E>(row, c, end, v);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int bits = __float_as_int(v[j]);
          top = max(top, ZEROS ? bits : bits & 0x7fffffff);
          if (ZEROS) bottom = max(bottom, (unsigned)bits);
        }
        if (ONCE) break;
      }
    top = max_over(top, lg);
    if (ZEROS) bottom = max_over(bottom, lg);
    const bool bad = top >= 0x7f800000 || (ZEROS && bottom >= 0xff800000u);
    const float hi = __int_as_float(top), lo = __uint_as_float(bottom);
    // rounded once: hi - lo may need more than fp32 holds
    const float s = ZEROS ? (float)(((double)hi - (double)lo) / 15.0) : hi / 7.0f;
    // a scale whose reciprocal would overflow is brought up with its weights, by a power of two
    const bool tiny = s < 0x1p-120f;
    const float lift = tiny ? 0x1p+64f : 1.0f, sl = s * lift, by = __builtin_amdgcn_rcpf(sl);
    if (ONCE && tiny)
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] *= lift;
    const bool codes = !bad && s > 0.0f;
    float z = 8.0f;
    if (ZEROS) z = codes ? fminf(rint_quotient(-lo * lift, sl, by), 15.0f) : 0.0f;
    if (live) {
      if (sub == 0) {
        scales[i] = bad ? NAN : s;
        if (ZEROS) zeros[i] = (uint8_t)z;
      }
      // the last group of a row also writes the zero nibbles behind it
      const int stop = g == groups - 1 ? 8 * words : c0 + group;
      for (int c = c0 + 8 * sub; c < stop; c += 8 * lg) {
        if (!ONCE && c < end) {
          load_w8<E>(row, c, end, v);
#pragma unroll
          for (int j = 0; j < 8; ++j) v[j] *= lift;
        }
        float n[8] = {};
        if (codes) rint_quotients(v, sl, by, n);
        unsigned word = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j)
          word |= (unsigned)__builtin_amdgcn_fmed3f(n[j] + z, 0.0f, 15.0f) << nibble_shift(j);
        if (c + 8 > end) {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (c + j >= end) word &= ~(15u << nibble_shift(j));
        }
        q[r * words + word_of(c / 8)] = word;
      }
    }
    r += dr;
    g += dg;
    if (g >= groups) {
      g -= groups;
      ++r;
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

}  // namespace

int launch_int4_quantize(const void* w, int dtype, int64_t rows, int64_t cols, int64_t group,
                         uint32_t* q, float* scales, uint8_t* zeros, void* stream) {
  const int64_t groups = (cols + group - 1) / group, span = group < cols ? group : cols;
  int lg = 1;
  while (lg < 64 && 8 * lg < span) lg *= 2;
  const int64_t per = 256 / lg, blocks = (rows * groups + per - 1) / per;
  // a few rounds a block, so that its one division is shared: at most 16 blocks for each of 256 CUs
  const int64_t most = blocks < 4096 ? blocks : 4096, stride = most * per;
  // a group longer than its row is its row
  const int length = (int)(group < cols ? group : (cols + 31) / 32 * 32);
  return with_type(dtype, [&](auto e) {
    using E = decltype(e);
    auto launch = [&](auto kernel) {
      hipLaunchKernelGGL(kernel, dim3((unsigned)most), dim3(256), 0, static_cast<hipStream_t>(stream),
                         static_cast<const typename E::T*>(w), (long long)rows, (int)cols, length, (int)groups,
                         (int)bcjr_int4_words(cols), lg, (long long)(stride / groups), (int)(stride % groups), q, scales,
                         zeros);
      return (int)hipGetLastError();
    };
    if (8 * lg >= span) return zeros ? launch(k_int4_quantize<E, true, true>) : launch(k_int4_quantize<E, true, false>);
    return zeros ? launch(k_int4_quantize<E, false, true>) : launch(k_int4_quantize<E, false, false>);
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

template <class E, int F, int RT, int NT, int GS, bool ZEROS>
int launch_tiles(Int4Args a, hipStream_t stream) {
  constexpr int kRowsOfWave = RT * 16 / F;
  const int steps = ((a.tile.cols + 127) / 128 + F - 1) / F;
  const int64_t units = (a.tile.rows + kRowsOfWave - 1) / kRowsOfWave;
  const int kw = waves_along(steps, units), waves = kw < 4 ? 4 : kw;
  a.tile.kw = kw;
  const int64_t rw = waves / kw, blocks = (units + rw - 1) / rw;
  const int64_t tokens = (a.tile.tokens + NT * tile_tokens<E, F>() - 1) / (NT * tile_tokens<E, F>());
  const size_t lds = (size_t)waves * NT * kXBytes;
  hipLaunchKernelGGL((k_int4_tiles<E, F, RT, NT, GS, ZEROS>), dim3(grid_of(blocks), (unsigned)tokens), dim3(64 * waves), lds,
                     stream, a);
  return (int)hipGetLastError();
}

template <class E, int F, int RT, int NT, int GS>
int launch_tiles_zeros(const Int4Args& a, hipStream_t stream) {
  return a.zeros ? launch_tiles<E, F, RT, NT, GS, true>(a, stream) : launch_tiles<E, F, RT, NT, GS, false>(a, stream);
}

template <class E, int F, int RT, int NT>
int launch_tiles_group(const Int4Args& a, int64_t units, hipStream_t stream) {
  return units % 4 == 0   ? launch_tiles_zeros<E, F, RT, NT, 4>(a, stream)
         : units % 2 == 0 ? launch_tiles_zeros<E, F, RT, NT, 2>(a, stream)
                          : launch_tiles_zeros<E, F, RT, NT, 1>(a, stream);
}

// Waves that four row tiles a wave leave.
template <int F>
int64_t waves_of_four(const Int4Args& a) {
  const int64_t steps = ((a.tile.cols + 127) / 128 + F - 1) / F;
  return a.tile.rows * F / 64 * (steps < kMaxWaves ? steps : kMaxWaves);
}

// Four row tiles a wave, which share the loads of x, where that leaves waves enough: 16384 x 16384 with one token
// takes 34 us against 47 with one tile, 2048 x 8192 5.1 against 7.3; 512 x 1024 3.9 against 3.3.
template <class E, int F>
int launch_tiles_rows(const Int4Args& a, int64_t per_group, hipStream_t stream) {
  return waves_of_four<F>(a) >= 1024 ? launch_tiles_group<E, F, 4, 1>(a, per_group, stream)
                                     : launch_tiles_group<E, F, 1, 1>(a, per_group, stream);
}

// The largest fold that the tokens leave room for and the columns fill; for more tokens than a tile holds two
// tiles of them, for which the codes are read and unpacked once, where that leaves waves enough (32 tokens: 16384 x 16384
// 55 us against 70 one by one, 8192 x 8192 27 against 20).
template <class E>
int launch_tiles_any(const Int4Args& a, int64_t per_group, hipStream_t stream) {
  const int blocks = (a.tile.cols + 127) / 128;
  if constexpr (TileOf<E>::T::kParts == 1) {
    if (a.tile.tokens == 1 && blocks > 8) return launch_tiles_rows<E, 16>(a, per_group, stream);
    if (a.tile.tokens <= 2 && blocks > 4) return launch_tiles_rows<E, 8>(a, per_group, stream);
  }
  if (a.tile.tokens <= tile_tokens<E, 4>() && blocks > 2) return launch_tiles_rows<E, 4>(a, per_group, stream);
  if (a.tile.tokens <= tile_tokens<E, 2>() && blocks > 1) return launch_tiles_rows<E, 2>(a, per_group, stream);
  if (a.tile.tokens > tile_tokens<E, 1>() && waves_of_four<1>(a) >= 2048) return launch_tiles_group<E, 1, 4, 2>(a, per_group, stream);
  return launch_tiles_rows<E, 1>(a, per_group, stream);
}

}  // namespace

int launch_int4_matvec(const uint32_t* q, const float* scales, const uint8_t* zeros, int64_t rows,
                       int64_t cols, int64_t group, const MatvecIO& io, void* stream) {
  Int4Args a;
  a.q = q;
  a.scales = scales;
  a.zeros = zeros;
  a.groups = (int)((cols + group - 1) / group);
  a.words = (int)bcjr_int4_words(cols);
  a.per_group = 1.0f / (float)(group / 32);
  return in_pieces(io, io.dtype == BCJR_F32 ? 4 : 2, [&](const MatvecIO& piece) {
    a.tile = tile_args(piece, rows, cols);
    return with_type(io.dtype, [&](auto e) {
      return launch_tiles_any<decltype(e)>(a, group / 32, static_cast<hipStream_t>(stream));
    });
  });
}

}  // namespace bcjr
