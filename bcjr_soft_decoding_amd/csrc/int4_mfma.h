// Products of a few tokens with 4-bit weights on the matrix cores (the tile: tiles.h).
//
// Codes become numbers without a subtraction: a nibble goes to the top four mantissa bits of a half or a
// bfloat16 with exponent 0 and is 1 + q / 16, exactly. With D = sum (1 + q / 16) x and S = sum x (the
// same instruction with weights of one, once for all rows of a wave), a group gives
// scale (16 D - (16 + z) S), in fp32: nothing is rounded before the last conversion.
#pragma once
#include "tiles.h"

namespace bcjr {

struct Int4Args {
  TileArgs tile;
  const unsigned* q;
  const float* scales;
  const uint8_t* zeros;
  int groups, words;
  float per_group;  // 1 / (units of 32 columns in a group)
};

namespace {

// The eight weights of a word as numbers 1 + q / 16.
template <class T>
__device__ inline typename T::V weights8(unsigned w) {
  u32x4 v;
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    const int up = T::kUp - 4 * p;
    v[p] = ((up >= 0 ? w << up : w >> -up) & T::kMask) | T::kOne;
  }
  return __builtin_bit_cast(typename T::V, v);
}

// F folds, RT tiles of rows and NT tiles of tokens a wave, GS products of 32 columns a scale.
template <class E, int F, int RT, int NT, int GS>
__global__ void __launch_bounds__(64 * kMaxWaves)
k_int4_tiles(const Int4Args a) {
  using T = typename TileOf<E>::T;
  using V = typename T::V;
  using Pl = Place<E, F>;
  constexpr int kRows = Pl::kRows, kKept = Pl::kKept;
  extern __shared__ float part_sums[];
  const Pl pl;
  const int kw = a.tile.kw, ki = pl.wave % kw, ri = pl.wave / kw, rw = pl.waves / kw;
  const int blocks = (a.tile.cols + 127) / 128, steps = (blocks + F - 1) / F;
  const long long rows = a.tile.rows, units = (rows + RT * kRows - 1) / (RT * kRows);  // of rows, one for a wave
  const long long m0 = (long long)blockIdx.y * (NT * Pl::kTokens);
  const typename E::T* xr[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) xr[n] = pl.x_row(a.tile, m0, n);
  const V ones = __builtin_bit_cast(V, u32x4{T::kOne, T::kOne, T::kOne, T::kOne});
  const V none = __builtin_bit_cast(V, u32x4{0, 0, 0, 0});

  for (long long ub = (long long)blockIdx.x * rw; ub < units; ub += (long long)gridDim.x * rw) {
    const long long row0 = (ub + ri) * (RT * kRows);
    // offsets from the wave's first row fit 32 bits; rows behind the last repeat it
    const long long base = row0 < rows ? row0 : rows - 1;
    const int last = (int)(rows - 1 - base < RT * kRows ? rows - 1 - base : RT * kRows);
    const unsigned* __restrict__ q = a.q + base * a.words;
    const float* __restrict__ scales = a.scales + base * a.groups;
    const uint8_t* __restrict__ zeros = a.zeros + base * a.groups;
    unsigned qo[RT], so[RT][kKept];
    float acc[RT][NT][kKept] = {};
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      qo[t] = (unsigned)(min(t * kRows + pl.weight_row(), last) * a.words + 4 * pl.g);
#pragma unroll
      for (int u = 0; u < kKept; ++u) so[t][u] = (unsigned)(min(t * kRows + pl.sum_row(u), last) * a.groups);
    }
    for (int s = ki; s < steps; s += kw) {
      const int block = s * F + pl.fold;
      const bool in = block < blocks;
      u32x4 w[RT];
#pragma unroll
      for (int t = 0; t < RT; ++t) w[t] = in ? *reinterpret_cast<const u32x4*>(q + (qo[t] + block * 16)) : u32x4{0, 0, 0, 0};
      V x[NT][4];
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          x[n][j] = none;
          if (in) x[n][j] = load_x8<E>(xr[n], block * 128 + 32 * j + 8 * pl.g, a.tile.cols, pl.x_part());
        }
#pragma unroll
      for (int j0 = 0; j0 < 4; j0 += GS) {
        const int group = min(divide(block * 4 + j0, a.per_group), a.groups - 1);
        f32x4 sum[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          sum[n] = f32x4{0, 0, 0, 0};
#pragma unroll
          for (int j = j0; j < j0 + GS; ++j) sum[n] = T::mfma(ones, x[n][j], sum[n]);
        }
#pragma unroll
        for (int t = 0; t < RT; ++t) {
          f32x4 d[NT];
#pragma unroll
          for (int n = 0; n < NT; ++n) d[n] = f32x4{0, 0, 0, 0};
#pragma unroll
          for (int j = j0; j < j0 + GS; ++j) {
            const V wj = weights8<T>(w[t][j]);
#pragma unroll
            for (int n = 0; n < NT; ++n) d[n] = T::mfma(wj, x[n][j], d[n]);
          }
#pragma unroll
          for (int u = 0; u < kKept; ++u) {
            const float sc = 16.0f * scales[so[t][u] + group];
            const float z = a.zeros != nullptr ? fmaf((float)zeros[so[t][u] + group], 0.0625f, 1.0f) : 1.5f;
#pragma unroll
            for (int n = 0; n < NT; ++n)
              acc[t][n][u] = fmaf(sc, fmaf(-z, sum[n][0], pl.kept(d[n], u)), acc[t][n][u]);
          }
        }
      }
    }
    join<E, F, RT, NT>(pl, a.tile, acc, ub, m0, part_sums);
  }
}

}  // namespace
}  // namespace bcjr
