// Products of a few tokens with 4-bit weights on the matrix cores (the tile: tiles.h).
//
// Codes become numbers without a subtraction: a nibble goes to the top four mantissa bits of a half or a
// bfloat16 with exponent 0 and is 1 + q / 16, exactly. With D = sum (1 + q / 16) x and S = sum x (the
// same instruction with weights of one, once for all rows of a wave), a group gives
// 16 scale (D - (1 + z / 16) S), in fp32: nothing is rounded before the last conversion.
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

// v of the 16 lanes of row t, for every row of 16 lanes.
template <int N>
__device__ inline void rows_apart(unsigned v, unsigned (&out)[N]) {
  if constexpr (N == 1) {
    out[0] = v;
  } else {
    const auto halves = __builtin_amdgcn_permlane32_swap(v, v, false, false);  // rows 0 1 0 1, rows 2 3 2 3
    const auto low = __builtin_amdgcn_permlane16_swap(halves[0], halves[0], false, false);
    out[0] = low[0];
    out[1] = low[1];
    if constexpr (N > 2) {
      const auto high = __builtin_amdgcn_permlane16_swap(halves[1], halves[1], false, false);
      out[2] = high[0];
      out[3] = high[1];
    }
  }
}

// What a step of a wave reads, in memory order: of a tile's codes a lane loads the 16 bytes next to its
// neighbour's, and of the scales those of tile g.
template <class E, int F, int RT, int NT, int GS, bool ZEROS>
struct Int4Step {
  using T = typename TileOf<E>::T;
  using V = typename T::V;
  using X = XTile<E, F, NT>;
  static constexpr int kKept = Place<E, F>::kKept, kGroups = 4 / GS;
  X x;
  u32x4 w[RT];
  float scale[kGroups];
  unsigned zero[kGroups];

  // qo: a lane's offset in the codes of tile t's step 0; so: its row of tile g in the scales.
  __device__ void load(const Int4Args& a, const Place<E, F>& pl, int s, int blocks, const unsigned* __restrict__ q,
                       const unsigned (&qo)[RT], const float* __restrict__ scales, const uint8_t* __restrict__ zeros,
                       unsigned so) {
    const int lane = threadIdx.x & 63;
    const bool in = s * F + (lane >> 2) % F < blocks;  // folds behind the last block have no codes
#pragma unroll
    for (int t = 0; t < RT; ++t)
      w[t] = in ? *reinterpret_cast<const u32x4*>(q + (qo[t] + s * (F * 16))) : u32x4{0, 0, 0, 0};
    const int unit = (s * F + pl.fold) * 4;
#pragma unroll
    for (int i = 0; i < kGroups; ++i) {
      const int group = min(divide(unit + i * GS, a.per_group), a.groups - 1);
      scale[i] = scales[so + group];
      if (ZEROS) zero[i] = zeros[so + group];
    }
    x.load(a.tile, s);
  }

  __device__ void add(const Place<E, F>& pl, char* lds, float (&acc)[RT][NT][kKept]) {
    x.put(lds);
    const int from = (4 * pl.c16 + pl.g) * 4;  // the lane that loaded this one's codes
#pragma unroll
    for (int t = 0; t < RT; ++t)
#pragma unroll
      for (int j = 0; j < 4; ++j) w[t][j] = __builtin_amdgcn_ds_bpermute(from, w[t][j]);
    V xo[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int j = 0; j < 4; ++j) xo[n][j] = X::get(lds, pl, n, 4 * j + pl.g);
    X::in_order();
    const V ones = __builtin_bit_cast(V, u32x4{T::kOne, T::kOne, T::kOne, T::kOne});
#pragma unroll
    for (int i = 0; i < kGroups; ++i) {
      f32x4 sum[NT];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        sum[n] = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int j = i * GS; j < i * GS + GS; ++j) sum[n] = T::mfma(xo[n][j], ones, sum[n]);
      }
      unsigned sc[RT], ze[RT];
      rows_apart<RT>(__float_as_uint(scale[i]), sc);
      if (ZEROS) rows_apart<RT>(zero[i], ze);
#pragma unroll
      for (int t = 0; t < RT; ++t) {
        f32x4 d[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n) d[n] = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int j = i * GS; j < i * GS + GS; ++j) {
          const V wj = weights8<T>(w[t][j]);
#pragma unroll
          for (int n = 0; n < NT; ++n) d[n] = T::mfma(xo[n][j], wj, d[n]);
        }
        const float z = ZEROS ? fmaf((float)ze[t], 0.0625f, 1.0f) : 1.5f;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int u = 0; u < kKept; ++u)
            acc[t][n][u] = fmaf(__uint_as_float(sc[t]), fmaf(-z, pl.kept(sum[n], u), pl.kept(d[n], u)), acc[t][n][u]);
      }
    }
  }
};

// F folds, RT tiles of rows and NT tiles of tokens a wave, GS products of 32 columns a scale.
template <class E, int F, int RT, int NT, int GS, bool ZEROS>
__global__ void __launch_bounds__(64 * kMaxWaves)
k_int4_tiles(const Int4Args a) {
  using Pl = Place<E, F>;
  constexpr int kRows = Pl::kRows, kKept = Pl::kKept;
  extern __shared__ __attribute__((aligned(16))) char lds[];
  const Pl pl;
  char* mine = lds + pl.wave * NT * kXBytes;
  const int kw = a.tile.kw, ki = pl.wave % kw, ri = pl.wave / kw, rw = pl.waves / kw;
  const int blocks = (a.tile.cols + 127) / 128, steps = (blocks + F - 1) / F;
  const long long rows = a.tile.rows, units = (rows + RT * kRows - 1) / (RT * kRows);  // of rows, one for a wave
  const long long m0 = (long long)blockIdx.y * (NT * Pl::kTokens);
  const int lane = threadIdx.x & 63;

  for (long long ub = (long long)blockIdx.x * rw; ub < units; ub += (long long)gridDim.x * rw) {
    const long long row0 = (ub + ri) * (RT * kRows);
    // offsets from the wave's first row fit 32 bits; rows behind the last repeat it
    const long long base = row0 < rows ? row0 : rows - 1;
    const int last = (int)(rows - 1 - base < RT * kRows ? rows - 1 - base : RT * kRows);
    const unsigned* __restrict__ q = a.q + base * a.words;
    const float* __restrict__ scales = a.scales + base * a.groups;
    const uint8_t* __restrict__ zeros = a.zeros + base * a.groups;
    unsigned qo[RT];
    float acc[RT][NT][kKept] = {};
#pragma unroll
    for (int t = 0; t < RT; ++t)
      qo[t] = (unsigned)(min(t * kRows + (lane >> 2) / F, last) * a.words + (lane >> 2) % F * 16 + 4 * (lane & 3));
    const unsigned so = (unsigned)(min(min(pl.g, RT - 1) * kRows + pl.row(), last) * a.groups);
    Int4Step<E, F, RT, NT, GS, ZEROS> one, two;
    one.x.init(a.tile, m0);
    two.x.init(a.tile, m0);
    if (ki < steps) one.load(a, pl, ki, blocks, q, qo, scales, zeros, so);
    for (int s = ki; s < steps; s += 2 * kw) {
      if (s + kw < steps) two.load(a, pl, s + kw, blocks, q, qo, scales, zeros, so);
      one.add(pl, mine, acc);
      if (s + 2 * kw < steps) one.load(a, pl, s + 2 * kw, blocks, q, qo, scales, zeros, so);
      if (s + kw < steps) two.add(pl, mine, acc);
    }
    // codes were sixteenths
#pragma unroll
    for (int t = 0; t < RT; ++t)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int u = 0; u < kKept; ++u) acc[t][n][u] *= 16.0f;
    join<E, F, RT, NT>(pl, a.tile, acc, ub, m0, lds);
  }
}

}  // namespace
}  // namespace bcjr
