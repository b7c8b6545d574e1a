// Products of a few tokens with 4-bit weights on the matrix cores (the tile: tiles.h).
//
// Codes become numbers without a subtraction: a nibble goes to the top four mantissa bits of a half or a
// bfloat16 with exponent 0 and is 1 + q / 16, exactly. With D = sum (1 + q / 16) x and S = sum x (the
// same instruction with weights of one, once for all rows of a wave), a group gives
// 16 scale (D - (1 + z / 16) S), in fp32: nothing is rounded before the last conversion.
//
// One token is bound by memory where the matrix is large (16384 x 16384 in 34.5 us, 4.1 TB/s) and by latency where it is
// not (2048 x 8192 5.5 us, 512 x 1024 3.2). 32 tokens through 16384 x 16384 take 55 us: 28 of memory, 18 of LDS, 16 of
// unpacking and 9 of products, which the 2 waves a SIMD that the registers leave room for overlap in part.
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

// The word of a row that holds columns 8 u .. 8 u + 7.
__device__ inline long long word_of(long long u) {
  return (u & ~15ll) + 4 * (u & 3) + ((u >> 2) & 3);
}
// The low bit of column c (0 .. 7) of a word.
__device__ inline int nibble_shift(int c) { return 4 * ((c >> 1) + 4 * (c & 1)); }

// The eight weights of a word as numbers 1 + q / 16.
template <class T>
__device__ inline typename T::V weights8(unsigned w, unsigned one) {
  u32x4 v;
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    const int up = T::kUp - 4 * p;
    const unsigned at = up >= 0 ? w << up : w >> -up;
    // one instruction, which the compiler makes of two constants only if one of them is in a vector register
    asm("v_and_or_b32 %0, %1, %2, %3" : "=v"(v[p]) : "v"(at), "s"(T::kMask), "v"(one));
  }
  return __builtin_bit_cast(typename T::V, v);
}

// What a step of a wave reads, asked for while the one before is computed, in memory order: of a tile's codes a lane loads the 16 bytes next to its
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

  // q: the codes of step s, qo: a lane's offset there in tile t; so: its row of tile g in the scales. With TAIL
  // some of the step's columns, and some folds, are not there.
  template <bool TAIL>
  __device__ void load(const Int4Args& a, const Place<E, F>& pl, int s, const unsigned* __restrict__ q,
                       const unsigned (&qo)[RT], const float* __restrict__ scales, const uint8_t* __restrict__ zeros,
                       unsigned so, const typename X::Rows& rows) {
    const int lane = threadIdx.x & 63;
    const bool in = !TAIL || (s * F + (lane >> 2) % F) * 128 < a.tile.cols;  // codes end with the last block
#pragma unroll
    for (int t = 0; t < RT; ++t)
      w[t] = in ? *reinterpret_cast<const u32x4*>(q + s * (F * 16) + qo[t]) : u32x4{0, 0, 0, 0};
    const int unit = (s * F + pl.fold) * 4;
#pragma unroll
    for (int i = 0; i < kGroups; ++i) {
      int group = divide(unit + i * GS, a.per_group);
      if (TAIL) group = min(group, a.groups - 1);
      scale[i] = pl.g < RT ? scales[so + group] : 0.0f;
      if (ZEROS) zero[i] = pl.g < RT ? zeros[so + group] : 0u;
    }
    x.template load<TAIL>(a.tile, rows, s);
  }

  // What the products take, from what was loaded: its registers are free for the next step's loads then.
  struct Operands {
    V x[NT][4];
    unsigned w[RT][4];
    unsigned scale[kGroups][RT], zero[kGroups][RT];

    __device__ void add(const Place<E, F>& pl, float (&acc)[RT][NT][kKept]) const {
      unsigned one = T::kOne;
      asm("" : "+v"(one));  // kept in a vector register
      const V ones = __builtin_bit_cast(V, u32x4{one, one, one, one});
#pragma unroll
      for (int i = 0; i < kGroups; ++i) {
        f32x4 sum[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          sum[n] = f32x4{0, 0, 0, 0};
#pragma unroll
          for (int j = i * GS; j < i * GS + GS; ++j) sum[n] = T::mfma(x[n][j], ones, sum[n]);
        }
#pragma unroll
        for (int t = 0; t < RT; ++t) {
          f32x4 d[NT];
#pragma unroll
          for (int n = 0; n < NT; ++n) d[n] = f32x4{0, 0, 0, 0};
#pragma unroll
          for (int j = i * GS; j < i * GS + GS; ++j) {
            const V wj = weights8<T>(w[t][j], one);
#pragma unroll
            for (int n = 0; n < NT; ++n) d[n] = T::mfma(x[n][j], wj, d[n]);
          }
          const float z = ZEROS ? fmaf((float)zero[i][t], 0.0625f, 1.0f) : 1.5f;
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int u = 0; u < kKept; ++u)
              acc[t][n][u] = fmaf(__uint_as_float(scale[i][t]), fmaf(-z, pl.kept(sum[n], u), pl.kept(d[n], u)), acc[t][n][u]);
        }
      }
    }
  };

  __device__ void exchange(const Place<E, F>& pl, char* lds, Operands& o) const {
    x.put(lds);
#pragma unroll
    for (int t = 0; t < RT; ++t)
#pragma unroll
      for (int j = 0; j < 4; ++j) o.w[t][j] = __builtin_amdgcn_ds_bpermute(pl.from(), w[t][j]);
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int j = 0; j < 4; ++j) o.x[n][j] = X::get(lds, pl, n, 4 * j + pl.g);
    X::in_order();
#pragma unroll
    for (int i = 0; i < kGroups; ++i) {
      rows_apart<RT>(__float_as_uint(scale[i]), o.scale[i]);
      if (ZEROS) rows_apart<RT>(zero[i], o.zero[i]);
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
  const int whole = a.tile.cols / (F * 128), steps = whole + (whole * (F * 128) < a.tile.whole8() ? 1 : 0);
  const long long rows = a.tile.rows, units = (rows + RT * kRows - 1) / (RT * kRows);  // of rows, one for a wave
  const long long m0 = (long long)blockIdx.y * (NT * Pl::kTokens);
  const int lane = threadIdx.x & 63;
  const XRows<E, F, NT> xrows(a.tile, m0);

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
    using Step = Int4Step<E, F, RT, NT, GS, ZEROS>;
    Step step;
    auto load = [&](int s) {
      if (s < whole)
        step.template load<false>(a, pl, s, q, qo, scales, zeros, so, xrows);
      else
        step.template load<true>(a, pl, s, q, qo, scales, zeros, so, xrows);
    };
    if (ki < steps) load(ki);
    for (int s = ki; s < steps; s += kw) {
      typename Step::Operands o;
      step.exchange(pl, mine, o);
      if (s + kw < steps) load(s + kw);
      o.add(pl, acc);
    }
    // codes were sixteenths
#pragma unroll
    for (int t = 0; t < RT; ++t)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int u = 0; u < kKept; ++u) acc[t][n][u] *= 16.0f;
    join<E, F, RT, NT>(pl, a.tile, acc, ub, m0, lds, [&](long long r, const typename E::T* x) {
      const int c8 = a.tile.whole8();
      float sum = 0.0f;
      if (c8 < a.tile.cols) {  // all in one word and one group
        const unsigned word = a.q[r * a.words + word_of(c8 / 8)];
        const float z = ZEROS ? (float)a.zeros[r * a.groups + a.groups - 1] : 8.0f;
        for (int c = c8; c < a.tile.cols; ++c) sum = fmaf((float)(word >> nibble_shift(c - c8) & 15u) - z, E::load(x + c), sum);
        sum *= a.scales[r * a.groups + a.groups - 1];
      }
      return sum;
    });
  }
}

}  // namespace
}  // namespace bcjr
