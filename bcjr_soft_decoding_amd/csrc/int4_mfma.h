// Products of a few tokens with 4-bit weights on the matrix cores.
//
// A 16 x 16 x 32 matrix instruction multiplies 16 rows of weights with 16 columns of x. With few
// tokens most of its columns would be idle, so the columns of W are folded F-fold: the tile's 16 rows are
// 16 / F rows of W times F neighbouring blocks of 128 columns, its 16 columns are 16 / F tokens times
// the same F blocks, and of the 16 x 16 sums those are kept whose blocks agree. One step of a
// wave covers F blocks of a row in consecutive memory, and one row at F = 16: 2048 columns.
//
// Codes become numbers without a subtraction: a nibble goes to the top four mantissa bits of a half or a
// bfloat16 with exponent 0 and is 1 + q / 16, exactly. With D = sum (1 + q / 16) x and S = sum x (the
// same instruction with weights of one, once for all rows of a wave), a group gives
// scale (16 D - (16 + z) S), in fp32: nothing is rounded before the last conversion. fp32 inputs are
// three bfloat16 parts that add up to them exactly, each in a column of its own.
#pragma once
#include <hip/hip_runtime.h>

#include "ops.h"
#include "ops_device.h"

namespace bcjr {

struct Int4Args {
  const unsigned* q;
  const float* scales;
  const uint8_t* zeros;
  long long rows, tokens, xs, ys;
  const void* x;
  void* y;
  int cols, groups, words;
  unsigned per_group, magic;  // units of 32 columns in a group; ceil(2^32 / per_group) for > 1
  int kw;                     // waves of a block that share a row, each with every kw-th step
  int wide;                   // rows of x are aligned to 16 bytes
};

namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef unsigned u32x4 __attribute__((ext_vector_type(4)));

// What differs between the types: the operand, the placing of nibbles, the parts of an x.
struct HalfTile {
  using V = f16x8;
  static constexpr int kParts = 1, kUp = 6;  // the nibble's place: mantissa bits 6 .. 9 of 10
  static constexpr unsigned kMask = 0x03c003c0u, kOne = 0x3c003c00u;
  static __device__ f32x4 mfma(V a, V b, f32x4 c) { return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0); }
};
struct BfTile {
  using V = bf16x8;
  static constexpr int kParts = 1, kUp = 3;  // mantissa bits 3 .. 6 of 7
  static constexpr unsigned kMask = 0x00780078u, kOne = 0x3f803f80u;
  static __device__ f32x4 mfma(V a, V b, f32x4 c) { return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0); }
};
struct FloatTile : BfTile {
  static constexpr int kParts = 3;
};
template <class E> struct TileOf;
template <> struct TileOf<F32> { using T = FloatTile; };
template <> struct TileOf<F16> { using T = HalfTile; };
template <> struct TileOf<BF16> { using T = BfTile; };

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

// Part `part` of x (0: the leading 8 bits, 1: the next 8, 2: the rest) as bfloat16 bits.
__device__ inline unsigned part_of(float x, int part) {
  const float hi = __uint_as_float(__float_as_uint(x) & 0xffff0000u), r = x - hi;
  const float mid = __uint_as_float(__float_as_uint(r) & 0xffff0000u);
  return __float_as_uint(part == 0 ? hi : part == 1 ? mid : r - mid) >> 16;
}

// x[col .. col + 7] as an operand, zeros from cols on.
template <class E>
__device__ inline typename TileOf<E>::T::V load_x8(const typename E::T* row, int col, int cols, int wide, int part) {
  using V = typename TileOf<E>::T::V;
  const typename E::T* p = row + col;
  if constexpr (TileOf<E>::T::kParts == 1) {
    if (wide && col + 8 <= cols) return *reinterpret_cast<const V*>(p);
    V v;
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = col + i < cols ? p[i] : (typename E::T)0.0f;
    return v;
  } else {
    float f[8];
    if (wide && col + 8 <= cols) {
      const f32x4 a = *reinterpret_cast<const f32x4*>(p), b = *reinterpret_cast<const f32x4*>(p + 4);
#pragma unroll
      for (int i = 0; i < 4; ++i) f[i] = a[i], f[4 + i] = b[i];
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = col + i < cols ? p[i] : 0.0f;
    }
    u32x4 v;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = part_of(f[2 * i], part) | part_of(f[2 * i + 1], part) << 16;
    return __builtin_bit_cast(V, v);
  }
}

// Tokens of a tile: 16 columns are parts times folds times tokens.
template <class E, int F>
constexpr int tile_tokens() { return 16 / F / TileOf<E>::T::kParts; }
constexpr int kMaxWaves = 8;

// F folds, RT tiles of rows and NT tiles of tokens a wave, GS products of 32 columns a scale.
template <class E, int F, int RT, int NT, int GS>
__global__ void __launch_bounds__(64 * kMaxWaves)
k_int4_tiles(const Int4Args a) {
  using T = typename TileOf<E>::T;
  using V = typename T::V;
  constexpr int kRows = 16 / F;                       // rows of W in a tile
  constexpr int kKept = F == 1 ? 4 : F == 2 ? 2 : 1;  // sums of a lane that are kept
  constexpr int kTokens = tile_tokens<E, F>();
  constexpr int kCols = 16 / F;                       // a tile's columns without their folds
  extern __shared__ float part_sums[];                // [waves][RT][kRows][NT][kCols]
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
  const int c16 = lane & 15, g = lane >> 4, fold = c16 % F, col = c16 / F;
  const int kw = a.kw, ki = wave % kw, ri = wave / kw, rw = waves / kw;
  const int blocks = (a.cols + 127) / 128, steps = (blocks + F - 1) / F;
  const long long units = (a.rows + RT * kRows - 1) / (RT * kRows);  // of rows, one for a wave
  const long long m0 = (long long)blockIdx.y * (NT * kTokens);
  const int xpart = col % T::kParts;
  const typename E::T* xr[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    long long m = m0 + n * kTokens + col / T::kParts;  // columns behind the last token repeat it
    m = m < a.tokens ? m : a.tokens - 1;
    xr[n] = static_cast<const typename E::T*>(a.x) + m * a.xs;
  }
  V ones;
  {
    u32x4 v;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = T::kOne;
    ones = __builtin_bit_cast(V, v);
  }

  for (long long ub = (long long)blockIdx.x * rw; ub < units; ub += (long long)gridDim.x * rw) {
    const long long row0 = (ub + ri) * (RT * kRows);
    // offsets from the wave's first row fit 32 bits; rows behind the last repeat it
    const long long base = row0 < a.rows ? row0 : a.rows - 1;
    const int last = (int)(a.rows - 1 - base < RT * kRows ? a.rows - 1 - base : RT * kRows);
    const unsigned* __restrict__ q = a.q + base * a.words;
    const float* __restrict__ scales = a.scales + base * a.groups;
    const uint8_t* __restrict__ zeros = a.zeros + base * a.groups;
    unsigned qo[RT], so[RT][kKept];
    float acc[RT][NT][kKept] = {};
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      qo[t] = (unsigned)(min(t * kRows + c16 / F, last) * a.words + 4 * g);
#pragma unroll
      for (int u = 0; u < kKept; ++u) {
        // the kept sums of a lane are of the tile's rows 4 g + i whose fold is the lane's own
        const int i = F >= 4 ? c16 % 4 : F == 2 ? 2 * u + fold : u;
        so[t][u] = (unsigned)(min(t * kRows + (4 * g + i) / F, last) * a.groups);
      }
    }
    for (int s = ki; s < steps; s += kw) {
      const int block = s * F + fold;
      const bool in = block < blocks;
      u32x4 w[RT];
#pragma unroll
      for (int t = 0; t < RT; ++t) w[t] = in ? *reinterpret_cast<const u32x4*>(q + (qo[t] + block * 16)) : u32x4{0, 0, 0, 0};
      V x[NT][4];
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (in) {
            x[n][j] = load_x8<E>(xr[n], block * 128 + 32 * j + 8 * g, a.cols, a.wide, xpart);
          } else {
            x[n][j] = __builtin_bit_cast(V, u32x4{0, 0, 0, 0});
          }
        }
#pragma unroll
      for (int j0 = 0; j0 < 4; j0 += GS) {
        const unsigned unit = (unsigned)block * 4 + j0;
        int group = (int)(a.per_group == 1 ? unit : __umulhi(unit, a.magic));
        group = group < a.groups ? group : a.groups - 1;
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
            for (int n = 0; n < NT; ++n) {
              float v;
              if constexpr (F == 1) {
                v = d[n][u];
              } else if constexpr (F == 2) {
                v = fold ? d[n][2 * u + 1] : d[n][2 * u];
              } else {
                const float lo = c16 & 1 ? d[n][1] : d[n][0], hi = c16 & 1 ? d[n][3] : d[n][2];
                v = c16 & 2 ? hi : lo;
              }
              acc[t][n][u] = fmaf(sc, fmaf(-z, sum[n][0], v), acc[t][n][u]);
            }
          }
        }
      }
    }
    // sums over the folds within the wave; for F > 4 only the lanes whose rows' folds are their own hold one
    const bool mine = F <= 4 || (F == 8 ? (c16 >> 2 & 1) == (g & 1) : c16 >> 2 == g);
#pragma unroll
    for (int t = 0; t < RT; ++t)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int u = 0; u < kKept; ++u) {
          float v = mine ? acc[t][n][u] : 0.0f;
#pragma unroll
          for (int d = 1; d < F; d <<= 1) v += __shfl_xor(v, d, 64);
          if constexpr (F == 8) v += __shfl_xor(v, 16, 64);
          if constexpr (F == 16) {
            v += __shfl_xor(v, 16, 64);
            v += __shfl_xor(v, 32, 64);
          }
          // row of the tile whose sum this is
          const int r = F == 1 ? 4 * g + u : F == 2 ? 2 * g + u : F == 4 ? g : F == 8 ? g >> 1 : 0;
          if (fold == 0 && (F <= 4 || (F == 8 ? (g & 1) == 0 : g == 0)))
            part_sums[(((wave * RT + t) * kRows + r) * NT + n) * kCols + col] = v;
        }
    __syncthreads();
    // one output at a time: over the waves of its rows and the parts of x
    const int outs = RT * kRows * NT * kTokens;
    for (int o = threadIdx.x; o < rw * outs; o += blockDim.x) {
      const int grp = o / outs, rest = o - grp * outs, tr = rest / (NT * kTokens), mt = rest % (NT * kTokens);
      const long long r = (ub + grp) * (RT * kRows) + tr, m = m0 + mt;
      if (r < a.rows && m < a.tokens) {
        float v = 0.0f;
        for (int k = 0; k < kw; ++k) {
          const float* ps = part_sums + (((grp * kw + k) * RT * kRows + tr) * NT + mt / kTokens) * kCols + mt % kTokens * T::kParts;
#pragma unroll
          for (int p = T::kParts - 1; p >= 0; --p) v += ps[p];
        }
        E::store(static_cast<typename E::T*>(a.y) + m * a.ys + r, v);
      }
    }
    __syncthreads();
  }
}

}  // namespace
}  // namespace bcjr
