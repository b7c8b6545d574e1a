// Products of a few tokens with decoded weights on the matrix cores: the tile that the 4-bit and the
// trellis-coded products share.
//
// A 16 x 16 x 32 matrix instruction multiplies 16 rows of weights with 16 columns of x. With few
// tokens most of its columns would be idle, so the columns of W are folded F-fold: the tile's 16 rows are
// 16 / F rows of W times F neighbouring blocks of 128 columns, its 16 columns are 16 / F tokens times
// the same F blocks, and of the 16 x 16 sums those are kept whose blocks agree. One step of a
// wave covers F blocks of a row in consecutive memory, and one row at F = 16: 2048 columns. fp32
// inputs are three bfloat16 parts that add up to them exactly, each in a column of its own.
#pragma once
#include <hip/hip_runtime.h>

#include <type_traits>

#include "ops.h"
#include "ops_device.h"

namespace bcjr {

// What every tiled product is told.
struct TileArgs {
  const void* x;
  void* y;
  long long rows, tokens, xs, ys;
  int cols;
  int kw;  // waves of a block that share a row, each with every kw-th step
};

namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef unsigned u32x4 __attribute__((ext_vector_type(4)));

// What differs between the types: the operand, the parts of an x, where a 4-bit code is placed.
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

// Part `part` of x (0: the leading 8 bits, 1: the next 8, 2: the rest) as bfloat16 bits.
__device__ inline unsigned part_of(float x, int part) {
  const float hi = __uint_as_float(__float_as_uint(x) & 0xffff0000u), r = x - hi;
  const float mid = __uint_as_float(__float_as_uint(r) & 0xffff0000u);
  return __float_as_uint(part == 0 ? hi : part == 1 ? mid : r - mid) >> 16;
}

// Vectors at any element's address: the memory system splits what crosses a line, so x needs no alignment
// and no second path.
template <class T, int N> struct Loose;
template <class T> struct Loose<T, 8> { typedef T V __attribute__((ext_vector_type(8), aligned(sizeof(T)))); };
template <class T> struct Loose<T, 4> { typedef T V __attribute__((ext_vector_type(4), aligned(sizeof(T)))); };

// x[col .. col + 7] as an operand, zeros from cols on.
template <class E>
__device__ inline typename TileOf<E>::T::V load_x8(const typename E::T* row, int col, int cols, int part) {
  using V = typename TileOf<E>::T::V;
  using X = typename E::T;
  const X* p = row + col;
  if constexpr (TileOf<E>::T::kParts == 1) {
    if (col + 8 <= cols) return *reinterpret_cast<const typename Loose<X, 8>::V*>(p);
    V v;
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = col + i < cols ? p[i] : (X)0.0f;
    return v;
  } else {
    float f[8];
    if (col + 8 <= cols) {
      const auto a = *reinterpret_cast<const Loose<float, 4>::V*>(p), b = *reinterpret_cast<const Loose<float, 4>::V*>(p + 4);
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

// floor(u / d) for u < 2^21 from the fp32 reciprocal of d: u + 1/2 is exact, and (u + 1/2) / d is at least 1 /
// (2 d) off any whole number, more than the two roundings' u / d 2^-23.
__device__ inline int divide(int u, float reciprocal) { return (int)(((float)u + 0.5f) * reciprocal); }

// Tokens of a tile: 16 columns are parts times folds times tokens.
template <class E, int F>
constexpr int tile_tokens() { return 16 / F / TileOf<E>::T::kParts; }
constexpr int kMaxWaves = 8;

// A lane's place: of the tile's rows and columns its operands are number c16, of the 32 products the
// eight from 8 g on.
template <class E, int F>
struct Place {
  static constexpr int kRows = 16 / F;                       // rows of W in a tile
  static constexpr int kCols = 16 / F;                       // a tile's columns without their folds
  static constexpr int kKept = F == 1 ? 4 : F == 2 ? 2 : 1;  // sums of a lane that are kept
  static constexpr int kTokens = tile_tokens<E, F>();
  int c16, g, fold, col, wave, waves;
  __device__ Place() {
    const int lane = threadIdx.x & 63;
    wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    waves = blockDim.x >> 6;
    c16 = lane & 15;
    g = lane >> 4;
    fold = c16 % F;
    col = c16 / F;
  }
  // Row of the tile that a lane's weights are of.
  __device__ int weight_row() const { return c16 / F; }
  // Row of the tile of kept sum u: the lane holds the sums of the tile's rows 4 g + i, and keeps those
  // whose fold is its own.
  __device__ int sum_row(int u) const {
    const int i = F >= 4 ? c16 % 4 : F == 2 ? 2 * u + fold : u;
    return (4 * g + i) / F;
  }
  // Kept sum u of four (F = 8 and 16: garbage in the lanes that keep none; join() drops it).
  __device__ float kept(f32x4 d, int u) const {
    if constexpr (F == 1) return d[u];
    if constexpr (F == 2) return fold ? d[2 * u + 1] : d[2 * u];
    const float lo = c16 & 1 ? d[1] : d[0], hi = c16 & 1 ? d[3] : d[2];
    return c16 & 2 ? hi : lo;
  }
  // x of column tile n, for tokens from m0 on: columns behind the last token repeat it.
  __device__ const typename E::T* x_row(const TileArgs& a, long long m0, int n) const {
    const long long m = m0 + n * kTokens + col / TileOf<E>::T::kParts;
    return static_cast<const typename E::T*>(a.x) + (m < a.tokens ? m : a.tokens - 1) * a.xs;
  }
  __device__ int x_part() const { return col % TileOf<E>::T::kParts; }
};

// The wave's sums over folds, the block's over waves and the parts of x, and the outputs. Rows
// from row0 on belong to this wave's group of kw; part_sums [waves][RT][kRows][NT][kCols] in LDS.
template <class E, int F, int RT, int NT>
__device__ inline void join(const Place<E, F>& pl, const TileArgs& a, float (&acc)[RT][NT][Place<E, F>::kKept],
                            long long first_unit, long long m0, float* part_sums) {
  using T = typename TileOf<E>::T;
  constexpr int kRows = Place<E, F>::kRows, kCols = Place<E, F>::kCols, kTokens = Place<E, F>::kTokens;
  const int c16 = pl.c16, g = pl.g, kw = a.kw, rw = pl.waves / kw;
  // sums over the folds within the wave; for F > 4 only the lanes whose rows' folds are their own hold one
  const bool mine = F <= 4 || (F == 8 ? (c16 >> 2 & 1) == (g & 1) : c16 >> 2 == g);
#pragma unroll
  for (int t = 0; t < RT; ++t)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int u = 0; u < Place<E, F>::kKept; ++u) {
        float v = mine ? acc[t][n][u] : 0.0f;
#pragma unroll
        for (int d = 1; d < F; d <<= 1) v += __shfl_xor(v, d, 64);
        if constexpr (F == 8) v += __shfl_xor(v, 16, 64);
        if constexpr (F == 16) {
          v += __shfl_xor(v, 16, 64);
          v += __shfl_xor(v, 32, 64);
        }
        if (pl.fold == 0 && (F <= 4 || (F == 8 ? (g & 1) == 0 : g == 0)))
          part_sums[(((pl.wave * RT + t) * kRows + pl.sum_row(u)) * NT + n) * kCols + pl.col] = v;
      }
  __syncthreads();
  // one output at a time: over the waves of its rows and the parts of x
  const int outs = RT * kRows * NT * kTokens;
  for (int o = threadIdx.x; o < rw * outs; o += blockDim.x) {
    const int grp = o / outs, rest = o - grp * outs, tr = rest / (NT * kTokens), mt = rest % (NT * kTokens);
    const long long r = (first_unit + grp) * (RT * kRows) + tr, m = m0 + mt;
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

}  // namespace

// Waves along a row while that leaves each at least one step and the chip is not yet full: 8
// waves on each of 256 CUs.
inline int waves_along(int steps, int64_t units) {
  int kw = 1;
  while (kw < kMaxWaves && kw * 2 <= steps && units * kw < 2048) kw *= 2;
  return kw;
}

// Products in tiles: columns are 32-bit numbers below 2^24 (divide()).
constexpr int64_t kTileColumns = (int64_t)1 << 24;

inline TileArgs tile_args(const MatvecIO& io, int64_t rows, int64_t cols) {
  TileArgs t;
  t.x = io.x;
  t.y = io.y;
  t.rows = rows;
  t.tokens = io.tokens;
  t.xs = io.x_stride;
  t.ys = io.y_stride;
  t.cols = (int)cols;
  t.kw = 1;
  return t;
}

// Calls f with the tokens in pieces that one launch's grid holds: 32768 tiles of at least 5.
template <class Fn>
inline int in_pieces(MatvecIO io, int dtype_size, Fn f) {
  const int64_t most = 5 * 32768, total = io.tokens;
  for (int64_t m = 0; m < total; m += most) {
    MatvecIO p = io;
    p.tokens = total - m < most ? total - m : most;
    p.x = static_cast<const char*>(io.x) + m * io.x_stride * dtype_size;
    p.y = static_cast<char*>(io.y) + m * io.y_stride * dtype_size;
    if (const int e = f(p)) return e;
  }
  return 0;
}

}  // namespace bcjr
