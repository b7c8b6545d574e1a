// Products of a few tokens with decoded weights on the matrix cores: the tile that the 4-bit and the
// trellis-coded products share.
//
// A 16 x 16 x 32 matrix instruction multiplies 16 rows of x with 16 rows of weights. With few tokens most of
// its rows of x would be idle, so the columns of W are folded F-fold: the tile's 16 rows of weights are
// 16 / F rows of W times F neighbouring blocks of 128 columns, its 16 rows of x are 16 / F tokens times
// the same F blocks, and of the 16 x 16 sums those are kept whose blocks agree. One step of a
// wave covers F blocks of a row in consecutive memory, and one row at F = 16: 2048 columns. fp32
// inputs are three bfloat16 parts that add up to them exactly, each in a row of its own. The weights
// are the second operand: a lane's sums are then all of the row of W whose codes it read, and so is
// the scale it needs.
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
  // Columns that whole loads of eight cover. The up to seven others, if any, are added to the outputs (join()).
  __host__ __device__ int whole8() const { return cols & ~7; }
};

struct CodeArgs {
  TileArgs tile;
  const unsigned* code;
  const float* codebook;
  const float* scales;         // of a chain, or NULL
  int n, chains, words;        // state bits; chains of a row; words of a chain
  int per_chain;               // blocks of 128 columns in a chain
  float reciprocal;            // 1 / per_chain
  int L, k;                    // of chains in any relation to the blocks (code_any.h), with reciprocal = 1 / L
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
// Halves as two bfloat16 parts, where the weights' range needs bfloat16.
struct F16Parts : F16 {};
struct HalfPartsTile : BfTile {
  static constexpr int kParts = 2;
};
template <class E> struct TileOf;
template <> struct TileOf<F16Parts> { using T = HalfPartsTile; };
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

// floor(u / d) for u < 2^21 from the fp32 reciprocal of d: u + 1/2 is exact, and (u + 1/2) / d is at least 1 /
// (2 d) off any whole number, more than the two roundings' u / d 2^-23.
__device__ inline int divide(int u, float reciprocal) { return (int)(((float)u + 0.5f) * reciprocal); }

// Tokens of a tile: 16 columns are parts times folds times tokens.
template <class E, int F>
constexpr int tile_tokens() { return 16 / F / TileOf<E>::T::kParts; }
constexpr int kMaxWaves = 8;

// A lane's place: of the tile's rows of x and of weights its operands are number c16, of the 32 products
// the eight from 8 g on.
template <class E, int F>
struct Place {
  static constexpr int kRows = 16 / F;                       // rows of W in a tile
  static constexpr int kCols = 16 / F;                       // a tile's rows of x without their folds
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
  // The lane that loaded this one's codes, for ds_bpermute: four neighbouring lanes load what four lanes of one row
  // of the tile, 16 apart, need.
  __device__ int from() const { return (4 * c16 + g) * 4; }
  // Row of W in the tile, of a lane's weights and of its sums.
  __device__ int row() const { return c16 / F; }
  // Row of x, without folds, of kept sum u: the lane holds the sums of the tile's rows 4 g + i of x, and keeps
  // those whose fold is its own.
  __device__ int sum_col(int u) const {
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
};

// v of the 16 lanes of row t, for every row of 16 lanes: what lane (t, c16) loaded for the rows of tile t.
template <int N>
__device__ inline void rows_apart(unsigned v, unsigned (&out)[N]) {
  const auto halves = __builtin_amdgcn_permlane32_swap(v, v, false, false);  // rows 0 1 0 1, rows 2 3 2 3
  const auto low = __builtin_amdgcn_permlane16_swap(halves[0], halves[0], false, false);
  out[0] = low[0];
  if constexpr (N > 1) out[1] = low[1];
  if constexpr (N > 2) {
    const auto high = __builtin_amdgcn_permlane16_swap(halves[1], halves[1], false, false);
    out[2] = high[0];
    out[3] = high[1];
  }
}

// The x of one step of a wave, NT tiles of 16 rows of 128 columns. Neighbouring lanes load neighbouring
// memory, 16 lanes a row: in the operands' own order every lane of a load would be in a row, and so a
// cache line, of its own, and take a cycle of the cache instead of a quarter. The rows then go through LDS
// (each wave its own kXBytes NT), where operands are read.
constexpr int kXBytes = 16 * 256;
// Place of chunk c (16 bytes) of row r: shifted about by the row, so that neither the 16 chunks of a row nor one
// chunk of eight rows meet a bank twice.
__device__ inline int x_place(int r, int c) { return r * 256 + (c ^ r) * 16; }

// Where a lane's loads begin, from the first token's row on (in_pieces() sees to it that 32 bits hold that):
// rows behind the last token repeat it (their sums are not kept).
template <class E, int F, int NT>
struct XRows {
  static constexpr int kTokens = tile_tokens<E, F>();
  static constexpr int kLoads = (kTokens * F + 3) / 4;  // of four rows each
  const typename E::T* first;
  unsigned at[NT][kLoads];
  __device__ XRows(const TileArgs& a, long long m0) {
    const int lane = threadIdx.x & 63;
    const int last = (int)(a.tokens - 1 - m0 < NT * kTokens ? a.tokens - 1 - m0 : NT * kTokens);
    first = static_cast<const typename E::T*>(a.x) + m0 * a.xs;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const int r = 4 * i + (lane >> 4);
        at[n][i] = (unsigned)min(n * kTokens + r / F, last) * (unsigned)a.xs + r % F * 128 + (lane & 15) * 8;
      }
  }
};

template <class E, int F, int NT>
struct XTile {
  using T = typename TileOf<E>::T;
  using V = typename T::V;
  using X = typename E::T;
  using Rows = XRows<E, F, NT>;
  static constexpr int kParts = T::kParts, kTokens = tile_tokens<E, F>(), kLoads = Rows::kLoads;
  typename Loose<X, 8>::V raw[NT][kLoads];

  // Step s: columns s F 128 and on. With TAIL those from a.whole8() on are not there and are zero.
  template <bool TAIL>
  __device__ void load(const TileArgs& a, const Rows& rows, int s) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const auto* p = reinterpret_cast<const typename Loose<X, 8>::V*>(rows.first + s * (F * 128) + rows.at[n][i]);
        if (!TAIL || s * (F * 128) + (4 * i + (lane >> 4)) % F * 128 + (lane & 15) * 8 < a.whole8())
          raw[n][i] = *p;
        else
          raw[n][i] = typename Loose<X, 8>::V{};
      }
  }
  __device__ void put(char* lds) const {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const int r = 4 * i + (lane >> 4);
        char* at = lds + n * kXBytes;
        if constexpr (kParts == 1) {
          *reinterpret_cast<V*>(at + x_place(r, lane & 15)) = raw[n][i];
        } else {
          // bfloat16 parts that add up to x: its leading 8 bits, the next 8 and (fp32) the rest
          u32x4 part[3];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            unsigned hi[2], mid[2], low[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const float x = (float)raw[n][i][2 * j + k];
              hi[k] = __float_as_uint(x);
              const float left = x - __uint_as_float(hi[k] & 0xffff0000u);
              mid[k] = __float_as_uint(left);
              low[k] = __float_as_uint(left - __uint_as_float(mid[k] & 0xffff0000u));
            }
            part[0][j] = __builtin_amdgcn_perm(hi[1], hi[0], 0x07060302);
            part[1][j] = __builtin_amdgcn_perm(mid[1], mid[0], 0x07060302);
            part[2][j] = __builtin_amdgcn_perm(low[1], low[0], 0x07060302);
          }
          if (kLoads * 4 == kTokens * F || r < kTokens * F)
#pragma unroll
            for (int p = 0; p < kParts; ++p)
              *reinterpret_cast<u32x4*>(at + x_place((r / F * kParts + p) * F + r % F, lane & 15)) = part[p];
        }
      }
    in_order();
  }
  // The operand of a lane from chunk `chunk` (8 columns) of its row.
  static __device__ V get(const char* lds, const Place<E, F>& pl, int n, int chunk) {
    return *reinterpret_cast<const V*>(lds + n * kXBytes + x_place(pl.c16, chunk));
  }
  // Lanes of a wave read what others wrote: LDS works in order, the compiler has to as well.
  static __device__ void in_order() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
  }
};

// The outputs: sums over the block's waves that share rows, the parts of x and the folds, and rest(row, x) for the
// columns behind the last eight. The kept sums [RT][kRows][NT][kCols][F] go to where each wave's x was.
template <class E, int F, int RT, int NT, class Rest>
__device__ inline void join(const Place<E, F>& pl, const TileArgs& a, float (&acc)[RT][NT][Place<E, F>::kKept],
                            long long first_unit, long long m0, char* lds, Rest rest) {
  using P = Place<E, F>;
  constexpr int kParts = TileOf<E>::T::kParts, kRows = P::kRows, kCols = P::kCols, kTokens = P::kTokens;
  static_assert(RT * kRows * kCols * F * 4 <= kXBytes, "a wave's sums take the place of its x");
  const int kw = a.kw, rw = pl.waves / kw;
  float* sums = reinterpret_cast<float*>(lds + pl.wave * NT * kXBytes);
  XTile<E, F, NT>::in_order();
  // for F > 4 only the lanes whose rows of x have their own fold hold a sum
  const bool mine = F <= 4 || (F == 8 ? (pl.c16 >> 2 & 1) == (pl.g & 1) : pl.c16 >> 2 == pl.g);
  if (mine) {
#pragma unroll
    for (int t = 0; t < RT; ++t)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int u = 0; u < P::kKept; ++u)
          sums[(((t * kRows + pl.row()) * NT + n) * kCols + pl.sum_col(u)) * F + pl.fold] = acc[t][n][u];
  }
  __syncthreads();
  // F neighbouring lanes an output, each a fold
  constexpr int kOuts = RT * kRows * NT * kTokens;
  for (int o = threadIdx.x / F; o < rw * kOuts; o += blockDim.x / F) {
    const int grp = o / kOuts, out = o % kOuts, tr = out / (NT * kTokens), mt = out % (NT * kTokens);
    const int at = ((tr * NT + mt / kTokens) * kCols + mt % kTokens * kParts) * F + threadIdx.x % F;
    float v = 0.0f;
    for (int k = 0; k < kw; ++k) {
      const float* s = reinterpret_cast<const float*>(lds + (grp * kw + k) * NT * kXBytes) + at;
#pragma unroll
      for (int p = kParts - 1; p >= 0; --p) v += s[p * F];
    }
#pragma unroll
    for (int d = 1; d < F; d <<= 1) v += __shfl_xor(v, d, 64);
    const long long r = (first_unit + grp) * (RT * kRows) + tr, m = m0 + mt;
    if (threadIdx.x % F == 0 && r < a.rows && m < a.tokens) {
      v += rest(r, static_cast<const typename E::T*>(a.x) + m * a.xs);
      E::store(static_cast<typename E::T*>(a.y) + m * a.ys + r, v);
    }
  }
  __syncthreads();
}

}  // namespace

constexpr size_t kLds = 160 * 1024;  // of a compute unit, all of which one block may take

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

// Calls f with the tokens in pieces that one launch's grid holds, 32768 tiles of at least 5, or, where the rows of
// x lie so far apart that 32-bit offsets do not reach over 32 of them, one by one.
template <class Fn>
inline int in_pieces(MatvecIO io, int dtype_size, Fn f) {
  const int64_t most = io.x_stride < ((int64_t)1 << 24) + 1 ? 5 * 32768 : 1, total = io.tokens;
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
