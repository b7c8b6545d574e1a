// Products of a few tokens with trellis-coded weights on the matrix cores (the tile: tiles.h).
//
// A lane decodes 32 neighbouring weights of a chain: they begin at a whole word of its code, whatever
// k, and lie in k + 1 words. A window of the bit string is two words shifted into one, which holds the
// states of several neighbours; a state is a shift and a mask away, and its codeword one read of a
// table in LDS. The table holds a codeword as two 16-bit parts, c = hi + lo to 2^-16 (bfloat16) or
// 2^-21 (half) of c, each multiplied on its own: one read serves both, and rounding weights to 16 bits
// alone would cost as much precision as rounding the result. fp32 inputs get fp32 codewords, taken
// apart into three bfloat16 after the read.
#pragma once
#include "tiles.h"

namespace bcjr {

struct CodeArgs {
  TileArgs tile;
  const unsigned* code;
  const float* codebook;
  const float* scales;         // of a chain, or NULL
  int n, chains, words;        // state bits; chains of a row; words of a chain
  int per_chain;               // blocks of 128 columns in a chain
  float reciprocal;            // 1 / per_chain
};

namespace {

// Part sums of 8 weights: what the table holds for a type, and its products with x.
template <class E>
struct Codeword {  // bfloat16: hi in the upper half, lo in the lower
  static __device__ unsigned entry(float c, float) {
    const __bf16 hi = (__bf16)c, lo = (__bf16)(c - (float)hi);
    return (unsigned)__builtin_bit_cast(unsigned short, hi) << 16 | __builtin_bit_cast(unsigned short, lo);
  }
};
template <>
struct Codeword<F16> {  // half, the codebook scaled by a power of two that brings its largest to [2^13, 2^14)
  static __device__ unsigned entry(float c, float scale) {
    c *= scale;
    const _Float16 hi = (_Float16)c, lo = (_Float16)(c - (float)hi);
    return (unsigned)__builtin_bit_cast(unsigned short, hi) << 16 | __builtin_bit_cast(unsigned short, lo);
  }
};
template <>
struct Codeword<F32> {
  static __device__ unsigned entry(float c, float) { return __float_as_uint(c); }
};

template <class T, int PARTS>
__device__ inline f32x4 add_products(const unsigned (&e)[8], typename T::V x, f32x4 d) {
  if constexpr (PARTS == 2) {
    u32x4 hi, lo;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      hi[i] = __builtin_amdgcn_perm(e[2 * i + 1], e[2 * i], 0x07060302);
      lo[i] = __builtin_amdgcn_perm(e[2 * i + 1], e[2 * i], 0x05040100);
    }
    d = T::mfma(x, __builtin_bit_cast(typename T::V, lo), d);
    return T::mfma(x, __builtin_bit_cast(typename T::V, hi), d);
  } else {
    u32x4 p[3];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float r[2];
      unsigned mid[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const unsigned u = e[2 * i + j];
        r[j] = __uint_as_float(u) - __uint_as_float(u & 0xffff0000u);
        mid[j] = __float_as_uint(r[j]);
        r[j] -= __uint_as_float(mid[j] & 0xffff0000u);
      }
      p[0][i] = __builtin_amdgcn_perm(e[2 * i + 1], e[2 * i], 0x07060302);
      p[1][i] = __builtin_amdgcn_perm(mid[1], mid[0], 0x07060302);
      p[2][i] = __builtin_amdgcn_perm(__float_as_uint(r[1]), __float_as_uint(r[0]), 0x07060302);
    }
#pragma unroll
    for (int i = 2; i >= 0; --i) d = T::mfma(x, __builtin_bit_cast(typename T::V, p[i]), d);
    return d;
  }
}

// Exponent e of the power of two 2^-e that the half table is scaled by; codewords that are not finite
// have no say.
template <class E>
__device__ inline int table_exponent(const float* codebook, int states, int* shared) {
  if constexpr (!std::is_same<E, F16>::value) return 0;
  if (threadIdx.x == 0) *shared = 0;
  __syncthreads();
  int top = 0;
  for (int i = threadIdx.x; i < states; i += blockDim.x) {
    const int e = __float_as_uint(codebook[i]) >> 23 & 0xff;
    if (e < 255) top = max(top, e);
  }
  for (int d = 32; d >= 1; d >>= 1) top = max(top, __shfl_xor(top, d, 64));
  if ((threadIdx.x & 63) == 0) atomicMax(shared, top);
  __syncthreads();
  const int e = *shared - 127 - 13;
  return max(e, -126);
}

// What a step of a wave reads.
template <class E, int F, int RT, int NT, int K>
struct CodeStep {
  using T = typename TileOf<E>::T;
  using V = typename T::V;
  using X = XTile<E, F, NT>;
  static constexpr int kKept = Place<E, F>::kKept;
  static constexpr int kParts = std::is_same<E, F32>::value ? 3 : 2;
  static constexpr int kShare = K <= 2 ? 8 : 4;  // states read from one 32-bit window: n + K (kShare - 1) <= 29
  X x;
  unsigned w[RT][K + 1];
  float scale[RT];

  // co, so: a lane's offsets in the rows' codes and scales. With TAIL some of the step's folds are not there.
  template <bool TAIL>
  __device__ void load(const CodeArgs& a, const Place<E, F>& pl, int s, const unsigned* __restrict__ code,
                       const unsigned (&co)[RT], const float* __restrict__ scales, const unsigned (&so)[RT],
                       const typename X::Rows& rows) {
    const int block = s * F + pl.fold;
    const bool in = !TAIL || block * 128 < a.tile.cols;
    int chain = divide(block, a.reciprocal);
    const unsigned at = chain * a.words + (block - chain * a.per_chain) * (4 * K);
    if (TAIL) chain = min(chain, a.chains - 1);
    const bool more = a.n > K;  // the last of the K + 1 words is there
#pragma unroll
    for (int t = 0; t < RT; ++t) {
#pragma unroll
      for (int i = 0; i <= K; ++i) w[t][i] = in && (i < K || more) ? code[co[t] + at + i] : 0u;
      scale[t] = a.scales != nullptr ? scales[so[t] + chain] : 1.0f;
    }
    x.template load<TAIL>(a.tile, rows, s);
  }

  __device__ void add(const Place<E, F>& pl, char* lds, const char* table, int shift, unsigned mask,
                      float (&acc)[RT][NT][kKept]) const {
    x.put(lds);
    V xo[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int j = 0; j < 4; ++j) xo[n][j] = X::get(lds, pl, n, 4 * pl.g + j);
    X::in_order();
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      f32x4 d[NT];
#pragma unroll
      for (int n = 0; n < NT; ++n) d[n] = f32x4{0, 0, 0, 0};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        unsigned e[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int p = K * (8 * j + i / kShare * kShare), q = p / 32, r = p % 32;
          const unsigned window = r == 0 ? w[t][q] : __builtin_amdgcn_alignbit(w[t][q], w[t][q + 1], 32 - r);
          e[i] = *reinterpret_cast<const unsigned*>(table + (window >> (shift - K * (i % kShare)) & mask));
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) d[n] = add_products<T, kParts>(e, xo[n][j], d[n]);
      }
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int u = 0; u < kKept; ++u) acc[t][n][u] = fmaf(scale[t], pl.kept(d[n], u), acc[t][n][u]);
    }
  }
};

// F folds, RT tiles of rows and NT tiles of tokens a wave, K bits a step.
template <class E, int F, int RT, int NT, int K>
__global__ void __launch_bounds__(64 * kMaxWaves)
k_code_tiles(const CodeArgs a) {
  using Pl = Place<E, F>;
  constexpr int kRows = Pl::kRows, kKept = Pl::kKept;
  extern __shared__ __attribute__((aligned(16))) char lds[];
  const int states = 1 << a.n;
  const Pl pl;
  char* mine = lds + pl.wave * NT * kXBytes;
  char* table = lds + pl.waves * NT * kXBytes;
  const int top = table_exponent<E>(a.codebook, states, reinterpret_cast<int*>(lds));
  const float down = ldexpf(1.0f, -top), up = ldexpf(1.0f, top);
  for (int i = threadIdx.x; i < states; i += blockDim.x)
    reinterpret_cast<unsigned*>(table)[i] = Codeword<E>::entry(a.codebook[i], down);
  __syncthreads();

  const int kw = a.tile.kw, ki = pl.wave % kw, ri = pl.wave / kw, rw = pl.waves / kw;
  const int whole = a.tile.cols / (F * 128), steps = whole + (whole * (F * 128) < a.tile.whole8() ? 1 : 0);
  const long long rows = a.tile.rows, units = (rows + RT * kRows - 1) / (RT * kRows);  // of rows, one for a wave
  const long long m0 = (long long)blockIdx.y * (NT * Pl::kTokens);
  const XRows<E, F, NT> xrows(a.tile, m0);
  const unsigned mask = (unsigned)(states - 1) << 2;
  const int shift = 30 - a.n;  // a state at the top of a window as the byte offset of its codeword

  for (long long ub = (long long)blockIdx.x * rw; ub < units; ub += (long long)gridDim.x * rw) {
    const long long row0 = (ub + ri) * (RT * kRows);
    // offsets from the wave's first row fit 32 bits; rows behind the last repeat it
    const long long base = row0 < rows ? row0 : rows - 1;
    const int last = (int)(rows - 1 - base < RT * kRows ? rows - 1 - base : RT * kRows);
    const unsigned* __restrict__ code = a.code + base * a.chains * a.words;
    const float* __restrict__ scales = a.scales + base * a.chains;
    unsigned co[RT], so[RT];
    float acc[RT][NT][kKept] = {};
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      so[t] = (unsigned)(min(t * kRows + pl.row(), last) * a.chains);
      co[t] = so[t] * a.words + K * pl.g;
    }
    CodeStep<E, F, RT, NT, K> one, two;
    auto load = [&](auto& step, int s) {
      if (s < whole)
        step.template load<false>(a, pl, s, code, co, scales, so, xrows);
      else
        step.template load<true>(a, pl, s, code, co, scales, so, xrows);
    };
    if (ki < steps) load(one, ki);
    for (int s = ki; s < steps; s += 2 * kw) {
      if (s + kw < steps) load(two, s + kw);
      one.add(pl, mine, table, shift, mask, acc);
      if (s + 2 * kw < steps) load(one, s + 2 * kw);
      if (s + kw < steps) two.add(pl, mine, table, shift, mask, acc);
    }
    if constexpr (std::is_same<E, F16>::value) {
#pragma unroll
      for (int t = 0; t < RT; ++t)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int u = 0; u < kKept; ++u) acc[t][n][u] *= up;
    }
    join<E, F, RT, NT>(pl, a.tile, acc, ub, m0, lds, [](long long, const typename E::T*) { return 0.0f; });
  }
}

}  // namespace
}  // namespace bcjr
