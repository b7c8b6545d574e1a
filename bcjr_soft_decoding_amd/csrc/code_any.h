// Products with trellis-coded weights whose chains do not cut into blocks of 128 columns, or whose table does not
// fit LDS as tiles need it (code_mfma.h has the others). A lane decodes its 32 columns eight at a time: from one 64-bit
// window of its chain, and from the start of the next chain where that begins among the eight (L >= 8). Chains and so
// scales may change anywhere in a sum, so the scale is multiplied into the weight, in fp32, before it is taken apart
// into bfloat16 parts. Halves are multiplied as two bfloat16 parts: scale times codeword may leave their range.
// Bound by unpacking and by the table's reads: 8192 x 8200 in chains of 100 with 16 tokens takes 82 us; with S = 2^16,
// whose table stays in memory, 8192 x 8192 takes 271 us.
#pragma once
#include "code_mfma.h"

namespace bcjr {
namespace {

// State at step t of a chain.
__device__ inline unsigned state_of(const unsigned* chain, int n, int k, long long t, int words) {
  const long long p = k * t;
  const int w = (int)(p >> 5);
  const unsigned long long x = (unsigned long long)chain[w] << 32 | (w + 1 < words ? chain[w + 1] : 0u);
  return (unsigned)(x << (p & 31) >> (64 - n));
}

template <class E, int F>
struct AnyStep {
  using T = typename TileOf<E>::T;
  using V = typename T::V;
  using X = XTile<E, F, 1>;
  static constexpr int kKept = Place<E, F>::kKept, kWords = Codeword<typename std::conditional<T::kParts == 3, F32, BF16>::type>::kWords;
  X x;
  unsigned long long window[4], next[4];  // of eight columns each; the next chain's beginning
  float scale[4], next_scale[4];
  int cross[4];  // of the eight, the first that is of the next chain, or 8

  // code, scales: of the lane's row; left: words from there to the end of all codes.
  template <bool TAIL>
  __device__ void load(const CodeArgs& a, const Place<E, F>& pl, int s, const unsigned* code, long long left,
                       const float* scales, const typename X::Rows& rows) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int col = (s * F + pl.fold) * 128 + 32 * pl.g + 8 * j;
      window[j] = next[j] = 0;
      scale[j] = next_scale[j] = 0.0f;
      cross[j] = 8;
      if (TAIL && col >= a.tile.whole8()) continue;
      const int chain = divide(col, a.reciprocal), t = col - chain * a.L, p = a.k * t, off = p & 31;
      const unsigned at = chain * a.words + (p >> 5);
      const unsigned w0 = code[at], w1 = at + 1 < left ? code[at + 1] : 0u, w2 = at + 2 < left ? code[at + 2] : 0u;
      window[j] = ((unsigned long long)w0 << 32 | w1) << off | (unsigned long long)w2 << off >> 32;
      scale[j] = a.scales != nullptr ? scales[chain] : 1.0f;
      if (t + 8 > a.L) {
        cross[j] = a.L - t;
        const unsigned b = (chain + 1) * a.words;
        next[j] = (unsigned long long)code[b] << 32 | (b + 1 < left ? code[b + 1] : 0u);
        next_scale[j] = a.scales != nullptr ? scales[chain + 1] : 1.0f;
      }
    }
    x.template load<TAIL>(a.tile, rows, s);
  }

  // Sums of the step; table: codewords, in LDS or in memory.
  template <class Table>
  __device__ f32x4 sums(const CodeArgs& a, const Place<E, F>& pl, char* lds, Table table) const {
    x.put(lds);
    f32x4 d = {0, 0, 0, 0};
    const int down = 64 - a.n;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      unsigned st[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) st[i] = (unsigned)(window[j] << (a.k * i) >> down);
      float sc[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) sc[i] = scale[j];
      if (cross[j] < 8) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (i >= cross[j]) {
            st[i] = (unsigned)(next[j] << (a.k * (i - cross[j])) >> down);
            sc[i] = next_scale[j];
          }
      }
      const u32x4 v = __builtin_bit_cast(u32x4, X::get(lds, pl, 0, 4 * pl.g + j));
      unsigned e[8 * kWords], twice[8 * kWords];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        Codeword<typename std::conditional<T::kParts == 3, F32, BF16>::type>::write(e + i * kWords, table[st[i]] * sc[i], 1.0f);
#pragma unroll
        for (int k = 0; k < kWords; ++k)
          twice[i * kWords + k] = __builtin_amdgcn_perm(v[i / 2], v[i / 2], i % 2 ? 0x03020302 : 0x01000100);
      }
#pragma unroll
      for (int o = 0; o < 2 * kWords; ++o) {
        const unsigned *u = e + 4 * o, *w = twice + 4 * o;
        d = T::mfma(__builtin_bit_cast(V, u32x4{w[0], w[1], w[2], w[3]}), __builtin_bit_cast(V, u32x4{u[0], u[1], u[2], u[3]}), d);
      }
    }
    X::in_order();
    return d;
  }
};

// One row tile and one tile of tokens a wave. IN_LDS: codewords in LDS at offset 0, else read from memory.
template <class E, int F, bool IN_LDS>
__global__ void __launch_bounds__(64 * kMaxWaves)
k_code_any(const CodeArgs a) {
  using Pl = Place<E, F>;
  constexpr int kRows = Pl::kRows, kKept = Pl::kKept;
  extern __shared__ __attribute__((aligned(16))) char lds[];
  const int states = 1 << a.n;
  const Pl pl;
  char* xs = lds + (IN_LDS ? max(states * 4, 64) : 0);
  char* mine = xs + pl.wave * kXBytes;
  const float* table = IN_LDS ? reinterpret_cast<const float*>(lds) : a.codebook;
  const int kw = a.tile.kw, ki = pl.wave % kw, ri = pl.wave / kw, rw = pl.waves / kw;
  const int whole = a.tile.cols / (F * 128), steps = whole + (whole * (F * 128) < a.tile.whole8() ? 1 : 0);
  const long long rows = a.tile.rows, units = (rows + kRows - 1) / kRows;  // of rows, one for a wave
  const long long m0 = (long long)blockIdx.y * Pl::kTokens;
  const XRows<E, F, 1> xrows(a.tile, m0);
  const long long row_words = (long long)a.chains * a.words;
  if (IN_LDS) {
    each_codeword(a.codebook, states, [&](int i, float c) { reinterpret_cast<float*>(lds)[i] = c; });
    __syncthreads();
  }
  for (long long ub = (long long)blockIdx.x * rw; ub < units; ub += (long long)gridDim.x * rw) {
    // rows behind the last repeat it
    long long row = (ub + ri) * kRows + pl.row();
    row = row < rows ? row : rows - 1;
    const unsigned* code = a.code + row * row_words;
    const float* scales = a.scales + row * a.chains;
    const long long left = (rows - row) * row_words;
    float acc[1][1][kKept] = {};
    AnyStep<E, F> step;
    auto load = [&](int s) {
      if (s < whole)
        step.template load<false>(a, pl, s, code, left, scales, xrows);
      else
        step.template load<true>(a, pl, s, code, left, scales, xrows);
    };
    for (int s = ki; s < steps; s += kw) {
      load(s);
      const f32x4 d = IN_LDS ? step.sums(a, pl, mine, reinterpret_cast<const float*>(lds)) : step.sums(a, pl, mine, table);
#pragma unroll
      for (int u = 0; u < kKept; ++u) acc[0][0][u] += pl.kept(d, u);
    }
    join<E, F, 1, 1>(pl, a.tile, acc, ub, m0, xs, [&](long long r, const typename E::T* x) {
      float sum = 0.0f;
      for (int c = a.tile.whole8(); c < a.tile.cols; ++c) {
        const int chain = divide(c, a.reciprocal);
        const float w = table[state_of(a.code + (r * a.chains + chain) * a.words, a.n, a.k, c - chain * a.L, a.words)];
        sum = fmaf(a.scales != nullptr ? a.scales[r * a.chains + chain] * w : w, E::load(x + c), sum);
      }
      return sum;
    });
  }
}

}  // namespace
}  // namespace bcjr
