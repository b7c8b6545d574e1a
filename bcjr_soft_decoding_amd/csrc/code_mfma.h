// Products of a few tokens with trellis-coded weights on the matrix cores (the tile: tiles.h).
//
// A lane decodes 32 neighbouring weights of a chain: they begin at a whole word of its code, whatever
// k, and lie in k + 1 words. A window of the bit string is two words shifted into one, which holds the
// states of several neighbours; a state is a shift and a mask away, and its codeword one read of a
// table in LDS. For 16-bit x the table holds a codeword as two parts, c = hi + lo to 2^-16 (bfloat16)
// or 2^-21 (half) of c, in the halves of a word (rounding weights to 16 bits alone would cost as much precision
// as rounding the result), and that word goes into the matrix operand as it is: the two parts are
// neighbours in the sum's index, and x is there twice. For fp32 x it holds three bfloat16 parts and a
// zero. Where it is small enough the table goes by windows of two states and gives two neighbours
// in one read: LDS serves 6.7 random 8-byte reads a clock and 8.8 of 4 bytes.
//
// Bound by making the table and by those reads: 8192 x 8192 with 16 tokens (S = 4096) takes 20 us, of which the reads
// are 8, 2048 x 8192 with one token 8 us, most of it before the first product, 512 x 1024 (S = 256) 4 us.
#pragma once
#include "tiles.h"

namespace bcjr {

namespace {

// What the table holds of a codeword: words of two neighbouring terms of the sum.
template <class E>
struct Codeword {  // bfloat16
  static constexpr int kWords = 1;
  static __device__ void write(unsigned* at, float c, float scale) {
    c *= scale;
    const __bf16 hi = (__bf16)c, lo = (__bf16)(c - (float)hi);
    at[0] = (unsigned)__builtin_bit_cast(unsigned short, lo) << 16 | __builtin_bit_cast(unsigned short, hi);
  }
};
template <>
struct Codeword<F16> {  // half
  static constexpr int kWords = 1;
  static __device__ void write(unsigned* at, float c, float scale) {
    c *= scale;
    const _Float16 hi = (_Float16)c, lo = (_Float16)(c - (float)hi);
    at[0] = (unsigned)__builtin_bit_cast(unsigned short, lo) << 16 | __builtin_bit_cast(unsigned short, hi);
  }
};
template <>
struct Codeword<F32> {  // the leading 8 bits, the next 8, the rest
  static constexpr int kWords = 2;
  static __device__ void write(unsigned* at, float c, float scale) {
    c *= scale;
    const unsigned hi = __float_as_uint(c);
    const float left = c - __uint_as_float(hi & 0xffff0000u);
    const unsigned mid = __float_as_uint(left);
    at[0] = __builtin_amdgcn_perm(mid, hi, 0x07060302);
    at[1] = __float_as_uint(left - __uint_as_float(mid & 0xffff0000u)) >> 16;
  }
};

// use(i, load(i)) for the block's share of count items, the loads of U items in flight together.
template <int U, class Load, class Use>
__device__ __forceinline__ void each(unsigned i, unsigned count, Load load, Use use) {
  const unsigned block = blockDim.x;
  for (; i + (U - 1) * block < count; i += U * block) {
    decltype(load(i)) v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) v[u] = load(i + u * block);
#pragma unroll
    for (int u = 0; u < U; ++u) use(i + u * block, v[u]);
  }
  if constexpr (U > 1) each<U / 2>(i, count, load, use);
}

// f(i, c(i)) for the block's share of the codewords, loaded four at a time.
template <class Fn>
__device__ __forceinline__ void each_codeword(const float* codebook, int states, Fn f) {
  if (states < 4) {
    if ((int)threadIdx.x < states) f(threadIdx.x, codebook[threadIdx.x]);
    return;
  }
  using V = typename Loose<float, 4>::V;
  each<4>(threadIdx.x, states / 4u, [&](unsigned i) { return *reinterpret_cast<const V*>(codebook + 4 * i); },
          [&](unsigned i, const V& v) {
#pragma unroll
            for (int j = 0; j < 4; ++j) f(4 * i + j, v[j]);
          });
}

// The table in LDS, at offset 0: [2^n] codewords, or with PAIR [2^(n + K)] of two neighbours' windows.
template <class E, int K, bool PAIR>
struct Table {
  static constexpr int kWords = Codeword<E>::kWords * (PAIR ? 2 : 1);  // of an entry
  static constexpr int kBytes = 4 * kWords, kShift = kWords == 1 ? 2 : kWords == 2 ? 3 : 4;
  typedef unsigned Entry __attribute__((ext_vector_type(kWords)));
  static __host__ __device__ size_t bytes(int n) {
    const size_t b = ((size_t)kBytes << n) << (PAIR ? K : 0);
    return b < 64 ? 64 : b;
  }

  // Makes the table of the codewords times 2^-e and returns e, a usual one where that brings the largest to where a
  // half holds it well, and a chain's sum, which its scale meets only afterwards, is far from an overflow; else the e that
  // brings it to [2^13, 2^14), in a second pass. Codewords that are not finite have no say in it. slots: LDS for a word of
  // each wave, free again afterwards.
  static __device__ __forceinline__ int make(char* lds, int* slots, const float* codebook, int n) {
    constexpr bool half = std::is_same<E, F16>::value;
    constexpr int usual = half ? -10 : 0, least = half ? -4 : -40, most = half ? 5 : 40;  // exponents of the largest
    int top = 0;
    fill(lds, codebook, n, ldexpf(1.0f, -usual), [&](float c) {
      const int bits = __float_as_uint(c) & 0x7fffffff;
      top = max(top, bits < 0x7f800000 ? bits : 0);
    });
    const int e = (top >> 23) - 127;
    // what a wave knows: whether it has seen one that is large enough, and one that is too large
    const int seen = (__any(e >= least) ? 1 : 0) | (__any(e > most) ? 2 : 0);
    if ((threadIdx.x & 63) == 0) slots[threadIdx.x >> 6] = seen;
    __syncthreads();
    int all = 0;
    for (int w = 0; w < kMaxWaves; ++w) all |= slots[w];
    __syncthreads();
    if (all == 1) return usual;
    for (int d = 32; d >= 1; d >>= 1) top = max(top, __shfl_xor(top, d, 64));
    if ((threadIdx.x & 63) == 0) slots[threadIdx.x >> 6] = top;
    __syncthreads();
    for (int w = 0; w < kMaxWaves; ++w) top = max(top, slots[w]);
    __syncthreads();
    const int fit = max((top >> 23) - 127 - 13, -126);
    fill(lds, codebook, n, ldexpf(1.0f, -fit), [](float) {});
    __syncthreads();
    return fit;
  }

  // see(c): every codeword, by one thread or another.
  template <class See>
  static __device__ __forceinline__ void fill(char* lds, const float* codebook, int n, float scale, See see) {
    unsigned* table = reinterpret_cast<unsigned*>(lds);
    if constexpr (!PAIR) {
      each_codeword(codebook, 1 << n, [&](int i, float c) {
        see(c);
        Codeword<E>::write(table + i * kWords, c, scale);
      });
    } else {
      // window i holds the states i >> K and i mod 2^n: those of one first state have neighbouring second ones
      struct Windows {
        float first, second[1 << K];
      };
      const unsigned states = 1u << n;
      each<(K <= 2 ? 4 : 1)>(
          threadIdx.x, states,
          [&](unsigned s) {
            Windows v;
            v.first = codebook[s];
#pragma unroll
            for (int b = 0; b < 1 << K; ++b) v.second[b] = codebook[((s << K) & (states - 1)) + b];
            return v;
          },
          [&](unsigned s, const Windows& v) {
            see(v.first);
#pragma unroll
            for (int b = 0; b < 1 << K; ++b) {
              unsigned* at = table + ((s << K) + b) * kWords;
              Codeword<E>::write(at, v.first, scale);
              Codeword<E>::write(at + Codeword<E>::kWords, v.second[b], scale);
            }
          });
    }
  }
};

// What a step of a wave reads.
template <class E, int F, int RT, int NT, int K, bool PAIR>
struct CodeStep {
  using T = typename TileOf<E>::T;
  using V = typename T::V;
  using X = XTile<E, F, NT>;
  using Tab = Table<E, K, PAIR>;
  static constexpr int kKept = Place<E, F>::kKept;
  static constexpr int kShare = K <= 2 ? 8 : 4;  // states read from one 32-bit window: n + K (kShare - 1) <= 29
  X x;
  unsigned w[RT][K + 1];
  float scale;

  // In memory order: four neighbouring lanes load the K + 1 words each of four chunks of 32 weights, and lane
  // (g, c16) the scale of tile g's row c16. co: a lane's offsets in the rows' codes, so: in the scales. With TAIL some
  // of the step's folds are not there.
  template <bool TAIL>
  __device__ void load(const CodeArgs& a, const Place<E, F>& pl, int s, const unsigned* __restrict__ code,
                       const unsigned (&co)[RT], const float* __restrict__ scales, unsigned so,
                       const typename X::Rows& rows) {
    typedef unsigned Words __attribute__((ext_vector_type(K < 4 ? K + 1 : 4), aligned(4)));
    {
      const int block = s * F + ((threadIdx.x & 63) >> 2) % F, chain = divide(block, a.reciprocal);
      const unsigned at = chain * a.words + (block - chain * a.per_chain) * (4 * K);
      const bool in = !TAIL || block * 128 < a.tile.cols;
      const bool more = a.n > K;  // the last of the K + 1 words is there
#pragma unroll
      for (int t = 0; t < RT; ++t) {
        const unsigned* p = code + co[t] + at;
#pragma unroll
        for (int i = 0; i <= K; ++i) w[t][i] = 0u;
        if (in) {
          if (K < 4 && more) {
            const Words v = *reinterpret_cast<const Words*>(p);
#pragma unroll
            for (int i = 0; i <= K; ++i) w[t][i] = v[i < 4 ? i : 3];
          } else {
#pragma unroll
            for (int i = 0; i < K; ++i) w[t][i] = p[i];
            if (more) w[t][K] = p[K];
          }
        }
      }
    }
    const int chain = divide(s * F + pl.fold, a.reciprocal);
    scale = a.scales == nullptr ? 1.0f : pl.g < RT ? scales[so + (TAIL ? min(chain, a.chains - 1) : chain)] : 0.0f;
    x.template load<TAIL>(a.tile, rows, s);
  }

  // What the products take, from what was loaded: its registers are free for the next step's loads then.
  struct Operands {
    static constexpr int kWords = Codeword<E>::kWords, kOps = 2 * kWords;  // operands of 8 weights
    V x[NT][4][kOps];  // x[i] twice (fp32: four times), for each word of weight i
    unsigned w[RT][K + 1], scale[RT];

    // The words of weights 8 j .. 8 j + 7 of tile t.
    __device__ void gather(int t, int j, const char* table, int shift, unsigned mask, unsigned (&e)[8 * kWords]) const {
      constexpr int kStates = PAIR ? 2 : 1;
#pragma unroll
      for (int i = 0; i < 8; i += kStates) {
        const int p = K * (8 * j + i / kShare * kShare), q = p / 32, r = p % 32;
        const unsigned window = r == 0 ? w[t][q] : __builtin_amdgcn_alignbit(w[t][q], w[t][q + 1], 32 - r);
        const auto v = *reinterpret_cast<const typename Tab::Entry*>(table + (window >> (shift - K * (i % kShare)) & mask));
#pragma unroll
        for (int k = 0; k < Tab::kWords; ++k) e[i * kWords + k] = v[k];
      }
    }

    __device__ void add(const Place<E, F>& pl, const char* table, int shift, unsigned mask, float (&acc)[RT][NT][kKept]) const {
      unsigned e[2][8 * kWords];
      gather(0, 0, table, shift, mask, e[0]);
      f32x4 d[NT];
#pragma unroll
      for (int tj = 0; tj < 4 * RT; ++tj) {  // the next eight weights are asked for before these are used
        const int t = tj / 4, j = tj % 4;
        if (tj + 1 < 4 * RT) gather((tj + 1) / 4, (tj + 1) % 4, table, shift, mask, e[(tj + 1) % 2]);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          if (j == 0) d[n] = f32x4{0, 0, 0, 0};
#pragma unroll
          for (int o = 0; o < kOps; ++o) {
            const unsigned* u = e[tj % 2] + 4 * o;
            d[n] = T::mfma(x[n][j][o], __builtin_bit_cast(V, u32x4{u[0], u[1], u[2], u[3]}), d[n]);
          }
        }
        if (j == 3)
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int u = 0; u < kKept; ++u) acc[t][n][u] = fmaf(__uint_as_float(scale[t]), pl.kept(d[n], u), acc[t][n][u]);
      }
    }
  };

  __device__ void exchange(const Place<E, F>& pl, char* lds, Operands& o) const {
    constexpr int kWords = Operands::kWords, kOps = Operands::kOps;
    x.put(lds);
#pragma unroll
    for (int t = 0; t < RT; ++t)
#pragma unroll
      for (int i = 0; i <= K; ++i) o.w[t][i] = __builtin_amdgcn_ds_bpermute(pl.from(), w[t][i]);
    rows_apart<RT>(__float_as_uint(scale), o.scale);
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const u32x4 v = __builtin_bit_cast(u32x4, X::get(lds, pl, n, 4 * pl.g + j));
        u32x4 twice[kOps];
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
          for (int k = 0; k < kWords; ++k)
            twice[(i * kWords + k) / 4][(i * kWords + k) % 4] = __builtin_amdgcn_perm(v[i / 2], v[i / 2], i % 2 ? 0x03020302 : 0x01000100);
#pragma unroll
        for (int p = 0; p < kOps; ++p) o.x[n][j][p] = __builtin_bit_cast(V, twice[p]);
      }
    X::in_order();
  }
};

// F folds, RT tiles of rows and NT tiles of tokens a wave, K bits a step.
template <class E, int F, int RT, int NT, int K, bool PAIR>
__global__ void __launch_bounds__(64 * kMaxWaves)
k_code_tiles(const CodeArgs a) {
  using Pl = Place<E, F>;
  constexpr int kRows = Pl::kRows, kKept = Pl::kKept;
  extern __shared__ __attribute__((aligned(16))) char lds[];
  const Pl pl;
  using Tab = Table<E, K, PAIR>;
  char* xs = lds + Tab::bytes(a.n);  // the waves' x, behind the table
  char* mine = xs + pl.wave * NT * kXBytes;
  const int kw = a.tile.kw, ki = pl.wave % kw, ri = pl.wave / kw, rw = pl.waves / kw;
  const int whole = a.tile.cols / (F * 128), steps = whole + (whole * (F * 128) < a.tile.whole8() ? 1 : 0);
  const long long rows = a.tile.rows, units = (rows + RT * kRows - 1) / (RT * kRows);  // of rows, one for a wave
  const long long m0 = (long long)blockIdx.y * (NT * Pl::kTokens);
  const XRows<E, F, NT> xrows(a.tile, m0);
  // a state, or two, at the top of a window as the byte offset of its entry
  const int bits = a.n + (PAIR ? K : 0), shift = 32 - Tab::kShift - bits;
  const unsigned mask = ((1u << bits) - 1u) << Tab::kShift;

  using Step = CodeStep<E, F, RT, NT, K, PAIR>;
  Step step;
  const unsigned* __restrict__ code;
  const float* __restrict__ scales;
  unsigned co[RT], so;
  const int lane = threadIdx.x & 63;
  auto load = [&](int s) {
    if (s < whole)
      step.template load<false>(a, pl, s, code, co, scales, so, xrows);
    else
      step.template load<true>(a, pl, s, code, co, scales, so, xrows);
  };
  // A unit's first loads, before the table for the first one: it takes as long as they do.
  auto begin = [&](long long unit) {
    const long long row0 = unit * (RT * kRows);
    // offsets from the wave's first row fit 32 bits; rows behind the last repeat it
    const long long base = row0 < rows ? row0 : rows - 1;
    const int last = (int)(rows - 1 - base < RT * kRows ? rows - 1 - base : RT * kRows);
    code = a.code + base * a.chains * a.words;
    scales = a.scales + base * a.chains;
#pragma unroll
    for (int t = 0; t < RT; ++t) co[t] = (unsigned)(min(t * kRows + (lane >> 2) / F, last) * a.chains * a.words + K * (lane & 3));
    so = (unsigned)(min(min(pl.g, RT - 1) * kRows + pl.row(), last) * a.chains);
    if (ki < steps) load(ki);
  };
  begin((long long)blockIdx.x * rw + ri);
  const float up = ldexpf(1.0f, Tab::make(lds, reinterpret_cast<int*>(xs), a.codebook, a.n));


  for (long long ub = (long long)blockIdx.x * rw; ub < units; ub += (long long)gridDim.x * rw) {
    float acc[RT][NT][kKept] = {};
    for (int s = ki; s < steps; s += kw) {
      typename Step::Operands o;
      step.exchange(pl, mine, o);
      if (s + kw < steps) load(s + kw);
      o.add(pl, lds, shift, mask, acc);
    }
#pragma unroll
    for (int t = 0; t < RT; ++t)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int u = 0; u < kKept; ++u) acc[t][n][u] *= up;
    if (ub + (long long)gridDim.x * rw < units) begin(ub + (long long)gridDim.x * rw + ri);
    join<E, F, RT, NT>(pl, a.tile, acc, ub, m0, xs, [](long long, const typename E::T*) { return 0.0f; });
  }
}

}  // namespace
}  // namespace bcjr
