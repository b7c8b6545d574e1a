// AdamW over a list of tensors in few launches, moments in fp32 or in 8 bits (include/bcjr.h).
// A pass reads and writes every element once and is bound by memory; the arithmetic, fp64 moments and
// their rounding included, hides behind it: 20M bf16 parameters with fp32 moments take 87 us, 168M fp32 ones with 8-bit
// moments 551 us, both 4.9 TB/s (a large copy's rate; the VALU is busy for 0.47 ms of the latter), and 0.5M 5.6 us.
#include <hip/hip_runtime.h>

#include <math.h>

#include "internal.h"
#include "ops.h"
#include "ops_device.h"

namespace bcjr {
namespace {

constexpr int kThreads = 256;
constexpr int kQuad = 4;                          // neighbouring elements of a thread
constexpr int kRound = kThreads * kQuad;          // elements of a block at a time, a multiple of 32
constexpr int kRounds = 2;                        // rounds whose loads are in flight together
constexpr int kChunk = kRound * kRounds;          // elements of a block
constexpr int kTensors = 96;                      // tensors of a launch: their table fits the 4 KiB of kernel arguments

struct TensorTable {
  void* param[kTensors];
  const void* grad[kTensors];
  long long numel[kTensors];
  long long first[kTensors];   // place of the tensor's first element in the moments
  unsigned chunk0[kTensors];   // block of the launch its first chunk is
  int count;
};

struct Hyper {
  double beta1, beta2, rest1, rest2;  // rest = 1 - beta
  float decay, rate, root2, eps;      // lr weight_decay, lr / (1 - beta1^t), 1 / sqrt(1 - beta2^t)
  unsigned key;                       // of the dither
};

// Multiply-xorshift mix; the multipliers are the odd 32-bit fractions of sqrt(2) and sqrt(3).
__host__ __device__ inline unsigned mix(unsigned x) {
  x ^= x >> 16;
  x *= 0x6A09E667u;
  x ^= x >> 15;
  x *= 0xBB67AE85u;
  return x ^ (x >> 16);
}

// What the dither of element `at` mixes; that of the next element is kDitherStep more (at is a multiple of 4, so four of
// them have the same upper half).
constexpr unsigned kDitherStep = 0x9E3779B1u;
__device__ inline unsigned dither_seed(long long at, unsigned key) {
  return (unsigned)at * kDitherStep + (unsigned)((unsigned long long)at >> 32) * 0x85EBCA6Bu + key;
}

__device__ inline float new_param(float p, float m, float r, const Hyper& h) {
  const float by = m / fmaf(r, h.root2, h.eps);
  return fmaf(-h.rate, by, fmaf(-h.decay, p, p));
}

// A moment that is not finite, from the upper half of its bits.
constexpr int kNotFinite = 0x7ff00000;

// Byte b of a block whose largest finite magnitude has these upper bits: its exponent less 7, in 0 .. 254. (No moment is
// a subnormal double but by betas below 2^-800; they count as zero.)
__device__ inline int block_exponent(int top) {
  return top < 0x100000 ? 0 : min(max((top >> 20) - 1023 + 120, 0), 254);
}

// One e4m3 code: u floor(|y| / u + d) with y = x 2^(127 - b), from the upper half of x's bits. Scaling by
// a power of two leaves the 20 upper bits of the mantissa as they are: 3 of the code's and 17 behind
// them. d = (2 h + 1) / 2^17 has no more bits than that, so the sum's floor n is that of the truncated
// value, an addition and a shift. With e the exponent of y held to at least -6, where the mantissa is shifted to the
// fixed spacing 2^-9, the code whose exponent field is e + 7 and whose mantissa is n - 8 is the number 8 (e + 6) + n, also
// where n < 8 (subnormal) and where n = 16 (the next binade). Zero is shifted to nothing.
__device__ inline unsigned e4m3(int bits, int b, unsigned d) {
  const int e6 = (bits >> 20) - (1023 + b - 127 - 6), held = max(e6, 0), down = min(held - e6, 31);
  const unsigned n = ((((unsigned)bits & 0xfffffu) | 0x100000u) >> down) + d;
  return ((unsigned)held << 3) + (n >> 17);
}

// sqrt(v) rounded to nearest for v = 0 or a normal number far from the ends (squares of fp32 numbers): two steps of
// Goldschmidt's iteration and two corrections by the residual, without the scaling that the general function needs.
// Inf gives NaN, which a moment that is not finite becomes anyway.
__device__ inline double root(double v) {
  const double y = __builtin_amdgcn_rsq(v);
  double s = v * y, h = 0.5 * y;
  const double r = fma(-h, s, 0.5);
  s = fma(s, r, s);
  h = fma(h, r, h);
  s = fma(fma(-s, s, v), h, s);
  s = fma(fma(-s, s, v), h, s);
  return v == 0.0 ? 0.0 : s;
}

// beta1 m + (1 - beta1) g and sqrt(beta2 r^2 + (1 - beta2) g^2), each product and the sum rounded by
// itself (the squares are exact): old codes and 16-bit gradients have so few bits that the exact
// value often lies right at a code's border, and a fused operation would fall on its other side.
__device__ inline double first_moment(double m, double g, const Hyper& h) {
#pragma clang fp contract(off)
  return h.beta1 * m + h.rest1 * g;
}
__device__ inline double second_root(double r, double g, const Hyper& h) {
#pragma clang fp contract(off)
  const double rr = r * r, gg = g * g;
  return root(h.beta2 * rr + h.rest2 * gg);
}

// Four elements from e on: one wide load where all of them are there and the tensor is aligned.
template <class E>
__device__ inline void load4(const typename E::T* p, int there, bool wide, float out[kQuad]) {
  typedef typename E::T V __attribute__((ext_vector_type(4)));
  if (there == kQuad && wide) {
    const V v = *reinterpret_cast<const V*>(p);
#pragma unroll
    for (int j = 0; j < kQuad; ++j) out[j] = (float)v[j];
  } else {
#pragma unroll
    for (int j = 0; j < kQuad; ++j) out[j] = j < there ? E::load(p + j) : 0.0f;
  }
}
template <class E>
__device__ inline void store4(typename E::T* p, int there, bool wide, const float in[kQuad]) {
  typedef typename E::T V __attribute__((ext_vector_type(4)));
  if (there == kQuad && wide) {
    V v;
#pragma unroll
    for (int j = 0; j < kQuad; ++j) v[j] = (typename E::T)in[j];
    *reinterpret_cast<V*>(p) = v;
  } else {
#pragma unroll
    for (int j = 0; j < kQuad; ++j)
      if (j < there) E::store(p + j, in[j]);
  }
}

// Four codes as numbers times 2^(b - 127), exact in fp32 (conversion in hardware, OCP e4m3).
__device__ inline void decode4(unsigned codes, int b, float out[kQuad]) {
  const float s = ldexpf(1.0f, b - 127);
  const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)codes, false);
  const auto hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)codes, true);
  out[0] = lo[0] * s;
  out[1] = lo[1] * s;
  out[2] = hi[0] * s;
  out[3] = hi[1] * s;
}

// Maximum over the 8 lanes that hold a block of 32: within pairs, fours, and the half row mirrored.
__device__ inline int max8(int v) {
  v = max(v, __builtin_amdgcn_update_dpp(0, v, 0xB1, 0xf, 0xf, true));   // quad_perm 1 0 3 2
  v = max(v, __builtin_amdgcn_update_dpp(0, v, 0x4E, 0xf, 0xf, true));   // quad_perm 2 3 0 1
  return max(v, __builtin_amdgcn_update_dpp(0, v, 0x141, 0xf, 0xf, true));  // row_half_mirror
}

// Elements e0 .. e0 + 3 of a tensor, `there` of them before its end (0: the lane only takes part in its
// block's maximum).
template <class P, class G, int BITS>
struct Quad {
  float p[kQuad], g[kQuad], m[kQuad], s[kQuad];  // s: v, or r with 8 bits
  unsigned mc, sc;
  int there;
  bool wide_p, wide_g;

  __device__ void load(const typename P::T* pp, const typename G::T* gg, const void* avg, const void* sq,
                       const uint8_t* avg_scale, const uint8_t* sq_scale, long long at) {
    if (there <= 0) return;
    load4<P>(pp, there, wide_p, p);
    load4<G>(gg, there, wide_g, g);
    if constexpr (BITS == 32) {
      load4<F32>(static_cast<const float*>(avg) + at, kQuad, true, m);
      load4<F32>(static_cast<const float*>(sq) + at, kQuad, true, s);
    } else {
      mc = *reinterpret_cast<const unsigned*>(static_cast<const uint8_t*>(avg) + at);
      sc = *reinterpret_cast<const unsigned*>(static_cast<const uint8_t*>(sq) + at);
      bm = avg_scale[at / kMomentBlock];
      bs = sq_scale[at / kMomentBlock];
    }
  }
  int bm, bs;

  __device__ void step32(const Hyper& h) {
#pragma unroll
    for (int j = 0; j < kQuad; ++j) {
      m[j] = fmaf((float)h.beta1, m[j], (float)h.rest1 * g[j]);
      s[j] = fmaf((float)h.beta2, s[j], (float)h.rest2 * g[j] * g[j]);
      p[j] = new_param(p[j], m[j], sqrtf(s[j]), h);
    }
  }

  __device__ void step8(const Hyper& h, long long at) {
    int hm[kQuad] = {}, hs[kQuad] = {}, tm = 0, ts = 0;  // upper halves of the moments, the largest magnitudes'
    if (there > 0) {
      decode4(mc, bm, m);
      decode4(sc, bs, s);
#pragma unroll
      for (int j = 0; j < kQuad; ++j) {
        const double mj = first_moment(m[j], g[j], h), rj = second_root(s[j], g[j], h);
        p[j] = new_param(p[j], (float)mj, (float)rj, h);
        hm[j] = j < there ? __double2hiint(mj) : 0;
        hs[j] = j < there ? __double2hiint(rj) & 0x7fffffff : 0;  // a NaN may have a sign
        tm = max(tm, hm[j] & 0x7fffffff);
        ts = max(ts, hs[j]);
      }
    }
    // Seldom: what is not finite has no say in the block's exponent, counts as zero and becomes a NaN in the end.
    const bool odd = max(tm, ts) >= kNotFinite;
    unsigned nm = 0, ns = 0;
    if (odd) {
      tm = ts = 0;
#pragma unroll
      for (int j = 0; j < kQuad; ++j) {
        if ((hm[j] & 0x7fffffff) >= kNotFinite) hm[j] = 0, nm |= 0x7fu << (8 * j);
        if (hs[j] >= kNotFinite) hs[j] = 0, ns |= 0x7fu << (8 * j);
        tm = max(tm, hm[j] & 0x7fffffff);
        ts = max(ts, hs[j]);
      }
    }
    bm = block_exponent(max8(tm));
    bs = block_exponent(max8(ts));
    if (there <= 0) return;
    const unsigned seed = dither_seed(at, h.key);
    mc = nm;
    sc = ns;
#pragma unroll
    for (int j = 0; j < kQuad; ++j) {
      const unsigned bits = mix(seed + j * kDitherStep);
      const unsigned cm = e4m3(hm[j] & 0x7fffffff, bm, (bits << 1 & 0x1fffeu) | 1u) | ((unsigned)hm[j] >> 24 & 0x80u);
      const unsigned cs = max(e4m3(hs[j], bs, (bits >> 15 & 0x1fffeu) | 1u), min((unsigned)hs[j], 1u));  // 0 only for 0
      mc |= cm << (8 * j);
      sc |= cs << (8 * j);
    }
  }

  __device__ void store(typename P::T* pp, void* avg, void* sq, uint8_t* avg_scale, uint8_t* sq_scale,
                        long long at) const {
    if (there <= 0) return;
    store4<P>(pp, there, wide_p, p);
    if constexpr (BITS == 32) {
      store4<F32>(static_cast<float*>(avg) + at, there, true, m);
      store4<F32>(static_cast<float*>(sq) + at, there, true, s);
    } else {
      uint8_t *a = static_cast<uint8_t*>(avg) + at, *b = static_cast<uint8_t*>(sq) + at;
      if (there == kQuad) {
        *reinterpret_cast<unsigned*>(a) = mc;
        *reinterpret_cast<unsigned*>(b) = sc;
      } else {
#pragma unroll
        for (int j = 0; j < kQuad; ++j)
          if (j < there) {
            a[j] = (uint8_t)(mc >> (8 * j));
            b[j] = (uint8_t)(sc >> (8 * j));
          }
      }
      if ((threadIdx.x & 7) == 0) {
        avg_scale[at / kMomentBlock] = (uint8_t)bm;
        sq_scale[at / kMomentBlock] = (uint8_t)bs;
      }
    }
  }
};

template <class P, class G, int BITS>
__global__ void __launch_bounds__(kThreads)
k_adamw(const TensorTable t, const Hyper h, void* avg, void* sq, uint8_t* avg_scale, uint8_t* sq_scale) {
  // the block's tensor: how many begin at or before it, each lane looking at one or two
  const int lane = threadIdx.x & 63;
  int i = __popcll(__ballot(lane < t.count && t.chunk0[lane] <= blockIdx.x));
  if (t.count > 64) i += __popcll(__ballot(lane + 64 < t.count && t.chunk0[min(lane + 64, kTensors - 1)] <= blockIdx.x));
  i = __builtin_amdgcn_readfirstlane(i - 1);
  const long long n = t.numel[i], e0 = (long long)(blockIdx.x - t.chunk0[i]) * kChunk + threadIdx.x * kQuad;
  typename P::T* p = static_cast<typename P::T*>(t.param[i]) + e0;
  const typename G::T* g = static_cast<const typename G::T*>(t.grad[i]) + e0;
  const long long s0 = t.first[i] + e0;
  Quad<P, G, BITS> q[kRounds];
#pragma unroll
  for (int k = 0; k < kRounds; ++k) {
    const long long left = n - e0 - k * kRound;
    q[k].there = left >= kQuad ? kQuad : left > 0 ? (int)left : 0;
    q[k].wide_p = ((uintptr_t)t.param[i] % (kQuad * sizeof(typename P::T))) == 0;
    q[k].wide_g = ((uintptr_t)t.grad[i] % (kQuad * sizeof(typename G::T))) == 0;
    q[k].load(p + k * kRound, g + k * kRound, avg, sq, avg_scale, sq_scale, s0 + k * kRound);
  }
#pragma unroll
  for (int k = 0; k < kRounds; ++k) {
    if constexpr (BITS == 32)
      q[k].step32(h);
    else
      q[k].step8(h, s0 + k * kRound);
    q[k].store(p + k * kRound, avg, sq, avg_scale, sq_scale, s0 + k * kRound);
  }
}

template <class P, class G>
void launch_table(const TensorTable& t, unsigned blocks, const Hyper& h, const AdamwState& s, void* stream) {
  if (s.bits == 32)
    hipLaunchKernelGGL((k_adamw<P, G, 32>), dim3(blocks), dim3(kThreads), 0, static_cast<hipStream_t>(stream), t, h,
                       s.avg, s.sq, s.avg_scale, s.sq_scale);
  else
    hipLaunchKernelGGL((k_adamw<P, G, 8>), dim3(blocks), dim3(kThreads), 0, static_cast<hipStream_t>(stream), t, h,
                       s.avg, s.sq, s.avg_scale, s.sq_scale);
}

}  // namespace

int launch_adamw(const bcjr_adamw_tensor* tensors, int64_t count, int param_type, int grad_type,
                 const bcjr_adamw& hyper, const AdamwState& state, void* stream) {
  Hyper h;
  h.beta1 = hyper.beta1;
  h.beta2 = hyper.beta2;
  h.rest1 = 1.0 - hyper.beta1;
  h.rest2 = 1.0 - hyper.beta2;
  h.decay = (float)(hyper.lr * hyper.weight_decay);
  h.rate = (float)(hyper.lr / (1.0 - pow(hyper.beta1, (double)hyper.step)));
  h.root2 = (float)(1.0 / sqrt(1.0 - pow(hyper.beta2, (double)hyper.step)));
  h.eps = (float)hyper.eps;
  h.key = mix(mix((unsigned)hyper.seed) + (unsigned)hyper.step);
  TensorTable t;
  t.count = 0;
  // A launch holds at most 2^32 - 1 threads: what would exceed that, within a tensor too, is left to
  // the next one.
  const int64_t most = ((int64_t)1 << 32) / kThreads - 1;
  const int psize = param_type == BCJR_F32 ? 4 : 2, gsize = grad_type == BCJR_F32 ? 4 : 2;
  int64_t first = 0, chunks = 0;
  auto flush = [&]() -> int {
    if (t.count == 0) return 0;
    with_type(param_type, [&](auto p) {
      return with_type(grad_type, [&](auto g) {
        launch_table<decltype(p), decltype(g)>(t, (unsigned)chunks, h, state, stream);
        return 0;
      });
    });
    t.count = 0;
    chunks = 0;
    return (int)hipGetLastError();
  };
  for (int64_t i = 0; i < count; ++i) {
    const int64_t numel = tensors[i].numel;
    for (int64_t done = 0; done < numel;) {
      if (t.count == kTensors || chunks == most) {
        if (const int e = flush()) return e;
      }
      const int64_t left = numel - done, room = (most - chunks) * kChunk, take = left < room ? left : room;
      t.param[t.count] = static_cast<char*>(tensors[i].param) + done * psize;
      t.grad[t.count] = static_cast<const char*>(tensors[i].grad) + done * gsize;
      t.numel[t.count] = take;
      t.first[t.count] = first + done;
      t.chunk0[t.count++] = (unsigned)chunks;
      chunks += (take + kChunk - 1) / kChunk;
      done += take;
    }
    first += moment_numel(numel);
  }
  return flush();
}

}  // namespace bcjr
