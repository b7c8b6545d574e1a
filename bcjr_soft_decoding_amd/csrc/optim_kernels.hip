// AdamW over a list of tensors in few launches, moments in fp32 or in 8 bits (include/bcjr.h).
// A pass reads and writes every element once and is bound by memory; the arithmetic, fp64 moments and
// their rounding included, hides behind it.
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

__device__ inline unsigned dither_bits(long long at, unsigned key) {
  return mix((unsigned)at * 0x9E3779B1u + (unsigned)((unsigned long long)at >> 32) * 0x85EBCA6Bu + key);
}

__device__ inline float new_param(float p, float m, float r, const Hyper& h) {
  const float by = m / fmaf(r, h.root2, h.eps);
  return fmaf(-h.rate, by, fmaf(-h.decay, p, p));
}

// floor(log2 |x|) of a finite x from the upper half of its bits, far below any other for zero and for
// what is not finite. (No x is a subnormal double but by betas below 2^-800.)
__device__ inline int exponent(int hi) {
  const int e = (hi >> 20) & 0x7ff;
  return e == 0 || e == 0x7ff ? -2000 : e - 1023;
}

// One e4m3 code: u floor(|y| / u + d) with y = x 2^(127 - b), from the upper half of x's bits. Scaling by
// a power of two leaves the 20 upper bits of the mantissa as they are: 3 of the code's and 17 behind
// them. d = (2 h + 1) / 2^17 has no more bits than that, so the sum's floor is that of the truncated
// value, an addition and a shift whose carry goes on into the exponent. Below 2^-6 the code has
// no leading one: there the mantissa with its leading one is shifted to the fixed spacing 2^-9.
__device__ inline unsigned e4m3(int hi, int b, unsigned h16, bool at_least_one) {
  const int bits = hi & 0x7fffffff, e = (bits >> 20) - 1023 - (b - 127);  // exponent of y
  const int d = (int)(2 * h16 + 1);
  const int normal = ((bits + d) >> 17) - ((1023 + b - 127 - 7) << 3);
  const int down = min(-6 - e, 31);
  const int low = ((((bits & 0xfffff) | 0x100000) >> max(down, 0)) + d) >> 17;
  int code = down > 0 ? low : normal;
  if (at_least_one) code = max(code, 1);
  if (bits < 0x100000) code = 0;                  // zero
  if (bits >= 0x7ff00000) return 0x7f;            // not finite
  return (unsigned)code | ((unsigned)hi >> 24 & 0x80u);
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
  return sqrt(h.beta2 * rr + h.rest2 * gg);
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
    int hm[kQuad] = {}, hs[kQuad] = {}, em = -2000, es = -2000;
    if (there > 0) {
      decode4(mc, bm, m);
      decode4(sc, bs, s);
#pragma unroll
      for (int j = 0; j < kQuad; ++j) {
        const double mj = first_moment(m[j], g[j], h), rj = second_root(s[j], g[j], h);
        p[j] = new_param(p[j], (float)mj, (float)rj, h);
        hm[j] = j < there ? __double2hiint(mj) : 0;
        hs[j] = j < there ? __double2hiint(rj) : 0;
        em = max(em, exponent(hm[j]));
        es = max(es, exponent(hs[j]));
      }
    }
    em = max8(em);
    es = max8(es);
    bm = em == -2000 ? 0 : min(max(em + 120, 0), 254);
    bs = es == -2000 ? 0 : min(max(es + 120, 0), 254);
    if (there <= 0) return;
    mc = sc = 0;
#pragma unroll
    for (int j = 0; j < kQuad; ++j) {
      const unsigned bits = dither_bits(at + j, h.key);
      mc |= e4m3(hm[j], bm, bits & 0xffff, false) << (8 * j);
      sc |= e4m3(hs[j], bs, bits >> 16, true) << (8 * j);
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
