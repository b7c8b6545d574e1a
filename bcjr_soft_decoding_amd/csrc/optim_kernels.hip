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
constexpr int kPer = 8;                    // elements of a thread
constexpr int kChunk = kThreads * kPer;    // elements of a block, a multiple of the moments' 32
constexpr int kTensors = 96;               // tensors of a launch: their table fits the 4 KiB of kernel arguments

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

// floor(log2 |x|) of a finite x, far below any other for zero; x here is 0 or a normal number.
__device__ inline int exponent(double x) {
  const int e = (__double2hiint(x) >> 20) & 0x7ff;
  return e == 0 ? -2000 : e == 0x7ff ? -2000 : e - 1023;
}
__device__ inline bool finite(double x) { return ((__double2hiint(x) >> 20) & 0x7ff) != 0x7ff; }

// One e4m3 code: u floor(|y| / u + d) for y = x 2^(127 - b), NaN for what is not finite. With e the
// exponent of y held to at least -6, |y| / u = |y| 2^(3 - e) is in [0, 16), and a code whose
// exponent field is e + 7 and whose mantissa is n - 8 is the number 8 (e + 6) + n, also where n < 8
// (subnormal) and where n = 16 (the next binade).
__device__ inline unsigned e4m3(double x, int b, unsigned h16, bool at_least_one) {
  if (!finite(x)) return 0x7f;
  if (x == 0.0) return 0;
  const double y = ldexp(fabs(x), 127 - b);
  const int ey = ilogb(y), e = ey > -6 ? ey : -6;
  int n = (int)(ldexp(y, 3 - e) + ((double)h16 + 0.5) * (1.0 / 65536));
  if (at_least_one && n < 1) n = 1;
  return (unsigned)(8 * (e + 6) + n) | (n > 0 && x < 0 ? 0x80u : 0u);
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

__device__ inline double from_e4m3(unsigned code, int b) {
  const int e = (code >> 3) & 15, n = code & 7;
  const double v = (code & 0x7f) == 0x7f ? (double)NAN : e ? ldexp(8.0 + n, e - 10) : ldexp((double)n, -9);
  return ldexp(code & 0x80 ? -v : v, b - 127);
}

template <class P, class G, int BITS>
__global__ void __launch_bounds__(kThreads)
k_adamw(const TensorTable t, const Hyper h, void* avg, void* sq, uint8_t* avg_scale, uint8_t* sq_scale) {
  int i = 0;
  while (i + 1 < t.count && t.chunk0[i + 1] <= blockIdx.x) ++i;
  const long long n = t.numel[i];
  const long long e0 = (long long)(blockIdx.x - t.chunk0[i]) * kChunk + threadIdx.x * kPer;
  typename P::T* p = static_cast<typename P::T*>(t.param[i]);
  const typename G::T* g = static_cast<const typename G::T*>(t.grad[i]);
  const long long s0 = t.first[i] + e0;
  if constexpr (BITS == 32) {
    float* ma = static_cast<float*>(avg) + s0;
    float* va = static_cast<float*>(sq) + s0;
    for (int j = 0; j < kPer; ++j) {
      if (e0 + j >= n) return;
      const float gj = G::load(g + e0 + j);
      const float m = fmaf((float)h.beta1, ma[j], (float)h.rest1 * gj);
      const float v = fmaf((float)h.beta2, va[j], (float)h.rest2 * gj * gj);
      ma[j] = m;
      va[j] = v;
      P::store(p + e0 + j, new_param(P::load(p + e0 + j), m, sqrtf(v), h));
    }
  } else {
    uint8_t* mc = static_cast<uint8_t*>(avg) + s0;
    uint8_t* rc = static_cast<uint8_t*>(sq) + s0;
    // a whole block of 32 is 4 neighbouring lanes; lanes behind the end take part in its maximum
    const long long block = s0 / kMomentBlock;
    const bool live = e0 < n;
    const int bm = live ? avg_scale[block] : 0, br = live ? sq_scale[block] : 0;
    double m[kPer], r[kPer];
    int em = -2000, er = -2000;
    for (int j = 0; j < kPer; ++j) {
      m[j] = r[j] = 0.0;
      if (e0 + j < n) {
        const double gj = G::load(g + e0 + j), old = from_e4m3(rc[j], br);
        m[j] = first_moment(from_e4m3(mc[j], bm), gj, h);
        r[j] = second_root(old, gj, h);
        P::store(p + e0 + j, new_param(P::load(p + e0 + j), (float)m[j], (float)r[j], h));
      }
      em = max(em, exponent(m[j]));
      er = max(er, exponent(r[j]));
    }
    for (int d = 1; d < 4; d <<= 1) {
      em = max(em, __shfl_xor(em, d, 64));
      er = max(er, __shfl_xor(er, d, 64));
    }
    const int nm = em == -2000 ? 0 : min(max(em + 120, 0), 254);
    const int nr = er == -2000 ? 0 : min(max(er + 120, 0), 254);
    for (int j = 0; j < kPer; ++j)
      if (e0 + j < n) {
        const unsigned bits = dither_bits(s0 + j, h.key);
        mc[j] = (uint8_t)e4m3(m[j], nm, bits & 0xffff, false);
        rc[j] = (uint8_t)e4m3(r[j], nr, bits >> 16, true);
      }
    if (live && (threadIdx.x & 3) == 0) {
      avg_scale[block] = (uint8_t)nm;
      sq_scale[block] = (uint8_t)nr;
    }
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
