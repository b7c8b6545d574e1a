// Launches of the tiled products with trellis-coded weights. Built three times, with CODE_TYPE one of F32,
// F16 and BF16: a type's variants (folds, row tiles, bits a step, tables) are a hundred kernels.
#include <hip/hip_runtime.h>

#include "code_any.h"
#include "code_mfma.h"
#include "ops.h"

namespace bcjr {
namespace {

template <class E, int F, int RT, int NT, int K, bool PAIR>
int launch_tiles(CodeArgs a, hipStream_t stream) {
  constexpr int kRowsOfWave = RT * 16 / F;
  const int steps = (a.tile.cols / 128 + F - 1) / F;
  const int64_t units = (a.tile.rows + kRowsOfWave - 1) / kRowsOfWave;
  // Every block makes a table, which its 8 waves share, and no more blocks than fit the chip are started.
  constexpr int waves = kMaxWaves;
  const size_t lds = Table<E, K, PAIR>::bytes(a.n) + (size_t)waves * NT * kXBytes;
  if (lds > kLds) return (int)hipErrorInvalidValue;  // the callers' rules leave room
  const int kw = waves_along(steps, units);
  a.tile.kw = kw;
  const int64_t rw = waves / kw, blocks = (units + rw - 1) / rw;
  const int64_t tokens = (a.tile.tokens + NT * tile_tokens<E, F>() - 1) / (NT * tile_tokens<E, F>());
  const void* kernel = reinterpret_cast<const void*>(k_code_tiles<E, F, RT, NT, K, PAIR>);
  if (lds > 65536) {
    const hipError_t e = hipFuncSetAttribute(kernel, hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
    if (e != hipSuccess) return (int)e;
  }
  const int64_t room = 256 * (lds > kLds / 2 ? 1 : 2);
  hipLaunchKernelGGL((k_code_tiles<E, F, RT, NT, K, PAIR>), dim3((unsigned)(blocks < room ? blocks : room), (unsigned)tokens),
                     dim3(64 * waves), lds, stream, a);
  return (int)hipGetLastError();
}

template <class E, int F, int RT, int NT, bool PAIR>
int launch_tiles_bits(const CodeArgs& a, int k, hipStream_t stream) {
  return k == 1   ? launch_tiles<E, F, RT, NT, 1, PAIR>(a, stream)
         : k == 2 ? launch_tiles<E, F, RT, NT, 2, PAIR>(a, stream)
         : k == 3 ? launch_tiles<E, F, RT, NT, 3, PAIR>(a, stream)
                  : launch_tiles<E, F, RT, NT, 4, PAIR>(a, stream);
}

// The table of two states' windows serves 13.3 weights a clock in place of 8.8, and costs no more to make up to 32
// KiB. At 128 KiB (n + k = 14: S = 4096 with two bits a step) making it takes a microsecond longer: 1024 x 2048
// with one token 5.8 against 4.8 us, 2048 x 8192 8.3 against 8.6, 8192 x 8192 with 16 tokens 21.7 against 25.6.
template <class E, int F, int RT, int NT>
int launch_tiles_table(const CodeArgs& a, int k, hipStream_t stream) {
  if constexpr (Codeword<E>::kWords == 1) {
    const bool large = NT == 1 && a.tile.rows * a.tile.cols >= ((int64_t)1 << 23);
    if (a.n + k <= (large ? 14 : 12)) return launch_tiles_bits<E, F, RT, NT, true>(a, k, stream);
  }
  return launch_tiles_bits<E, F, RT, NT, false>(a, k, stream);
}

// Waves that RT tiles a wave leave.
template <int F>
int64_t waves_of(const CodeArgs& a, int rt) {
  const int64_t steps = (a.tile.cols / 128 + F - 1) / F;
  return (a.tile.rows * F + 16 * rt - 1) / (16 * rt) * (steps < kMaxWaves ? steps : kMaxWaves);
}

// As many row tiles a wave, which share the x, as leave 8 waves for each of 256 CUs: 8192 x 8192 with 16 tokens takes
// 24.8 / 21.2 / 29.7 us with 1 / 2 / 4 (4096 / 2048 / 1024 waves), 16384 x 16384 74 / 59 / 53 us (2048 with 4).
template <class E, int F>
int launch_tiles_rows(const CodeArgs& a, int k, hipStream_t stream) {
  return waves_of<F>(a, 4) >= 2048   ? launch_tiles_table<E, F, 4, 1>(a, k, stream)
         : waves_of<F>(a, 2) >= 2048 ? launch_tiles_table<E, F, 2, 1>(a, k, stream)
                                     : launch_tiles_table<E, F, 1, 1>(a, k, stream);
}

// The largest fold that the tokens leave room for and the columns fill; for more tokens than a tile holds two
// tiles of them, decoded for once, where that leaves waves enough (32 tokens: 8192 x 8192 31 us against 37 one by
// one, 2048 x 8192 27 us against 14).
template <class E>
int launch_tiles_any(const CodeArgs& a, int k, hipStream_t stream) {
  const int blocks = a.tile.cols / 128;
  if constexpr (TileOf<E>::T::kParts == 1) {
    if (a.tile.tokens == 1 && blocks > 8) return launch_tiles_rows<E, 16>(a, k, stream);
    if (a.tile.tokens <= 2 && blocks > 4) return launch_tiles_rows<E, 8>(a, k, stream);
  }
  if (a.tile.tokens <= tile_tokens<E, 4>() && blocks > 2) return launch_tiles_rows<E, 4>(a, k, stream);
  if (a.tile.tokens <= tile_tokens<E, 2>() && blocks > 1) return launch_tiles_rows<E, 2>(a, k, stream);
  if constexpr (Codeword<E>::kWords == 1)
    if (a.tile.tokens > tile_tokens<E, 1>() && waves_of<1>(a, 2) >= 2048 && a.n < 15)
      return launch_tiles_table<E, 1, 2, 2>(a, k, stream);
  return launch_tiles_rows<E, 1>(a, k, stream);
}

template <class E, int F, bool IN_LDS>
int launch_any_table(CodeArgs a, hipStream_t stream) {
  const int steps = ((a.tile.cols + 127) / 128 + F - 1) / F;
  const int64_t units = (a.tile.rows + 16 / F - 1) / (16 / F);
  const size_t lds = (IN_LDS ? (a.n < 4 ? 64 : (size_t)4 << a.n) : 0) + (size_t)kMaxWaves * kXBytes;
  const int kw = waves_along(steps, units);
  a.tile.kw = kw;
  const int64_t rw = kMaxWaves / kw, blocks = (units + rw - 1) / rw;
  const int64_t tokens = (a.tile.tokens + tile_tokens<E, F>() - 1) / tile_tokens<E, F>();
  const void* kernel = reinterpret_cast<const void*>(k_code_any<E, F, IN_LDS>);
  if (lds > 65536) {
    const hipError_t e = hipFuncSetAttribute(kernel, hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
    if (e != hipSuccess) return (int)e;
  }
  const int64_t room = 256 * (lds > kLds / 2 ? 1 : 2);
  hipLaunchKernelGGL((k_code_any<E, F, IN_LDS>), dim3((unsigned)(blocks < room ? blocks : room), (unsigned)tokens),
                     dim3(64 * kMaxWaves), lds, stream, a);
  return (int)hipGetLastError();
}

template <class E, int F>
int launch_any_fold(const CodeArgs& a, hipStream_t stream) {
  return a.n <= 15 ? launch_any_table<E, F, true>(a, stream) : launch_any_table<E, F, false>(a, stream);
}

template <class E>
int launch_any(const CodeArgs& a, hipStream_t stream) {
  const int blocks = (a.tile.cols + 127) / 128;
  if constexpr (TileOf<E>::T::kParts == 1)
    if (a.tile.tokens == 1 && blocks > 8) return launch_any_fold<E, 16>(a, stream);
  if constexpr (TileOf<E>::T::kParts <= 2)
    if (a.tile.tokens <= tile_tokens<E, 8>() && blocks > 4) return launch_any_fold<E, 8>(a, stream);
  if (a.tile.tokens <= tile_tokens<E, 4>() && blocks > 2) return launch_any_fold<E, 4>(a, stream);
  if (a.tile.tokens <= tile_tokens<E, 2>() && blocks > 1) return launch_any_fold<E, 2>(a, stream);
  return launch_any_fold<E, 1>(a, stream);
}

}  // namespace

#define CODE_LAUNCH_(type) launch_code_tiles_##type
#define CODE_LAUNCH(type) CODE_LAUNCH_(type)
int CODE_LAUNCH(CODE_NAME)(const CodeArgs& a, int k, void* stream) {
  if (a.L == 0) return launch_tiles_any<CODE_TYPE>(a, k, static_cast<hipStream_t>(stream));
  using Parts = std::conditional<std::is_same<CODE_TYPE, F16>::value, F16Parts, CODE_TYPE>::type;
  return launch_any<Parts>(a, static_cast<hipStream_t>(stream));
}

}  // namespace bcjr
