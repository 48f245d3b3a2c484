// ex_fp8.cuh -- the 8-bit block rule: scale, rounding, and the scales' layout.
#pragma once

#include "ex_common.cuh"

namespace zc {
namespace ex {

constexpr int kBlock = ZC_FP8_BLOCK;

__host__ __device__ inline size_t ceil_div(size_t a, size_t b) { return (a + b - 1) / b; }
// Byte of row r's scale for block b (`rows` rows).
__host__ __device__ inline size_t scale_at(size_t r, size_t b, size_t rows) { return (b / 4 * rows + r) * 4 + b % 4; }

// A block's exponent s from its largest finite magnitude's fp32 bits: the smallest s with
// amax <= MAX 2^s, MAX = 1.75 * 2^8 (e4m3) or 1.75 * 2^15 (e5m2).  With amax = 1.f * 2^(E - 127)
// that is E - 127 - 8 (or 15), and one more when the fraction is above 0.75.  Clamped to
// [-127, 127] (a subnormal amax has E = 0 and lands on the clamp); 0 for amax = 0.
__device__ __forceinline__ int block_exponent(uint32_t amax_bits, int fmt) {
  const int e = static_cast<int>(amax_bits >> 23) - 127 - (fmt == ZC_FP8_E4M3 ? 8 : 15) +
                ((amax_bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return amax_bits == 0 ? 0 : max(-127, e);
}
// 2^-s, s in [-127, 126]: exact (2^-126 and above are normal; no s here exceeds 126).
__device__ __forceinline__ float inverse_scale(int s) { return __uint_as_float(static_cast<uint32_t>(127 - s) << 23); }

// Two values rounded to 8 bits, a in the low byte; saturating (no finite scaled value passes MAX).
__device__ __forceinline__ unsigned short round8x2(float a, float b, int fmt) {
  unsigned short r;
  if (fmt == ZC_FP8_E4M3) asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
  else asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
  return r;
}
// The 8-bit form of Inf or NaN: NaN for NaN, and for Inf where the format has none.
__device__ __forceinline__ unsigned nonfinite8(float v, int fmt) {
  const unsigned sign = __float_as_uint(v) >> 31 << 7;
  return fmt == ZC_FP8_E5M2 && isinf(v) ? sign | 0x7Cu : sign | 0x7Fu;
}

}  // namespace ex
}  // namespace zc
