// e4m3 values and the scales of the 8-bit cache.
#pragma once

#include "common.cuh"

namespace hf {

// Scales are 2^e, kScaleLow <= e <= kScaleHigh: the attention keeps its weights times a scale and
// their sum without one in the same 32 bits, which this range leaves room for.
constexpr int kScaleLow = -64, kScaleHigh = 63;
constexpr float kE4m3Top = 448.f;

__device__ __forceinline__ float pow2f(int e) { return __int_as_float((e + 127) << 23); }  // -126 <= e <= 127

// The least scale that brings the magnitude `top` (finite, >= 0) to 448 = 1.75 * 2^8 at most. Read off
// the bits: with top = m 2^k, 1 <= m < 2, it is 2^(k - 8) up to m = 1.75 and 2^(k - 7) above.
__device__ __forceinline__ float scale_for(float top) {
  const int bits = __float_as_int(top);
  const int e = (bits >> 23) - 127 - 8 + ((bits & 0x7fffff) > 0x600000);
  return pow2f(min(max(e, kScaleLow), kScaleHigh));
}
// A scale as the cache holds it; what a page that nobody wrote holds counts as the least.
__device__ __forceinline__ float held_scale(float s) {
  // (positive floats are in the order of their bits; NaN and negative ones lie above)
  const uint32_t low = (uint32_t)(kScaleLow + 127) << 23, high = (uint32_t)(kScaleHigh + 127) << 23;
  return __float_as_uint(s) - low <= high - low ? s : pow2f(kScaleLow);
}

// Two values to codes, x in the lower byte: nearest, ties to even, magnitudes held to 448.
__device__ __forceinline__ uint32_t to_e4m3x2(float x, float y) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(y), "f"(x));
  return r;
}
// Infinities become NaN (a code holds none), so that they are not held to 448.
__device__ __forceinline__ float no_inf(float x) { return fabsf(x) < INFINITY ? x : NAN; }
// Two codes to values, exactly.
__device__ __forceinline__ float2 from_e4m3x2(uint32_t codes) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)codes));
  float2 v;
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
      : "=f"(v.x), "=f"(v.y)
      : "r"(h));
  return v;
}
__device__ __forceinline__ float from_e4m3(uint8_t code) { return from_e4m3x2(code).x; }

}  // namespace hf
