// e4m3.cuh -- the 8-bit format of the key / value cache: e4m3 codes with one
// scale per head and 32 tokens.
//
// A scale is a power of two, 2^ceil(log2(amax / 448)) with the exponent held
// in [-40, 40] (448 is the largest e4m3 value), so multiplying by it is exact:
// a value's code does not depend on how the division is rounded, and moving a
// code to a larger scale rounds only codes that become subnormal.
#pragma once
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

namespace rfb {

constexpr int kCacheBlock = 32;  // tokens per scale
constexpr int kScaleMinExp = -40, kScaleMaxExp = 40;

__device__ __forceinline__ float pow2f(int e) { return __int_as_float((e + 127) << 23); }

// Scale for values of largest magnitude amax (finite, >= 0), from the bits of
// amax as fp32: amax = m 2^e with m in [1/2, 1); 448 = 0.875 2^9.
__device__ __forceinline__ float scale_for(float amax) {
  const int bits = __float_as_int(amax);
  int e = (bits >> 23) - 126;                       // subnormal and zero amax: far below the floor
  e = (bits & 0x7fffff) > 0x600000 ? e - 8 : e - 9;  // m > 0.875
  return pow2f(min(max(e, kScaleMinExp), kScaleMaxExp));
}

// Two e4m3 codes, the low or the high half of a register, as two fp16 values; exact.
__device__ __forceinline__ uint32_t e4m3_lo(uint32_t w) {
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}" : "=r"(r) : "r"(w));
  return r;
}
__device__ __forceinline__ uint32_t e4m3_hi(uint32_t w) {
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, hi;\n\t}" : "=r"(r) : "r"(w));
  return r;
}
__device__ __forceinline__ float2 f16x2_to_f32x2(uint32_t h) {
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}
// Round to nearest even; magnitudes above 448 become 448, NaN the NaN code.
__device__ __forceinline__ uint32_t f32x2_to_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
// Four codes to a scale that is 1 / ratio times theirs.
__device__ __forceinline__ uint32_t requantise4(uint32_t v, float ratio) {
  const float2 a = f16x2_to_f32x2(e4m3_lo(v)), b = f16x2_to_f32x2(e4m3_hi(v));
  return f32x2_to_e4m3x2(a.x * ratio, a.y * ratio) |
         (f32x2_to_e4m3x2(b.x * ratio, b.y * ratio) << 16);
}
// Larger magnitude of two fp16 pairs, NaN ignored.
__device__ __forceinline__ uint32_t max_mag_f16x2(uint32_t a, uint32_t b) {
  const __half2 r = __hmax2(*reinterpret_cast<const __half2*>(&a),
                            __habs2(*reinterpret_cast<const __half2*>(&b)));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t max_mag_e4m3x4(uint32_t top, uint32_t codes) {
  return max_mag_f16x2(max_mag_f16x2(top, e4m3_lo(codes)), e4m3_hi(codes));
}
// Four codes to a scale that is 2^-k times theirs, ratio = (2^k, 2^k) as fp16, k in
// [-14, 15] and no result above 448.  The product in fp16 is exact, or, where it loses
// bits, so far below half the smallest code that it becomes zero either way.
__device__ __forceinline__ uint32_t shift_codes4(uint32_t v, __half2 ratio) {
  const uint32_t lo = e4m3_lo(v), hi = e4m3_hi(v);
  const __half2 a = __hmul2(*reinterpret_cast<const __half2*>(&lo), ratio);
  const __half2 b = __hmul2(*reinterpret_cast<const __half2*>(&hi), ratio);
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\tcvt.rn.satfinite.e4m3x2.f16x2 lo, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f16x2 hi, %2;\n\tmov.b32 %0, {lo, hi};\n\t}"
      : "=r"(r)
      : "r"(*reinterpret_cast<const uint32_t*>(&a)), "r"(*reinterpret_cast<const uint32_t*>(&b)));
  return r;
}

}  // namespace rfb
