// Rows kept in 8 bits: one e4m3 code per element, one power of two per 32
// columns of a row (a byte: its exponent + 127).  The power is the least that
// takes the block's largest finite magnitude to 448, e4m3's largest value, or
// below, and at least 2^-126; dividing by it is exact, so that an element is
// off by one rounding: at most 2^-4 of its value, or, below 2^-6 of the power,
// 2^-10 of the power.  What would round to 2^128 becomes the value below,
// 15/16 of that, no further off.  Infinities and NaN are kept as NaN.
#pragma once

#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "row_common.cuh"

namespace gemm_f32_dev {

constexpr int kSavedBlock = 32;

// Bits of a magnitude as the block's largest counts it.
__device__ __forceinline__ uint32_t finite_bits(float x) {
  const uint32_t u = __float_as_uint(x) & 0x7FFFFFFFu;
  return u < 0x7F800000u ? u : 0u;
}

// The largest bits of 8 magnitudes, with what is not finite above all others.
__device__ __forceinline__ uint32_t largest_bits(const Raw<float, 8>& x) {
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) top = max(top, x.w[i] & 0x7FFFFFFFu);
  return top;
}
__device__ __forceinline__ uint32_t largest_bits(const Raw<__nv_bfloat16, 8>& x) {
  uint32_t top = 0;                      // two at a time
#pragma unroll
  for (int i = 0; i < 4; ++i) top = __vmaxu2(top, x.w[i] & 0x7FFF7FFFu);
  return max(top & 0xFFFF0000u, top << 16);
}

// The byte of a block whose largest finite magnitude has these bits.
__device__ __forceinline__ uint32_t block_exponent(uint32_t top) {
  // top = 1.m 2^(field - 127): into (224, 448] by 8 powers less, one more of
  // them where 1.m is above 1.75
  const int e = static_cast<int>(top >> 23) - 8 + ((top & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return static_cast<uint32_t>(max(e, 1));
}

__device__ __forceinline__ float power_of(uint32_t byte) { return __uint_as_float(byte << 23); }
__device__ __forceinline__ float inverse_of(uint32_t byte) { return __uint_as_float((254u - byte) << 23); }

// Two values, already divided by the power, as codes.
__device__ __forceinline__ uint32_t finite_codes(float a, float b) {
  return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}
// The same, at most `most`, where they may not be finite, which has to stay
// visible: the conversion takes infinity to 448.
__device__ __forceinline__ uint32_t codes_of(float a, float b, float most) {
  return finite_codes(fabsf(a) < INFINITY ? fminf(fmaxf(a, -most), most) : NAN,
                      fabsf(b) < INFINITY ? fminf(fmaxf(b, -most), most) : NAN);
}
// Magnitudes from here on need that: they round to 2^128 or are not finite.
constexpr uint32_t kOddBits = 0x7F780000u;
constexpr uint32_t kLargestExponent = 247;   // of finite values: codes of 256 stand for 2^128

// Two codes, the low one first, as fp32 (before the power).
__device__ __forceinline__ float2 values_of(uint32_t codes) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(codes), __NV_E4M3);
  return __half22float2(__half2(h));
}

}  // namespace gemm_f32_dev
