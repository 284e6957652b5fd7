// e4m3.cuh -- conversions of the 8-bit KV cache: e4m3 values with a
// power-of-two scale for each (page, kv head), kept as an exponent byte e (the
// scale is 2^(e - 127)).  A power-of-two scale costs a floating format no
// precision, makes scaling exact, and lets a page's rows move to a larger
// scale without a second rounding (but where they fall below e4m3's normal
// range).
#pragma once

#include <stdint.h>

#include <cuda_fp16.h>

namespace spec {

constexpr int kExpBias = 127;
constexpr int kExpMin = SPEC_Q8_EXP_MIN;

// 2^(e - 127) for e in [1, 254]
__device__ __forceinline__ float exp_scale(int e) { return __uint_as_float(uint32_t(e) << 23); }
// 2^(127 - e) for e in [1, 254] (of 254, the subnormal 2^-127)
__device__ __forceinline__ float inv_scale(int e) { return __uint_as_float(e < 254 ? uint32_t(254 - e) << 23 : 1u << 22); }

// Exponent byte of the smallest power-of-two scale at which a bf16 magnitude
// (its 15 bits below the sign, finite) is at most 448 = 1.75 * 2^8.
__device__ __forceinline__ int scale_exp_of(uint32_t bits) {
  const int e = int(bits >> 7);                        // biased exponent
  const int x = e - 8 + ((bits & 0x7fu) > 0x60u ? 1 : 0);  // mantissa above 1.75: one more
  return x < kExpMin ? kExpMin : x;                    // (a subnormal or zero magnitude lands on kExpMin)
}

// two e4m3 bytes (low half of w) to f16x2, exactly
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t w) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(uint16_t(w)));
  return r;
}
// four e4m3 bytes to two f16x2 (one asm, so that the halves of w need no instructions of their own)
__device__ __forceinline__ void e4m3x4_to_f16x4(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n.reg .b16 a, b;\nmov.b32 {a, b}, %2;\ncvt.rn.f16x2.e4m3x2 %0, a;\ncvt.rn.f16x2.e4m3x2 %1, b;\n}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}
// two floats to e4m3 (nearest even; +-inf and anything past 448 saturates, NaN stays NaN); lo in the low byte
__device__ __forceinline__ uint32_t pack_e4m3(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

}  // namespace spec
