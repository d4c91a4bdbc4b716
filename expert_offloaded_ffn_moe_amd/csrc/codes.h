// 8-bit codes of a row of known largest size: round half even(127 v / max|v|).
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

namespace moe {

__device__ __forceinline__ uint32_t abs_bits(float f) { return __float_as_uint(f) & 0x7FFFFFFFu; }
constexpr uint32_t kNotFinite = 0x7F800000u;  // abs_bits from here on: an infinity or a NaN
constexpr uint32_t kNoCodes = 27u << 23;      // abs_bits under it (2^-100): a row whose codes are 0

__device__ __forceinline__ float power_of_two(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// Codes under the row's largest size: a = 127 p 2^(1-e) and b = max|p| 2^(1-e) in [2, 4), so
// that nothing over- or underflows; q = a y, corrected once, is a / b rounded correctly.
// Adding 1.5 2^23 (2^52) rounds to a whole number, half to even, and leaves its two's
// complement in the low bits.
struct Quotient32 {
  float c, b, y;
  __device__ __forceinline__ explicit Quotient32(float top) {
    const float f = power_of_two(128 - (int)(__float_as_uint(top) >> 23));
    c = 127.f * f;
    b = top * f;
    y = 1.f / b;
  }
  __device__ __forceinline__ uint32_t code(float p) const {
    const float a = p * c;
    const float q = a * y;
    return __float_as_uint(fmaf(fmaf(-b, q, a), y, q) + 12582912.f) & 0xFFu;
  }
};
struct Quotient64 {
  double b, y;
  __device__ __forceinline__ explicit Quotient64(double top) : b(top), y(1.0 / top) {}
  __device__ __forceinline__ uint32_t code(double p) const {
    const double a = 127.0 * p;
    const double q = a * y;
    return (uint32_t)__double_as_longlong(fma(fma(-b, q, a), y, q) + 6755399441055744.0) & 0xFFu;
  }
};

// The scale of a row whose largest size has abs_bits `top_bits`: what the codes multiply
// with, NaN where the row is not finite.
__device__ __forceinline__ float code_scale(uint32_t top_bits, double top) {
  return top_bits >= kNotFinite ? __uint_as_float(0x7FC00000u) : top_bits < kNoCodes ? 0.f : (float)(top * (1.0 / 127.0));
}

}  // namespace moe
