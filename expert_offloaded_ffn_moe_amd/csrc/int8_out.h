// The epilogue that the 8-bit matrix products share, and their lane layouts.
//
// A product's sum over K is exact in int32 (K <= 131056 codes of -128..127), so it
// does not depend on how K is split over lanes, waves or tiles. The scales, the bias
// and what is added multiply and add in fp32; the output is rounded once.
#pragma once

#include <hip/hip_runtime.h>

#include "dense.h"

namespace moe {

typedef int32_t i32x4 __attribute__((ext_vector_type(4)));
typedef int32_t i32x16 __attribute__((ext_vector_type(16)));
typedef __attribute__((address_space(1))) const i32x4 gi32x4;

// act(v) as stored: fp32, or bf16 to nearest even with a NaN kept one
template <bool BF16>
struct OutElem;
template <>
struct OutElem<false> {
  typedef float T;
  static __device__ __forceinline__ float load(float v) { return v; }
  static __device__ __forceinline__ float rounded(float v) { return v; }
};
template <>
struct OutElem<true> {
  typedef uint16_t T;
  static __device__ __forceinline__ float load(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }
  static __device__ __forceinline__ uint16_t rounded(float f) {
    const uint32_t u = __float_as_uint(f);
    if ((u & 0x7FFFFFFFu) > 0x7F800000u) return (uint16_t)((u >> 16) | 0x40u);
    return (uint16_t)((u + 0x7FFFu + ((u >> 16) & 1u)) >> 16);
  }
};

// acc sx sw, each step rounded on its own, so that every kernel gives a token the same bits,
// whatever other tokens a call has. A sum of up to 2^31 times a token's scale of 2^96 and more
// may leave fp32 where the product does not: such a scale is taken 2^-32 fold and the product
// 2^32 fold, which changes no bit of what is finite.
__device__ __forceinline__ float int8_product(int acc, float sx, float sw) {
#pragma clang fp contract(off)
  const bool large = fabsf(sx) >= 0x1p96f;
  return (float)acc * (large ? sx * 0x1p-32f : sx) * sw * (large ? 0x1p32f : 1.f);
}

// The product's value before the output's rounding.
__device__ __forceinline__ float int8_scaled(int acc, float sx, float sw, float bias) {
#pragma clang fp contract(off)
  return int8_product(acc, sx, sw) + bias;
}

// What one output adds to its product, loaded before the sum is known (its latency would
// otherwise follow the sum's: one token on 7168 x 7168 9.9 us, 9.3 with it).
template <bool BF16>
struct OutTerms {
  typedef typename OutElem<BF16>::T E;
  float sw, bias, y;
  E res;
  __device__ __forceinline__ void load(const Int8Out& o, int t, int n) {
    sw = o.sw[n];
    bias = o.bias ? o.bias[n] : 0.f;
    y = o.y ? o.y[t * o.ld_y + n] : 0.f;
    res = o.res ? static_cast<const E*>(o.res)[t * o.ld_res + n] : E{};
  }
  __device__ __forceinline__ void store(const Int8Out& o, int t, int n, float sx, int acc) const {
    float v = int8_scaled(acc, sx, sw, bias);
    if (o.y) v += y;
    if (o.res) v += OutElem<BF16>::load(res);
    static_cast<E*>(o.out)[t * o.ld_out + n] = OutElem<BF16>::rounded(v);
  }
};

// Four neighbouring elements of a row, at any element's alignment (gfx950 performs such
// accesses whole).
struct __attribute__((packed, aligned(4))) F32x4u {
  float v[4];
};
struct __attribute__((packed, aligned(2))) Bf16x4u {
  uint32_t v[2];
};
__device__ __forceinline__ void load4(const float* p, int n, float* v) {
  if (n >= 4) {
    const F32x4u w = *reinterpret_cast<const F32x4u*>(p);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = w.v[i];
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = i < n ? p[i] : 0.f;
  }
}
__device__ __forceinline__ void load4(const uint16_t* p, int n, float* v) {
  if (n >= 4) {
    const Bf16x4u w = *reinterpret_cast<const Bf16x4u*>(p);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      v[2 * i] = __uint_as_float(w.v[i] << 16);
      v[2 * i + 1] = __uint_as_float(w.v[i] & 0xFFFF0000u);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = i < n ? OutElem<true>::load(p[i]) : 0.f;
  }
}
__device__ __forceinline__ void store4(float* p, int n, const float* v) {
  if (n >= 4) {
    F32x4u w;
#pragma unroll
    for (int i = 0; i < 4; ++i) w.v[i] = v[i];
    *reinterpret_cast<F32x4u*>(p) = w;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < n) p[i] = v[i];
  }
}
__device__ __forceinline__ void store4(uint16_t* p, int n, const float* v) {
  if (n >= 4) {
    Bf16x4u w;
#pragma unroll
    for (int i = 0; i < 2; ++i)
      w.v[i] = (uint32_t)OutElem<true>::rounded(v[2 * i]) | (uint32_t)OutElem<true>::rounded(v[2 * i + 1]) << 16;
    *reinterpret_cast<Bf16x4u*>(p) = w;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < n) p[i] = OutElem<true>::rounded(v[i]);
  }
}

// silu(g) u, each from its exact sum; exp(-g) past fp32's range gives the limit 0
__device__ __forceinline__ float gated_value(int g_acc, int u_acc, float sx, float sg, float su) {
  const float g = int8_product(g_acc, sx, sg), u = int8_product(u_acc, sx, su);
  return g / (1.f + __expf(-g)) * u;
}

}  // namespace moe
