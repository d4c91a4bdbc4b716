// e4m3 codes as operands of the bf16 matrix instruction, on which their products are exact.
//
// Lane layout of the 16x16x32 bf16 MFMA: lane l supplies 8 values of row l % 16 of each
// operand at K offset 8 (l / 16), and receives the sums of column l % 16 and rows 4 (l / 16)
// .. + 3. Which of a block's K a lane supplies is free as long as both operands agree.
//
// Few tokens. A load instruction takes a cycle for each line that each four neighbouring lanes
// touch (16 rows of 64 bytes: 65 cycles, 8 rows of 128: 32), so lanes are given two neighbouring
// pieces of a row: the MFMA's rows 2 a and 2 a + 1 are both row a of the weights, at a block's even
// and odd pieces of 16 codes (piece 2 q + (row & 1) for lane quarter q), and its columns 2 v and
// 2 v + 1 both vector v, at even and odd pieces. Of the products of rows and columns those of like
// parity are the sums wanted, of 8 rows with 8 vectors; a row's whole sum is that of two
// neighbouring lanes.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

namespace moe {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef int32_t f8i4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2v __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8v __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(1))) const f8i4 g_f8i4;

// Eight codes as bf16 (every e4m3 number is one, and so is its product with a power of two from
// 2^-100 to 2^100; a NaN stays one).
__device__ __forceinline__ bf16x8v f8_to_bf16(int lo, int hi, float power = 1.f) {
  const bf16x2v a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, power, false), b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, power, true);
  const bf16x2v c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, power, false), d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, power, true);
  return bf16x8v{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

__device__ __forceinline__ f32x4 mfma_bf16(const bf16x8v& a, const bf16x8v& b, const f32x4& c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// 0 that the compiler takes for a lane's own: a load with it in its address is a vector load, which is
// waited for in the order of the vector loads. (A scalar load is waited for with every LDS read.)
__device__ __forceinline__ int lane_zero() {
  int z;
  asm volatile("v_mov_b32 %0, 0" : "=v"(z));
  return z;
}

// Of a lane's two sums of a row, the one of its parity.
__device__ __forceinline__ float of_parity(float even, float odd) { return threadIdx.x & 1 ? odd : even; }

// Every wave's LDS accesses are done; loads from memory stay under way.
__device__ __forceinline__ void meet() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

}  // namespace moe
