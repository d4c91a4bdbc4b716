// e4m3 codes of blocks: 128 neighbours of a row, or 128 x 128.
//
//   scale = max|v| / 448,  code = the e4m3 number nearest to 448 v / max|v|, ties to even
//
// The quotient is correctly rounded (a product with the correctly rounded reciprocal and one
// correction step; of bf16 values in fp32, where 448 v is exact, of fp32 values in fp64),
// and then rounded once more to e4m3. The second rounding goes wrong only where the first
// one reaches a tie of the second without the exact quotient being one. A tie b has at most 5 bits,
// and 448 v and b max|v| are whole multiples of one step of their own: of bf16 values they
// differ by 2^-13 of b max|v| at least or not at all, of fp32 values by 2^-29, far more than
// fp32's (fp64's) half step. On its way from fp64 to e4m3 the quotient passes through fp32
// rounded to odd, which no tie is.
//
// One pass: 16 lanes take a row's 128 values, 8 a lane, so that a block's maximum is four
// steps within a row of lanes. The bound is the bytes, and for a few rows the launch: with inputs
// from HBM one row of 7168 takes 2.1 us, 1023 x 2000 fp32 5.6 (1.8 TB/s: four rounds of loads are
// short), 2048 x 7168 bf16 14.4 (3.1 TB/s), 7168 x 2048 in 128 x 128 blocks 13.9 in bf16 (3.2), 19.3 in fp32
// (3.8).
#include <hip/hip_runtime.h>

#include <type_traits>

#include "codes.h"
#include "fp8.h"
#include "int8_out.h"
#include "wave.h"

namespace moe {
namespace {

// The quotient 448 p / top as the conversion instruction takes it.
struct F8Quotient32 {
  float c, b, y;
  __device__ __forceinline__ explicit F8Quotient32(float top) {
    // b = top 2^e in [2, 4): nothing over- or underflows that counts
    const float f = power_of_two(128 - (int)(__float_as_uint(top) >> 23));
    c = 448.f * f;
    b = top * f;
    y = 1.f / b;
  }
  __device__ __forceinline__ float operator()(float p) const {
    const float a = p * c, q = a * y;
    return fmaf(fmaf(-b, q, a), y, q);
  }
};
struct F8Quotient64 {
  double b, y;
  __device__ __forceinline__ explicit F8Quotient64(float top) : b(top), y(1.0 / (double)top) {}
  __device__ __forceinline__ float operator()(float p) const {
    const double a = 448.0 * (double)p, q0 = a * y, q = fma(fma(-b, q0, a), y, q0);
    const uint64_t u = __double_as_longlong(q);
    const uint64_t low = (1ull << 29) - 1;  // the bits that fp32 does not hold
    return (float)__longlong_as_double((u & ~low) | ((u & low) ? 1ull << 29 : 0));
  }
};

// largest over the 16 lanes of a row of lanes
__device__ __forceinline__ uint32_t row_max_u(uint32_t v) {
  v = max(v, (uint32_t)dpp<kDppXor1, 0xF>(0, (int)v));
  v = max(v, (uint32_t)dpp<kDppXor2, 0xF>(0, (int)v));
  v = max(v, (uint32_t)dpp<kDppHalfMirror, 0xF>(0, (int)v));
  v = max(v, (uint32_t)dpp<kDppMirror, 0xF>(0, (int)v));
  return v;
}

// Eight neighbours of a row, those from `n` on as zeros.
__device__ __forceinline__ void load8(const uint16_t* p, int n, float* v) {
  load4(p, n, v);
  load4(p + 4, n - 4, v + 4);
}
__device__ __forceinline__ void load8(const float* p, int n, float* v) {
  load4(p, n, v);
  load4(p + 4, n - 4, v + 4);
}

struct __attribute__((packed, aligned(1))) Codes8 {
  uint32_t v[2];
};

template <typename ACT>
__device__ __forceinline__ void store_codes(uint8_t* p, int n, const float* v, uint32_t top) {
  typedef typename std::conditional<sizeof(ACT) == 2, F8Quotient32, F8Quotient64>::type Quotient;
  const bool none = top >= kNotFinite || top < kNoCodes;
  const Quotient quot(none ? 1.f : __uint_as_float(top));
  Codes8 c;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(quot(v[4 * i]), quot(v[4 * i + 1]), 0, false);
    w = __builtin_amdgcn_cvt_pk_fp8_f32(quot(v[4 * i + 2]), quot(v[4 * i + 3]), w, true);
    c.v[i] = none ? 0u : (uint32_t)w;
  }
  if (n >= 8) {
    *reinterpret_cast<Codes8*>(p) = c;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = (uint8_t)(c.v[i / 4] >> (8 * (i % 4)));
  }
}

__device__ __forceinline__ float f8_scale(uint32_t top) {
  return top >= kNotFinite ? __uint_as_float(0x7FC00000u) : top < kNoCodes ? 0.f : (float)((double)__uint_as_float(top) * (1.0 / 448.0));
}

constexpr int kThreads = 256, kSquareThreads = 1024;

// Blocks of one row: 16 lanes a block, a workgroup's blocks side by side.
template <typename ACT>
__global__ __launch_bounds__(kThreads) void k_fp8_rows(Fp8QuantArgs a, int per_row) {
  constexpr int kAt = kThreads / 16;
  const int64_t blocks = (int64_t)a.T * per_row;
  for (int64_t first = (int64_t)blockIdx.x * kAt; first < blocks; first += (int64_t)gridDim.x * kAt) {
    const int64_t block = first + threadIdx.x / 16, row = block / per_row;
    const int b = (int)(block - row * per_row), j = b * kF8Block + 8 * (threadIdx.x & 15), n = a.H - j;
    const bool mine = block < blocks;
    float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (mine && n > 0) load8(static_cast<const ACT*>(a.x) + row * a.ld_x + j, n, v);
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, abs_bits(v[i]));
    top = row_max_u(top);
    if (mine && n > 0) store_codes<ACT>(a.q + row * a.ld_q + j, n, v, top);
    if (mine && (threadIdx.x & 15) == 0) a.s[row * a.ld_s + b] = f8_scale(top);
  }
}

// Blocks of 128 rows: a workgroup a block, 64 rows at a time, all held in registers (7168 x 2048: 13.7
// us; with 512 threads 14.8, with 256 15.6).
template <typename ACT>
__global__ __launch_bounds__(kSquareThreads) void k_fp8_squares(Fp8QuantArgs a) {
  constexpr int kRows = kSquareThreads / 16, kPasses = kF8Block / kRows;
  const int64_t r0 = (int64_t)blockIdx.y * kF8Block + threadIdx.x / 16;
  const int j = blockIdx.x * kF8Block + 8 * (threadIdx.x & 15), n = a.H - j;
  float v[kPasses][8];
  uint32_t top = 0;
#pragma unroll
  for (int p = 0; p < kPasses; ++p) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[p][i] = 0.f;
    const int64_t row = r0 + p * kRows;
    if (row < a.T && n > 0) load8(static_cast<const ACT*>(a.x) + row * a.ld_x + j, n, v[p]);
  }
#pragma unroll
  for (int p = 0; p < kPasses; ++p)
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, abs_bits(v[p][i]));
  top = wave_max_u(top);
  __shared__ uint32_t tops[kSquareThreads / 64];
  if (threadIdx.x % 64 == 0) tops[threadIdx.x / 64] = top;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kSquareThreads / 64; ++i) top = max(top, tops[i]);
#pragma unroll
  for (int p = 0; p < kPasses; ++p) {
    const int64_t row = r0 + p * kRows;
    if (row < a.T && n > 0) store_codes<ACT>(a.q + row * a.ld_q + j, n, v[p], top);
  }
  if (threadIdx.x == 0) a.s[blockIdx.y * a.ld_s + blockIdx.x] = f8_scale(top);
}

template <typename ACT>
void quantize(const Fp8QuantArgs& a, int block_rows, hipStream_t s) {
  const int per_row = f8_blocks(a.H);
  if (block_rows == 1) {
    const int64_t groups = ((int64_t)a.T * per_row - 1) / (kThreads / 16) + 1;
    const int64_t most = 1 << 22;  // a grid's threads are counted in 32 bits
    hipLaunchKernelGGL((k_fp8_rows<ACT>), dim3((unsigned)(groups < most ? groups : most)), dim3(kThreads), 0, s, a, per_row);
  } else {
    hipLaunchKernelGGL((k_fp8_squares<ACT>), dim3(per_row, f8_blocks(a.T)), dim3(kSquareThreads), 0, s, a);
  }
}

}  // namespace

void launch_fp8_quantize(const Fp8QuantArgs& a, bool act_bf16, int block_rows, hipStream_t s) {
  if (act_bf16)
    quantize<uint16_t>(a, block_rows, s);
  else
    quantize<float>(a, block_rows, s);
}

}  // namespace moe
