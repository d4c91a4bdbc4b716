// Product of e4m3 codes with a scale for each block of 128, for up to 8 tokens.
//
//   out[t][n] = sum_b sx[t][b] sw[n / 128][b] sum_{k in b} x[t][k] w[n][k] + ...
//
// The weights are the row operand and the tokens the column operand of the bf16 MFMA, both at two
// parities of the pieces of K (f8_dev.h). A workgroup takes 16 weight rows and all tokens; its waves
// take blocks of 128 of K in turn and meet in LDS. A block's sum starts from zero and is added to
// the wave's with both scales, in fp32.
//
// Bound: the weights' bytes, which go from memory to registers with 16-byte loads: one token on 7168 x
// 7168 11.0 us (4.7 TB/s) with all inputs from HBM, on 4096 x 7168 7.5. Scales are multiplied into LDS
// first: loaded with each block, they took two of its five loads (12.7 us).
#include <hip/hip_runtime.h>

#include "f8_dev.h"
#include "fp8.h"
#include "int8_out.h"
#include "wave.h"

namespace moe {
namespace {

// Tokens up to which this kernel runs, on any weights, so that how exact a token's sums are turns on the
// number of tokens alone: 8 on 4096 x 7168 10.4 us (fp32 tiles 12.3), on 7168 x 7168 12.9 (13.0), on 2048 x
// 2048 6.0 (6.6), on 14336 x 4096 17.8 (16.6); bf16 tiles, whose products are cut, take 11.4, 12.4, 6.1 and
// 15.2.
constexpr int kSkinnyRows = 8;
constexpr int kWaves = 8;  // of a workgroup, splitting K

// A wave has kAhead blocks of K under way. A turn but the last loads as many, past the end the last
// block again: a load that a branch leaves out would make every wait one for all loads. The last
// turn loads nothing (with its loads one token on 7168 x 7168 12.4 us, 10.9 without; seven under way: 11.3).
template <bool BF16>
__global__ __launch_bounds__(64 * kWaves, 4) void k_fp8_skinny(Fp8Args a) {
  typedef typename OutElem<BF16>::T E;
  constexpr int kAhead = 4;
  extern __shared__ float scales[];         // [T][blocks], of both operands
  __shared__ float part[kWaves][2][2][64];  // [wave][operand][row of the lane's two][lane]
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), i = lane & 15, q = lane >> 4;
  const int n0 = blockIdx.x * 16, pieces = a.K / 16, blocks = f8_blocks(a.K), own = 2 * q + (i & 1);  // own: piece of a block
  // rows past the last one are read as the last: not stored
  g_f8i4* w0 = (g_f8i4*)(a.w + (int64_t)min(n0 + i / 2, a.N - 1) * a.ld_w);
  g_f8i4* w1 = (g_f8i4*)(a.w + (int64_t)min(n0 + 8 + i / 2, a.N - 1) * a.ld_w);
  g_f8i4* x = (g_f8i4*)(a.x + min(i / 2, a.T - 1) * a.ld_x);
  const float* scale = scales + min(i / 2, a.T - 1) * blocks;
  struct Unit {
    f8i4 w[2], x;
  };
  auto load = [&](Unit& f, int b) {
    b = min(b, blocks - 1);
    const int p = min(b * 8 + own, pieces - 1);
    f.w[0] = w0[p];
    f.w[1] = w1[p];
    f.x = x[p];
  };
  for (int t = 0; t < a.T; ++t)
    for (int b = threadIdx.x; b < blocks; b += 64 * kWaves) scales[t * blocks + b] = a.sx[t * a.ld_sx + b] * a.sw[n0 / kF8Block * a.ld_sw + b];
  Unit f[kAhead];
#pragma unroll
  for (int k = 0; k < kAhead; ++k) load(f[k], wave + k * kWaves);
  // this thread's output (token t, row r), and what it adds
  const int r = threadIdx.x % 16, t = threadIdx.x / 16, n = n0 + r;
  const bool is = t < a.T && n < a.N;
  const float bias = is && a.o.bias ? a.o.bias[n] : 0.f, y = is && a.o.y ? a.o.y[t * a.o.ld_y + n] : 0.f;
  const float res = is && a.o.res ? OutElem<BF16>::load(static_cast<const E*>(a.o.res)[t * a.o.ld_res + n]) : 0.f;
  meet();             // the scales; loads stay under way
  f32x4 acc[2] = {};  // all parities of rows 2 q and 2 q + 1, and 8 on
  auto products = [&](Unit& u, int b) {
    if (b >= blocks) return;
    if (b * 8 + own >= pieces) u.w[0] = u.w[1] = u.x = f8i4{0, 0, 0, 0};  // K ends inside the block
    const bf16x8v lo = f8_to_bf16(u.x[0], u.x[1]), hi = f8_to_bf16(u.x[2], u.x[3]);
    const float sxw = scale[b];
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      f32x4 sum = mfma_bf16(f8_to_bf16(u.w[c][0], u.w[c][1]), lo, f32x4{0.f, 0.f, 0.f, 0.f});
      sum = mfma_bf16(f8_to_bf16(u.w[c][2], u.w[c][3]), hi, sum);
#pragma unroll
      for (int v = 0; v < 4; ++v) acc[c][v] = fmaf(sxw, sum[v], acc[c][v]);
    }
  };
  int b0 = wave;
  for (; b0 + kAhead * kWaves < blocks; b0 += kAhead * kWaves) {
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      products(f[k], b0 + k * kWaves);
      load(f[k], b0 + (k + kAhead) * kWaves);
    }
  }
#pragma unroll
  for (int k = 0; k < kAhead; ++k) products(f[k], b0 + k * kWaves);
#pragma unroll
  for (int c = 0; c < 2; ++c)
#pragma unroll
    for (int v = 0; v < 2; ++v) {
      const float s = of_parity(acc[c][2 * v], acc[c][2 * v + 1]);
      part[wave][c][v][lane] = s + dppf<kDppXor1, 0xF>(0.f, s);
    }
  __syncthreads();
  if (!is) return;
  const float* p = &part[0][r / 8][r % 2][16 * (r % 8 / 2) + 2 * t];
  float v = 0.f;
#pragma unroll
  for (int k = 0; k < kWaves; ++k) v += p[k * 2 * 2 * 64];
  v += bias;
  v += y;
  v += res;
  static_cast<E*>(a.o.out)[t * a.o.ld_out + n] = OutElem<BF16>::rounded(v);
}

}  // namespace

void launch_fp8_matmul(const Fp8Args& a, bool out_bf16, hipStream_t s) {
  const int grid = (a.N - 1) / 16 + 1;
  if (a.T > kSkinnyRows) return launch_fp8_gemm(a, out_bf16, s);
  const size_t lds = sizeof(float) * a.T * f8_blocks(a.K);
  if (out_bf16)
    hipLaunchKernelGGL((k_fp8_skinny<true>), dim3(grid), dim3(64 * kWaves), lds, s, a);
  else
    hipLaunchKernelGGL((k_fp8_skinny<false>), dim3(grid), dim3(64 * kWaves), lds, s, a);
}

}  // namespace moe
