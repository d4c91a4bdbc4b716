// Product of e4m3 codes with a scale for each block of 128, for up to 16 tokens.
//
//   out[t][n] = sum_b sx[t][b] sw[n / 128][b] sum_{k in b} x[t][k] w[n][k] + ...
//
// The weights are the row operand and the tokens the column operand of the bf16 MFMA, so a
// lane ends with four neighbouring channels of one token. A workgroup takes 16 weight rows
// and all tokens; its waves take blocks of 128 of K in turn and meet in LDS. A block's sum
// starts from zero and is added to the wave's with both scales, in fp32.
//
// Bound: the weights' bytes, which go from memory to registers with 16-byte loads.
#include <hip/hip_runtime.h>

#include "f8_dev.h"
#include "fp8.h"
#include "int8_out.h"

namespace moe {
namespace {

constexpr int kSkinnyRows = 16;
constexpr int kWaves = 8;  // of a workgroup, splitting K

template <bool BF16>
__global__ __launch_bounds__(64 * kWaves) void k_fp8_skinny(Fp8Args a) {
  typedef typename OutElem<BF16>::T E;
  __shared__ f32x4 part[kWaves][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, i = lane & 15, q = lane >> 4;
  const int n0 = blockIdx.x * 16, pieces = a.K / 16, blocks = f8_blocks(a.K);
  // rows past the last one are read as the last: not stored
  g_f8i4* w = (g_f8i4*)(a.w + (int64_t)min(n0 + i, a.N - 1) * a.ld_w);
  g_f8i4* x = (g_f8i4*)(a.x + min(i, a.T - 1) * a.ld_x);
  const float* sx = a.sx + min(i, a.T - 1) * a.ld_sx;
  const float* sw = a.sw + n0 / kF8Block * a.ld_sw;
  f32x4 acc = {0.f, 0.f, 0.f, 0.f};
  for (int b = wave; b < blocks; b += kWaves) {
    f8i4 wv[2], xv[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int p = b * 8 + 4 * h + q;
      wv[h] = w[min(p, pieces - 1)];
      xv[h] = x[min(p, pieces - 1)];
    }
    const float scale = sx[b] * sw[b];
    f32x4 sum = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (b * 8 + 4 * h + q >= pieces) wv[h] = xv[h] = f8i4{0, 0, 0, 0};
#pragma unroll
      for (int s = 0; s < 4; s += 2) sum = mfma_bf16(f8_to_bf16(wv[h][s], wv[h][s + 1]), f8_to_bf16(xv[h][s], xv[h][s + 1]), sum);
    }
#pragma unroll
    for (int v = 0; v < 4; ++v) acc[v] = fmaf(scale, sum[v], acc[v]);
  }
  part[wave][lane] = acc;
  __syncthreads();
  const int t = threadIdx.x / 16, r = threadIdx.x % 16, n = n0 + r;
  if (t >= a.T || n >= a.N) return;
  const float* p = reinterpret_cast<const float*>(&part[0][16 * (r / 4) + t]) + r % 4;
  float v = 0.f;
#pragma unroll
  for (int k = 0; k < kWaves; ++k) v += p[k * 64 * 4];
  if (a.o.bias) v += a.o.bias[n];
  if (a.o.y) v += a.o.y[t * a.o.ld_y + n];
  if (a.o.res) v += OutElem<BF16>::load(static_cast<const E*>(a.o.res)[t * a.o.ld_res + n]);
  static_cast<E*>(a.o.out)[t * a.o.ld_out + n] = OutElem<BF16>::rounded(v);
}

}  // namespace

void launch_fp8_matmul(const Fp8Args& a, bool out_bf16, hipStream_t s) {
  if (a.T > kSkinnyRows) return launch_fp8_gemm(a, out_bf16, s);
  const int blocks = (a.N - 1) / 16 + 1;
  if (out_bf16)
    hipLaunchKernelGGL((k_fp8_skinny<true>), dim3(blocks), dim3(64 * kWaves), 0, s, a);
  else
    hipLaunchKernelGGL((k_fp8_skinny<false>), dim3(blocks), dim3(64 * kWaves), 0, s, a);
}

}  // namespace moe
