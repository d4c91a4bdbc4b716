// Product of e4m3 codes with a scale for each block of 128, for many tokens: tiles of
// 64 x 64, a wave 32 x 32 of them, through one pair of LDS buffers a block of 128 of K.
#include <hip/hip_runtime.h>

#include "f8_dev.h"
#include "fp8.h"
#include "int8_out.h"

namespace moe {
namespace {

constexpr int kTile = 64;

template <bool BF16>
__global__ __launch_bounds__(256) void k_fp8_gemm(Fp8Args a, int mtiles) {
  typedef typename OutElem<BF16>::T E;
  __shared__ f8i4 sh[2][kTile][9];  // rows 16 bytes longer than a block
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, l16 = lane & 15, q = lane >> 4;
  const int m0 = blockIdx.x % mtiles * kTile, n0 = blockIdx.x / mtiles * kTile;
  const int wm = wave / 2 * 32, wn = wave % 2 * 32, pieces = a.K / 16, blocks = f8_blocks(a.K);
  f32x4 acc[2][2];
  for (int i = 0; i < 2; ++i)
    for (int j = 0; j < 2; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  for (int b = 0; b < blocks; ++b) {
    __syncthreads();
    for (int o = threadIdx.x; o < 2 * kTile * 8; o += 256) {
      const int side = o / (kTile * 8), r = o / 8 % kTile, p = o % 8;
      const uint8_t* row = side == 0 ? a.x + (int64_t)min(m0 + r, a.T - 1) * a.ld_x : a.w + (int64_t)min(n0 + r, a.N - 1) * a.ld_w;
      sh[side][r][p] = b * 8 + p < pieces ? ((g_f8i4*)row)[b * 8 + p] : f8i4{0, 0, 0, 0};
    }
    __syncthreads();
    const float sw = a.sw[(int64_t)(n0 / kF8Block) * a.ld_sw + b];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float s[4];
#pragma unroll
      for (int v = 0; v < 4; ++v) s[v] = a.sx[(int64_t)min(m0 + wm + 16 * i + 4 * q + v, a.T - 1) * a.ld_sx + b] * sw;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        f32x4 sum = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const f8i4 x = sh[0][wm + 16 * i + l16][4 * h + q], w = sh[1][wn + 16 * j + l16][4 * h + q];
#pragma unroll
          for (int e = 0; e < 4; e += 2) sum = mfma_bf16(f8_to_bf16(x[e], x[e + 1]), f8_to_bf16(w[e], w[e + 1]), sum);
        }
#pragma unroll
        for (int v = 0; v < 4; ++v) acc[i][j][v] = fmaf(s[v], sum[v], acc[i][j][v]);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const int64_t t = m0 + wm + 16 * i + 4 * q + v;
        const int n = n0 + wn + 16 * j + l16;
        if (t >= a.T || n >= a.N) continue;
        float o = acc[i][j][v];
        if (a.o.bias) o += a.o.bias[n];
        if (a.o.y) o += a.o.y[t * a.o.ld_y + n];
        if (a.o.res) o += OutElem<BF16>::load(static_cast<const E*>(a.o.res)[t * a.o.ld_res + n]);
        static_cast<E*>(a.o.out)[t * a.o.ld_out + n] = OutElem<BF16>::rounded(o);
      }
}

}  // namespace

void launch_fp8_gemm(const Fp8Args& a, bool out_bf16, hipStream_t s) {
  const int mt = (a.T - 1) / kTile + 1, nt = (a.N - 1) / kTile + 1;
  if (out_bf16)
    hipLaunchKernelGGL((k_fp8_gemm<true>), dim3(mt * nt), dim3(256), 0, s, a, mt);
  else
    hipLaunchKernelGGL((k_fp8_gemm<false>), dim3(mt * nt), dim3(256), 0, s, a, mt);
}

}  // namespace moe
