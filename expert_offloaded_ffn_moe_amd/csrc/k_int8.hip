// 8-bit matrix product for few rows: out[t][n] = sum_k x[t][k] w[n][k] on
// v_mfma_i32_16x16x64_i8, and the gated form h = silu(x Wg) (x Wu).
//
// Lane layout of the 16x16x64 MFMA: lane l supplies 16 bytes of row l % 16 of each
// operand at K offset 16 (l / 16), and receives the four sums of column l % 16 and rows
// 4 (l / 16) .. + 3. The weights are the row operand and the tokens the column operand,
// so a lane ends with four neighbouring outputs of one token.
//
// Bound: the weights' bytes. A workgroup takes 16 weight rows (gated: 8 gate rows and
// their 8 up rows) and 16 TT tokens; its waves split K, each reading blocks of kStep
// 64-byte steps, and meet in LDS. Weights go from memory to registers with 16-byte loads,
// all loads of a block before its products; the activations, which every workgroup
// reads, come from cache the same way.
#include <hip/hip_runtime.h>

#include "int8_out.h"

namespace moe {
namespace {

constexpr int kSkinnyRows = 16;  // tokens up to which these kernels run
constexpr int kSkinnyWaves = 8;  // waves of a workgroup, splitting K
constexpr int kStep = 4;         // 64-byte K steps of a wave's load block

__device__ __forceinline__ i32x4 mfma16(const i32x4& a, const i32x4& b, const i32x4& c) {
  return __builtin_amdgcn_mfma_i32_16x16x64_i8(a, b, c, 0, 0, 0);
}

template <int TT, bool GATED, bool BF16>
__global__ __launch_bounds__(64 * kSkinnyWaves) void k_int8_skinny(Int8Args a) {
  __shared__ i32x4 part[kSkinnyWaves][TT][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int i = lane & 15, q = lane >> 4;
  constexpr int kN = GATED ? 8 : 16;  // outputs of a workgroup
  const int n0 = blockIdx.x * kN, t0 = blockIdx.y * 16 * TT;
  // this lane's weight row (rows past the last one are read as the last: not stored)
  const int64_t wrow = GATED ? (int64_t)min(n0 + (i & 7), a.N - 1) + (i < 8 ? 0 : a.N) : min(n0 + i, a.N - 1);
  gi32x4* w = (gi32x4*)(a.w + wrow * a.ld_w);
  gi32x4* x[TT];
#pragma unroll
  for (int tt = 0; tt < TT; ++tt) x[tt] = (gi32x4*)(a.x + min(t0 + 16 * tt + i, a.T - 1) * a.ld_x);
  const int pieces = a.K / 16;  // 16-byte pieces of a row; lane q of a step takes piece 4 step + q
  i32x4 acc[TT];
#pragma unroll
  for (int tt = 0; tt < TT; ++tt) acc[tt] = i32x4{0, 0, 0, 0};
  const int blocks = (pieces + 4 * kStep - 1) / (4 * kStep);
  for (int b = wave; b < blocks; b += kSkinnyWaves) {
    i32x4 wv[kStep], xv[TT][kStep];
    const int p0 = b * 4 * kStep + q;
#pragma unroll
    for (int s = 0; s < kStep; ++s) wv[s] = w[min(p0 + 4 * s, pieces - 1)];
#pragma unroll
    for (int s = 0; s < kStep; ++s)
#pragma unroll
      for (int tt = 0; tt < TT; ++tt) xv[tt][s] = x[tt][min(p0 + 4 * s, pieces - 1)];
#pragma unroll
    for (int s = 0; s < kStep; ++s) {
      if (p0 + 4 * s >= pieces) wv[s] = i32x4{0, 0, 0, 0};
#pragma unroll
      for (int tt = 0; tt < TT; ++tt) acc[tt] = mfma16(wv[s], xv[tt][s], acc[tt]);
    }
  }
#pragma unroll
  for (int tt = 0; tt < TT; ++tt) part[wave][tt][lane] = acc[tt];
  __syncthreads();
  // output (token tile tt, token j, row r): component r % 4 of lane 16 (r / 4) + j
  for (int o = threadIdx.x; o < TT * 16 * kN; o += 64 * kSkinnyWaves) {
    const int r = o % kN, j = o / kN % 16, tt = o / (16 * kN);
    const int t = t0 + 16 * tt + j, n = n0 + r;
    if (t >= a.T || n >= a.N) continue;
    const int* p = reinterpret_cast<const int*>(&part[0][tt][16 * (r / 4) + j]) + r % 4;
    int sum = 0;
#pragma unroll
    for (int v = 0; v < kSkinnyWaves; ++v) sum += p[v * TT * 64 * 4];
    if (GATED) {  // the up row is 8 rows on: lane 32 further
      int up = 0;
#pragma unroll
      for (int v = 0; v < kSkinnyWaves; ++v) up += p[v * TT * 64 * 4 + 32 * 4];
      static_cast<float*>(a.o.out)[t * a.o.ld_out + n] =
          gated_value(sum, up, a.o.sx[t], a.o.sw[n], a.o.sw[n + a.N]);
    } else {
      int8_store<BF16>(a.o, t, n, a.o.sx[t], a.o.sw[n], sum);
    }
  }
}

template <bool GATED, bool BF16>
void skinny(const Int8Args& a, hipStream_t s) {
  const int nb = (a.N - 1) / (GATED ? 8 : 16) + 1;
#define SKINNY(TT) \
  hipLaunchKernelGGL((k_int8_skinny<TT, GATED, BF16>), dim3(nb, (a.T - 1) / (16 * TT) + 1), dim3(64 * kSkinnyWaves), 0, s, a)
  if (a.T <= 16)
    SKINNY(1);
  else if (a.T <= 32)
    SKINNY(2);
  else
    SKINNY(4);
#undef SKINNY
}

}  // namespace

void launch_int8_matmul(const Int8Args& a, bool out_bf16, hipStream_t s) {
  if (a.T > kSkinnyRows) return launch_int8_gemm(a, out_bf16, s);
  if (out_bf16)
    skinny<false, true>(a, s);
  else
    skinny<false, false>(a, s);
}

void launch_int8_gated(const Int8Args& a, hipStream_t s) {
  if (a.T > kSkinnyRows) return launch_int8_gated_gemm(a, s);
  skinny<true, false>(a, s);
}

}  // namespace moe
