// 8-bit matrix product for few rows: out[t][n] = sum_k x[t][k] w[n][k] on
// v_mfma_i32_16x16x64_i8, and the gated form h = silu(x Wg) (x Wu).
//
// Lane layout of the 16x16x64 MFMA: lane l supplies 16 bytes of row l % 16 of each
// operand at K offset 16 (l / 16), and receives the four sums of column l % 16 and rows
// 4 (l / 16) .. + 3. The weights are the row operand and the tokens the column operand,
// so a lane ends with four neighbouring outputs of one token.
//
// Bound: the weights' bytes. A workgroup takes CT blocks of 16 weight rows (gated: 8 gate
// rows and their 8 up rows) and 16 TT tokens; its eight waves split K, each reading blocks of
// two 64-byte steps, and meet in LDS. Weights go from memory to registers with 16-byte loads,
// all loads of a block before its products; the activations, which every workgroup reads,
// come from cache the same way. Measured with weights from HBM (a plain copy: 5.1 TB/s): one
// token on 7168 x 7168 10.5 us (4.9 TB/s), gated 2 x 2048 x 7168 6.5 us (4.5 TB/s), 16 tokens
// 14.2 and 8.4 us. Four steps a block: 11.6 us for the first; sixteen waves: the same within
// 3%, four: 13.0.
#include <hip/hip_runtime.h>

#include "int8_out.h"

namespace moe {
namespace {

// Tokens up to which these kernels run. 32 tokens on 4096 x 2048: 5.1 us, in tiles 7.5; on
// 7168 x 7168: 18.6, in tiles 17.4; 64 tokens: 33.6, in tiles 17.3.
constexpr int kSkinnyRows = 32;
constexpr int kWaves = 8;  // of a workgroup, splitting K
constexpr int kStep = 2;   // 64-byte K steps of a wave's load block

__device__ __forceinline__ i32x4 mfma16(const i32x4& a, const i32x4& b, const i32x4& c) {
  return __builtin_amdgcn_mfma_i32_16x16x64_i8(a, b, c, 0, 0, 0);
}

template <int TT, int CT, bool GATED, bool BF16>
__global__ __launch_bounds__(64 * kWaves) void k_int8_skinny(Int8Args a) {
  __shared__ i32x4 part[kWaves][CT][TT][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int i = lane & 15, q = lane >> 4;
  constexpr int kN = GATED ? 8 : 16;  // outputs of a block of weight rows
  const int n0 = blockIdx.x * kN * CT;  // every token is in this workgroup's tiles
  // this lane's weight rows (rows past the last one are read as the last: not stored)
  gi32x4* w[CT];
#pragma unroll
  for (int c = 0; c < CT; ++c) {
    const int n = n0 + c * kN + (GATED ? i & 7 : i);
    w[c] = (gi32x4*)(a.w + ((int64_t)min(n, a.N - 1) + (GATED && i >= 8 ? a.N : 0)) * a.ld_w);
  }
  gi32x4* x[TT];
#pragma unroll
  for (int tt = 0; tt < TT; ++tt) x[tt] = (gi32x4*)(a.x + min(16 * tt + i, a.T - 1) * a.ld_x);
  const int pieces = a.K / 16;  // 16-byte pieces of a row; lane q of a step takes piece 4 step + q
  i32x4 acc[CT][TT];
#pragma unroll
  for (int c = 0; c < CT; ++c)
#pragma unroll
    for (int tt = 0; tt < TT; ++tt) acc[c][tt] = i32x4{0, 0, 0, 0};
  const int blocks = (pieces + 4 * kStep - 1) / (4 * kStep);
  for (int b = wave; b < blocks; b += kWaves) {
    i32x4 wv[CT][kStep], xv[TT][kStep];
    const int p0 = b * 4 * kStep + q;
#pragma unroll
    for (int s = 0; s < kStep; ++s)
#pragma unroll
      for (int c = 0; c < CT; ++c) wv[c][s] = w[c][min(p0 + 4 * s, pieces - 1)];
#pragma unroll
    for (int s = 0; s < kStep; ++s)
#pragma unroll
      for (int tt = 0; tt < TT; ++tt) xv[tt][s] = x[tt][min(p0 + 4 * s, pieces - 1)];
#pragma unroll
    for (int s = 0; s < kStep; ++s) {
      if (p0 + 4 * s >= pieces)
#pragma unroll
        for (int c = 0; c < CT; ++c) wv[c][s] = i32x4{0, 0, 0, 0};
#pragma unroll
      for (int c = 0; c < CT; ++c)
#pragma unroll
        for (int tt = 0; tt < TT; ++tt) acc[c][tt] = mfma16(wv[c][s], xv[tt][s], acc[c][tt]);
    }
  }
#pragma unroll
  for (int c = 0; c < CT; ++c)
#pragma unroll
    for (int tt = 0; tt < TT; ++tt) part[wave][c][tt][lane] = acc[c][tt];
  __syncthreads();
  // output (block c, token tile tt, token j, row r): component r % 4 of lane 16 (r / 4) + j
  for (int o = threadIdx.x; o < CT * TT * 16 * kN; o += 64 * kWaves) {
    const int r = o % kN, c = o / kN % CT, j = o / (kN * CT) % 16, tt = o / (16 * kN * CT);
    const int t = 16 * tt + j, n = n0 + c * kN + r;
    if (t >= a.T || n >= a.N) continue;
    const int* p = reinterpret_cast<const int*>(&part[0][c][tt][16 * (r / 4) + j]) + r % 4;
    constexpr int kWave = CT * TT * 64 * 4;  // ints from one wave's sums to the next's
    int sum = 0;
#pragma unroll
    for (int v = 0; v < kWaves; ++v) sum += p[v * kWave];
    if (GATED) {  // the up row is 8 rows on: lane 32 further
      int up = 0;
#pragma unroll
      for (int v = 0; v < kWaves; ++v) up += p[v * kWave + 32 * 4];
      static_cast<float*>(a.o.out)[t * a.o.ld_out + n] =
          gated_value(sum, up, a.o.sx[t], a.o.sw[n], a.o.sw[n + a.N]);
    } else {
      int8_store<BF16>(a.o, t, n, a.o.sx[t], a.o.sw[n], sum);
    }
  }
}

// Two blocks a workgroup share each load of the activations, if that leaves three quarters of
// the 256 CUs a workgroup: 16 tokens on 7168 x 7168 14.2 us (one block: 16.9), on 4096 x 2048
// 5.2 us (4.0).
template <bool GATED, bool BF16>
void skinny(const Int8Args& a, hipStream_t s) {
  const int blocks = (a.N - 1) / (GATED ? 8 : 16) + 1;
  const bool two = blocks >= 2 * 192;
#define SKINNY(TT, CT) \
  hipLaunchKernelGGL((k_int8_skinny<TT, CT, GATED, BF16>), dim3((blocks - 1) / CT + 1), dim3(64 * kWaves), 0, s, a)
  if (a.T <= 16) {
    if (two)
      SKINNY(1, 2);
    else
      SKINNY(1, 1);
  } else {
    if (two)
      SKINNY(2, 2);
    else
      SKINNY(2, 1);
  }
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
