// 8-bit matrix product for up to 16 rows: out[t][n] = sum_k x[t][k] w[n][k] on
// v_mfma_i32_16x16x64_i8, and the gated form h = silu(x Wg) (x Wu).
//
// Lane layout of the 16x16x64 MFMA: lane l supplies 16 bytes of row l % 16 of each
// operand at K offset 16 (l / 16), and receives the four sums of column l % 16 and rows
// 4 (l / 16) .. + 3. The weights are the row operand and the tokens the column operand,
// so a lane ends with four neighbouring outputs of one token.
//
// Bound: the weights' bytes. A workgroup takes CT blocks of 16 weight rows (gated: 8 gate
// rows and their 8 up rows) and all tokens; its eight waves split K, each reading blocks of
// two 64-byte steps, and meet in LDS. Weights go from memory to registers with 16-byte loads,
// all loads of a block before its products; the activations, which every workgroup reads,
// come from cache the same way. Measured with inputs and outputs all from HBM (a plain copy:
// 5.1 TB/s): one token on 7168 x 7168 10.9 us (4.7 TB/s), on 4096 x 7168 8.1, 16 tokens 9.4 us (one
// set of buffers in a loop: 9.6, 5.9 and 8.2). Four steps a block: 7% longer for the first;
// sixteen waves: the same within 3%, four: 20% longer; the next block's loads ahead of this
// one's products, in twice the registers: 15% longer.
#include <hip/hip_runtime.h>

#include "codes.h"
#include "int8_out.h"
#include "wave.h"

namespace moe {
namespace {

// Tokens up to which these kernels run. 16 tokens: 4096 x 7168 8.3 us (in tiles 8.2), 4096 x
// 2048 4.1 (5.3), gated blocks of 7168 / 2048 and 2048 / 768 17.4 and 9.2 (19.2, 10.1); two
// token blocks a wave would take 20.0 us for 32 tokens on 7168 x 7168 (10.8). Long rows of many
// channels, where two blocks a workgroup fill the chip, go to tiles sooner: 7168 x 7168 12.1
// (tiles 11.8), 13.3 (12.1) us for 12 and 16 tokens, 6144 x 4096 8.4 (7.2) and 14336 x 4096 16.9
// (15.1 to 15.7) for 16, but 10000 x 2064 7.2 (8.1), and 7168 x 7168 12.0 (12.3) for 9.
constexpr int kSkinnyRows = 16, kSkinnyRowsWide = 12, kWideK = 4096;
constexpr int kWaves = 8;  // of a workgroup, splitting K
constexpr int kStep = 2;   // 64-byte K steps of a wave's load block

__device__ __forceinline__ i32x4 mfma16(const i32x4& a, const i32x4& b, const i32x4& c) {
  return __builtin_amdgcn_mfma_i32_16x16x64_i8(a, b, c, 0, 0, 0);
}

template <int CT, bool GATED, bool BF16>
__global__ __launch_bounds__(64 * kWaves) void k_int8_skinny(Int8Args a) {
  __shared__ i32x4 part[kWaves][CT][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int i = lane & 15, q = lane >> 4;
  constexpr int kN = GATED ? 8 : 16;  // outputs of a block of weight rows
  const int n0 = blockIdx.x * kN * CT;
  // this lane's weight rows (rows past the last one are read as the last: not stored)
  gi32x4* w[CT];
#pragma unroll
  for (int c = 0; c < CT; ++c) {
    const int n = n0 + c * kN + (GATED ? i & 7 : i);
    w[c] = (gi32x4*)(a.w + ((int64_t)min(n, a.N - 1) + (GATED && i >= 8 ? a.N : 0)) * a.ld_w);
  }
  gi32x4* x = (gi32x4*)(a.x + min(i, a.T - 1) * a.ld_x);
  const int pieces = a.K / 16;  // 16-byte pieces of a row; lane q of a step takes piece 4 step + q
  i32x4 acc[CT];
#pragma unroll
  for (int c = 0; c < CT; ++c) acc[c] = i32x4{0, 0, 0, 0};
  // this thread's output (block c, token t, row r), one at most, and what it adds
  static_assert(CT * 16 * kN <= 64 * kWaves, "an output a thread");
  const int r = threadIdx.x % kN, oc = threadIdx.x / kN % CT, t = threadIdx.x / (kN * CT), n = n0 + oc * kN + r;
  const bool is = t < a.T && n < a.N;
  float sx = 0.f, su = 0.f;
  OutTerms<BF16> terms;
  if (is) {
    sx = a.o.sx[t];
    if (GATED) {
      terms.sw = a.o.sw[n];
      su = a.o.sw[n + a.N];
    } else {
      terms.load(a.o, t, n);
    }
  }
  const int blocks = (pieces + 4 * kStep - 1) / (4 * kStep);
  for (int b = wave; b < blocks; b += kWaves) {
    i32x4 wv[CT][kStep], xv[kStep];
    const int p0 = b * 4 * kStep + q;
#pragma unroll
    for (int s = 0; s < kStep; ++s)
#pragma unroll
      for (int c = 0; c < CT; ++c) wv[c][s] = w[c][min(p0 + 4 * s, pieces - 1)];
#pragma unroll
    for (int s = 0; s < kStep; ++s) xv[s] = x[min(p0 + 4 * s, pieces - 1)];
    __builtin_amdgcn_sched_barrier(0);  // every load before the first product: the compiler put one behind it (9.3 us, 11.0)
#pragma unroll
    for (int s = 0; s < kStep; ++s) {
      if (p0 + 4 * s >= pieces) xv[s] = i32x4{0, 0, 0, 0};
#pragma unroll
      for (int c = 0; c < CT; ++c) acc[c] = mfma16(wv[c][s], xv[s], acc[c]);
    }
  }
#pragma unroll
  for (int c = 0; c < CT; ++c) part[wave][c][lane] = acc[c];
  __syncthreads();
  if (!is) return;
  // its sum: component r % 4 of lane 16 (r / 4) + t
  const int* p = reinterpret_cast<const int*>(&part[0][oc][16 * (r / 4) + t]) + r % 4;
  int sum = 0;
#pragma unroll
  for (int v = 0; v < kWaves; ++v) sum += p[v * CT * 64 * 4];
  if (GATED) {  // the up row is 8 rows on: lane 32 further
    int up = 0;
#pragma unroll
    for (int v = 0; v < kWaves; ++v) up += p[v * CT * 64 * 4 + 32 * 4];
    static_cast<float*>(a.o.out)[t * a.o.ld_out + n] = gated_value(sum, up, sx, terms.sw, su);
  } else {
    terms.store(a.o, t, n, sx, sum);
  }
}

// The second half of the gated block for up to 16 tokens: as k_int8_skinny, with the
// activations' codes formed in LDS from h first, while the first weights are on their way.
// Each workgroup reads and codes all of h, which costs less than a launch of its own for as
// long as h is small: calls of one token of the 7168/2048 block 12.3 us (with the codes in a
// launch of their own 14.7), of 16 of the 2048/768 one 11.3 (15.0), but of 16 of the first,
// 32768 elements, 17.4 (17.0). A row of h is shared by kWaves / T waves at least, in registers
// of kHeld elements a lane.
constexpr int kHeld = 32;
constexpr int kDownTokens = 16, kDownElements = 16384;

__host__ __device__ constexpr int waves_per_row(int T) { return T == 1 ? 8 : T == 2 ? 4 : T <= 4 ? 2 : 1; }

template <int CT, bool BF16>
__global__ __launch_bounds__(64 * kWaves) void k_int8_down(Int8Args a, const float* h) {
  extern __shared__ __attribute__((aligned(16))) uint8_t codes[];  // [T][K + 16]: rows on different banks
  __shared__ i32x4 part[kWaves][CT][64];
  __shared__ float scale[kDownTokens];
  __shared__ uint32_t tops[kWaves];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int i = lane & 15, q = lane >> 4;
  const int n0 = blockIdx.x * 16 * CT, ld = a.K + 16;
  gi32x4* w[CT];
#pragma unroll
  for (int c = 0; c < CT; ++c) w[c] = (gi32x4*)(a.w + min(n0 + 16 * c + i, a.N - 1) * a.ld_w);
  const int pieces = a.K / 16, blocks = (pieces + 4 * kStep - 1) / (4 * kStep);
  // two blocks of weights ahead: all of them for K up to 2048
  struct Weights {
    i32x4 v[CT][kStep];
  };
  auto load = [&](Weights& f, int b) {
#pragma unroll
    for (int s = 0; s < kStep; ++s)
#pragma unroll
      for (int c = 0; c < CT; ++c) f.v[c][s] = w[c][min(b * 4 * kStep + 4 * s + q, pieces - 1)];
  };
  Weights w0, w1;
  load(w0, wave);
  load(w1, wave + kWaves);
  // this thread's output (block c, token t, row r), 512 of them at most, and what it adds
  static_assert(CT * 16 * kDownTokens <= 64 * kWaves, "an output a thread");
  const int out_r = threadIdx.x % 16, out_c = threadIdx.x / 16 % CT, out_t = threadIdx.x / (16 * CT);
  const int out_n = n0 + out_c * 16 + out_r;
  const bool out_is = out_t < a.T && out_n < a.N;
  OutTerms<BF16> terms;
  if (out_is) terms.load(a.o, out_t, out_n);

  const int wpr = waves_per_row(a.T), part_of_row = (wave % wpr) * 64 + lane;
  for (int r0 = 0; r0 < a.T; r0 += kWaves / wpr) {
    const int row = r0 + wave / wpr;
    const bool mine = row < a.T;
    float v[kHeld];
    uint32_t top = 0;
    if (mine) {
#pragma unroll
      for (int k = 0; k < kHeld / 4; ++k) {
        const int j = 4 * (part_of_row + k * 64 * wpr);
        const float4 f = j < a.K ? *reinterpret_cast<const float4*>(h + (int64_t)row * a.K + j) : float4{0.f, 0.f, 0.f, 0.f};
        v[4 * k] = f.x;
        v[4 * k + 1] = f.y;
        v[4 * k + 2] = f.z;
        v[4 * k + 3] = f.w;
#pragma unroll
        for (int e = 0; e < 4; ++e) top = max(top, abs_bits(v[4 * k + e]));
      }
    }
    top = wave_max_u(top);
    if (wpr > 1) {  // one round of rows then
      if (lane == 0) tops[wave] = top;
      __syncthreads();
      for (int k = 0; k < wpr; ++k) top = max(top, tops[wave / wpr * wpr + k]);
    }
    if (!mine) continue;
    const float size = __uint_as_float(top);
    const bool none = top >= kNotFinite || top < kNoCodes;
    if (lane == 0) scale[row] = code_scale(top, (double)size);  // every wave of the row the same
    const Quotient64 quot(none ? 1.0 : (double)size);
    const uint32_t keep = none ? 0u : ~0u;
#pragma unroll
    for (int k = 0; k < kHeld / 4; ++k) {
      const int j = 4 * (part_of_row + k * 64 * wpr);
      if (j >= a.K) break;
      uint32_t c = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) c |= quot.code((double)v[4 * k + e]) << (8 * e);
      *reinterpret_cast<uint32_t*>(codes + row * ld + j) = c & keep;
    }
  }
  __syncthreads();

  const i32x4* x = reinterpret_cast<const i32x4*>(codes + min(i, a.T - 1) * ld);
  i32x4 acc[CT];
#pragma unroll
  for (int c = 0; c < CT; ++c) acc[c] = i32x4{0, 0, 0, 0};
  auto products = [&](const Weights& f, int b) {
#pragma unroll
    for (int s = 0; s < kStep; ++s) {
      const int p = b * 4 * kStep + 4 * s + q;
      i32x4 xv = x[min(p, pieces - 1)];
      if (p >= pieces) xv = i32x4{0, 0, 0, 0};
#pragma unroll
      for (int c = 0; c < CT; ++c) acc[c] = mfma16(f.v[c][s], xv, acc[c]);
    }
  };
  for (int b = wave; b < blocks; b += 2 * kWaves) {  // a block past the last is of zeros
    products(w0, b);
    if (b + 2 * kWaves < blocks) load(w0, b + 2 * kWaves);
    products(w1, b + kWaves);
    if (b + 3 * kWaves < blocks) load(w1, b + 3 * kWaves);
  }
#pragma unroll
  for (int c = 0; c < CT; ++c) part[wave][c][lane] = acc[c];
  __syncthreads();
  if (!out_is) return;
  const int* p = reinterpret_cast<const int*>(&part[0][out_c][16 * (out_r / 4) + out_t]) + out_r % 4;
  int sum = 0;
#pragma unroll
  for (int v = 0; v < kWaves; ++v) sum += p[v * CT * 64 * 4];
  terms.store(a.o, out_t, out_n, scale[out_t], sum);
}

// Two blocks a workgroup share each load of the activations, if that leaves three quarters of
// the 256 CUs a workgroup: 12 tokens on 7168 x 7168 12.4 us (one block: 15.1), on 4096 x 2048
// 16 tokens take 5.9 us that way (4.8); for one token it makes no difference.
bool two_blocks(int blocks) { return blocks >= 2 * 192; }

template <bool GATED, bool BF16>
void skinny(const Int8Args& a, hipStream_t s) {
  const int blocks = (a.N - 1) / (GATED ? 8 : 16) + 1;
  if (two_blocks(blocks))
    hipLaunchKernelGGL((k_int8_skinny<2, GATED, BF16>), dim3((blocks - 1) / 2 + 1), dim3(64 * kWaves), 0, s, a);
  else
    hipLaunchKernelGGL((k_int8_skinny<1, GATED, BF16>), dim3(blocks), dim3(64 * kWaves), 0, s, a);
}

}  // namespace

void launch_int8_matmul(const Int8Args& a, bool out_bf16, hipStream_t s) {
  const bool wide = a.K >= kWideK && two_blocks((a.N - 1) / 16 + 1);
  if (a.T > (wide ? kSkinnyRowsWide : kSkinnyRows)) return launch_int8_gemm(a, out_bf16, s);
  if (out_bf16)
    skinny<false, true>(a, s);
  else
    skinny<false, false>(a, s);
}

bool int8_down_fits(int T, int K) {
  return T <= kDownTokens && (int64_t)T * K <= kDownElements && K <= 64 * kHeld * waves_per_row(T);
}

void launch_int8_down(const Int8Args& a, const float* h, bool out_bf16, hipStream_t s) {
  const int blocks = (a.N - 1) / 16 + 1;
  const size_t lds = (size_t)a.T * (a.K + 16);
#define DOWN(CT, BF16) \
  hipLaunchKernelGGL((k_int8_down<CT, BF16>), dim3((blocks - 1) / CT + 1), dim3(64 * kWaves), lds, s, a, h)
  if (two_blocks(blocks)) {
    if (out_bf16)
      DOWN(2, true);
    else
      DOWN(2, false);
  } else {
    if (out_bf16)
      DOWN(1, true);
    else
      DOWN(1, false);
  }
#undef DOWN
}

void launch_int8_gated(const Int8Args& a, hipStream_t s) {
  if (a.T > kSkinnyRows) return launch_int8_gated_gemm(a, s);
  skinny<true, false>(a, s);
}

}  // namespace moe
