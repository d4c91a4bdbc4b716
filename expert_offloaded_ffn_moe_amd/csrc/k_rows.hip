// Row kernels: root-mean-square norm with the residual's addition, and the 8-bit
// codes of a row.
//
//   s_j = act(x_j + r_j),  p_j = s_j g_j,  n_j = p_j / sqrt(mean(s^2) + eps)
//   code_j = round half even(127 p_j / max|p|),  scale = max|p| / (127 sqrt(mean(s^2) + eps))
//
// The row's root mean square divides every n_j alike, so the codes are those of p and
// do not depend on its rounding. With bf16 activations p (8 x 8 bits of mantissa) and
// 127 p (23 bits) are exact in fp32, and the quotient is rounded correctly by Markstein's
// two-step correction of a product with a correctly rounded reciprocal (IBM J. Res.
// Dev. 34, 1990): a code differs from the definition's only where the quotient's own fp32
// rounding reaches a half, which it cannot (the quotient is either k + 1/2 or at least
// 2^-17 from it at |code| >= 64, less below in step with the spacing of fp32). With fp32
// activations the same steps run in fp64. mean(s^2) is summed in fp64: squares of large
// activations would leave fp32's range.
//
// One pass: a row is held in registers between the sums and the outputs, so each input
// is read once and each output written once. The bound is the bytes, and for a few rows
// the latency of a load, two reductions and a store.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <type_traits>

#include "codes.h"
#include "dense.h"
#include "wave.h"

namespace moe {
namespace {

constexpr int kChunk = 8;  // elements of a row that a thread takes at a time

// Rows may start at any element: 16-byte accesses at the element's alignment, which
// gfx950 performs as one access.
struct __attribute__((packed, aligned(2))) Bf16x8 {
  uint32_t v[4];
};
struct __attribute__((packed, aligned(4))) F32x4 {
  float v[4];
};
struct __attribute__((packed, aligned(1))) I8x8 {
  uint32_t v[2];
};

__device__ __forceinline__ float bf16_value(uint16_t b) { return __uint_as_float((uint32_t)b << 16); }

// round to nearest even; a NaN stays one
__device__ __forceinline__ uint16_t to_bf16(float f) {
  const uint32_t u = __float_as_uint(f);
  if ((u & 0x7FFFFFFFu) > 0x7F800000u) return (uint16_t)((u >> 16) | 0x40u);
  return (uint16_t)((u + 0x7FFFu + ((u >> 16) & 1u)) >> 16);
}

// Eight elements as loaded, and their values.
template <typename E>
struct Raw;
template <>
struct Raw<uint16_t> {
  Bf16x8 w;
  __device__ __forceinline__ void load(const uint16_t* p, int n) {
    if (n >= kChunk) {
      w = *reinterpret_cast<const Bf16x8*>(p);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        w.v[i] = (2 * i < n ? (uint32_t)p[2 * i] : 0u) | (2 * i + 1 < n ? (uint32_t)p[2 * i + 1] << 16 : 0u);
    }
  }
  __device__ __forceinline__ void values(float* v) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w.v[i] << 16);
      v[2 * i + 1] = __uint_as_float(w.v[i] & 0xFFFF0000u);
    }
  }
};
template <>
struct Raw<float> {
  F32x4 a, b;
  __device__ __forceinline__ void load(const float* p, int n) {
    if (n >= kChunk) {
      a = reinterpret_cast<const F32x4*>(p)[0];
      b = reinterpret_cast<const F32x4*>(p)[1];
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        a.v[i] = i < n ? p[i] : 0.f;
        b.v[i] = 4 + i < n ? p[4 + i] : 0.f;
      }
    }
  }
  __device__ __forceinline__ void values(float* v) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = a.v[i];
      v[4 + i] = b.v[i];
    }
  }
};

__device__ __forceinline__ void store8(uint16_t* p, int n, const float* v) {
  if (n >= kChunk) {
    Bf16x8 w;
#pragma unroll
    for (int i = 0; i < 4; ++i) w.v[i] = (uint32_t)to_bf16(v[2 * i]) | (uint32_t)to_bf16(v[2 * i + 1]) << 16;
    *reinterpret_cast<Bf16x8*>(p) = w;
  } else {
#pragma unroll
    for (int i = 0; i < kChunk; ++i)
      if (i < n) p[i] = to_bf16(v[i]);
  }
}

__device__ __forceinline__ void store8(float* p, int n, const float* v) {
  if (n >= kChunk) {
    F32x4 a, b;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      a.v[i] = v[i];
      b.v[i] = v[4 + i];
    }
    reinterpret_cast<F32x4*>(p)[0] = a;
    reinterpret_cast<F32x4*>(p)[1] = b;
  } else {
#pragma unroll
    for (int i = 0; i < kChunk; ++i)
      if (i < n) p[i] = v[i];
  }
}

template <typename ACT>
struct Act;
template <>
struct Act<uint16_t> {
  typedef float P;  // the type of p, its largest size and the quotient
  static __device__ __forceinline__ float rounded(float f) { return bf16_value(to_bf16(f)); }
};
template <>
struct Act<float> {
  typedef double P;
  static __device__ __forceinline__ float rounded(float f) { return f; }
};

template <int CTRL, int ROWS>
__device__ __forceinline__ double dppd(double v) {  // a lane left out of ROWS keeps 0
  const uint64_t u = __double_as_longlong(v);
  const uint32_t lo = dpp<CTRL, ROWS>(0, (int)(uint32_t)u), hi = dpp<CTRL, ROWS>(0, (int)(uint32_t)(u >> 32));
  return __longlong_as_double((int64_t)((uint64_t)hi << 32 | lo));
}

__device__ __forceinline__ double lane63(double v) {
  const uint64_t u = __double_as_longlong(v);
  const uint32_t lo = __builtin_amdgcn_readlane((int)(uint32_t)u, 63);
  const uint32_t hi = __builtin_amdgcn_readlane((int)(uint32_t)(u >> 32), 63);
  return __longlong_as_double((int64_t)((uint64_t)hi << 32 | lo));
}

__device__ __forceinline__ double wave_sum(double v) {
  v += dppd<kDppXor1, 0xF>(v);
  v += dppd<kDppXor2, 0xF>(v);
  v += dppd<kDppHalfMirror, 0xF>(v);
  v += dppd<kDppMirror, 0xF>(v);
  v += dppd<kDppBcast15, 0xA>(v);
  v += dppd<kDppBcast31, 0xC>(v);
  return lane63(v);
}

// largest of non-negative values (a lane left out contributes 0)
__device__ __forceinline__ double wave_max_pos(double v) {
  v = fmax(v, dppd<kDppXor1, 0xF>(v));
  v = fmax(v, dppd<kDppXor2, 0xF>(v));
  v = fmax(v, dppd<kDppHalfMirror, 0xF>(v));
  v = fmax(v, dppd<kDppMirror, 0xF>(v));
  v = fmax(v, dppd<kDppBcast15, 0xA>(v));
  v = fmax(v, dppd<kDppBcast31, 0xC>(v));
  return lane63(v);
}

template <typename P>
struct QuotientOf;
template <>
struct QuotientOf<float> {
  typedef Quotient32 T;
};
template <>
struct QuotientOf<double> {
  typedef Quotient64 T;
};

// 1 / sqrt(m) to about 2^-44: the fp32 estimate and one Newton step in fp64 (m in fp32's range)
__device__ __forceinline__ double rsqrt64(double m) {
  if (!(m > 1e-36 && m < 1e36)) return 1.0 / sqrt(m);
  const double r = (double)__frsqrt_rn((float)m);
  return r * fma(-0.5 * m * r, r, 1.5);
}

// v w 2^e for bf16 v and w, with e the exponent of 1 / rms, at least -128 (-140 for a row whose
// rms is infinite): exact unless the result itself leaves fp32's normal range. Where e < 0 the
// larger factor is scaled: its 8 bits stay whole down to 2^-142, and under that both factors
// are under 2^-14 and the result is 0. Else the smaller one, which stays under 2^8, as |v| 2^e does.
__device__ __forceinline__ float product_far(float v, float w, int e) {
  const bool v_larger = fabsf(v) >= fabsf(w);
  return ldexpf(v_larger ? v : w, min(e, 0)) * ldexpf(v_larger ? w : v, max(e, 0));
}

// A row is taken by a workgroup of up to MAX threads, or, with WAVE, by one of its waves:
// `tpr` threads with NC chunks of 8 elements each (chunk c of thread t: elements
// 8 (t + c tpr) ..). Then follows the row `gridDim.x` workgroups on, whose loads are under way
// before the first is reduced. ADD: 0 none, 1 act, 2 fp32.
template <typename ACT, bool NORM, int ADD, bool WAVE, int MAX, int NC>
__global__ __launch_bounds__(MAX) void k_rows(RowArgs a) {
  typedef typename Act<ACT>::P P;
  typedef typename std::conditional<ADD == 1, ACT, float>::type AddT;
  constexpr int kRows = WAVE ? MAX / 64 : 1, kMaxWaves = WAVE ? 1 : MAX / 64;
  const int tpr = WAVE ? 64 : NC > 1 ? MAX : (int)blockDim.x, t = WAVE ? threadIdx.x % 64 : threadIdx.x;
  const int step = gridDim.x * kRows;
  int row = WAVE ? blockIdx.x * kRows + (int)threadIdx.x / 64 : blockIdx.x;
  if (WAVE && row >= a.T) return;  // nothing waits for it

  Raw<ACT> x[NC], g[NC];
  Raw<AddT> r[NC];
  auto load = [&](int at) {
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int j = kChunk * (t + c * tpr), n = a.H - j;
      x[c].load(static_cast<const ACT*>(a.x) + at * a.ld_x + j, n);
      if (ADD) r[c].load(static_cast<const AddT*>(a.add) + at * a.ld_add + j, n);
    }
  };
  load(row);
  if (NORM) {
#pragma unroll
    for (int c = 0; c < NC; ++c) g[c].load(static_cast<const ACT*>(a.weight) + kChunk * (t + c * tpr), a.H - kChunk * (t + c * tpr));
  }
  const double inv_h = 1.0 / a.H;
  for (int turn = 0; row < a.T; row += step, turn ^= 1) {
    float v[NC][kChunk], w[NC][kChunk];
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      x[c].values(v[c]);
      if (ADD) {
        float rv[kChunk];
        r[c].values(rv);
#pragma unroll
        for (int i = 0; i < kChunk; ++i) v[c][i] = Act<ACT>::rounded(v[c][i] + rv[i]);
      }
    }
    if (row + step < a.T) load(row + step);
    double sum = 0.0;
    uint32_t top_bits = 0;  // of |p| as fp32: a NaN's are the largest
    P top = 0;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int j = kChunk * (t + c * tpr), n = a.H - j;
      if (NORM) g[c].values(w[c]);
      if (NORM) {
#pragma unroll
        for (int i = 0; i < kChunk; ++i) sum = fma((double)v[c][i], (double)v[c][i], sum);
      }
      if (ADD && a.x_out && n > 0) store8(static_cast<ACT*>(a.x_out) + row * a.ld_x_out + j, n, v[c]);
      if (!NORM || a.q) {
#pragma unroll
        for (int i = 0; i < kChunk; ++i) {
          const P p = NORM ? (P)v[c][i] * (P)w[c][i] : (P)v[c][i];
          top_bits = max(top_bits, abs_bits((float)p));
          if (NORM && sizeof(P) == 8) top = fmax((double)top, fabs((double)p));
        }
      }
    }
    if (NORM) sum = wave_sum(sum);
    if (!NORM || a.q) {
      top_bits = wave_max_u(top_bits);
      if (NORM && sizeof(P) == 8) top = wave_max_pos(top);
    }
    if (!WAVE) {
      // two sets, so that a wave that is a row ahead writes another than the others read
      __shared__ double part_sum[2][kMaxWaves];
      __shared__ uint32_t part_bits[2][kMaxWaves];
      __shared__ P part_top[2][kMaxWaves];
      if (t % 64 == 0) {
        part_sum[turn][t / 64] = sum;
        part_bits[turn][t / 64] = top_bits;
        part_top[turn][t / 64] = top;
      }
      __syncthreads();
      sum = 0.0;
#pragma unroll
      for (int i = 0; i < kMaxWaves; ++i) {
        if (64 * i >= tpr) break;
        if (NORM) sum += part_sum[turn][i];
        top_bits = max(top_bits, part_bits[turn][i]);
        if (NORM && sizeof(P) == 8) top = fmax((double)top, (double)part_top[turn][i]);
      }
    }
    if (!NORM || sizeof(P) == 4) top = __uint_as_float(top_bits);
    const double rstd = NORM ? rsqrt64(fma(sum, inv_h, (double)a.eps)) : 1.0;
    if (NORM && a.out) {
      const float rs = (float)rstd;
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const int j = kChunk * (t + c * tpr), n = a.H - j;
        float o[kChunk];
#pragma unroll
        for (int i = 0; i < kChunk; ++i)
          o[i] = sizeof(P) == 8 ? (float)((double)v[c][i] * (double)w[c][i] * rstd) : v[c][i] * w[c][i] * rs;
        if (n > 0) store8(static_cast<ACT*>(a.out) + row * a.ld_out + j, n, o);
      }
    }
    if (!NORM || a.q) {
      // A NaN or an infinity in the row: scale NaN and codes 0, so that every product
      // with the row is NaN. A row of (next to) nothing: scale and codes 0.
      if (NORM && !(rstd > 0.0)) top_bits = kNotFinite;
      const bool none = top_bits >= kNotFinite || top_bits < kNoCodes;
      if (t == 0) a.s[row] = code_scale(top_bits, (double)top * rstd);
      const typename QuotientOf<P>::T quot(none ? (P)1 : top);
      const uint32_t keep = none ? 0u : ~0u;
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const int j = kChunk * (t + c * tpr), n = a.H - j;
        uint32_t code[kChunk];
#pragma unroll
        for (int i = 0; i < kChunk; ++i) code[i] = quot.code(NORM ? (P)v[c][i] * (P)w[c][i] : (P)v[c][i]) & keep;
        int8_t* q = a.q + row * a.ld_q + j;
        if (n >= kChunk) {
          I8x8 o;
          o.v[0] = code[0] | code[1] << 8 | code[2] << 16 | code[3] << 24;
          o.v[1] = code[4] | code[5] << 8 | code[6] << 16 | code[7] << 24;
          *reinterpret_cast<I8x8*>(q) = o;
        } else {
#pragma unroll
          for (int i = 0; i < kChunk; ++i)
            if (i < n) q[i] = (int8_t)code[i];
        }
      }
    }
    // bf16: v w is exact in fp32 where |v| <= sqrt(H) / rstd and |w| keep it under 2^127; where it
    // falls among the subnormals, it is off by 2^-150 and n by 2^-140, 1/64 of what n's own
    // rounding to bf16's subnormals may be. Elsewhere the norm is formed once more, behind
    // the usual stores, which costs one row of 7168 0.09 us (chosen ahead of them: 0.15).
    if (NORM && sizeof(P) == 4 && a.out) {
      uint32_t top_w = 0;  // of this thread's |weight|
#pragma unroll
      for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int i = 0; i < kChunk; ++i) top_w = max(top_w, abs_bits(w[c][i]));
      if (__builtin_expect(!(rstd >= 0x1p-60 && rstd <= 0x1p10 && top_w < (127u + 60u) << 23), 0)) {
        const int e = rstd < 0x1p80 ? max(ilogb(rstd), -140) : 0;  // rstd is under 2^75, or NaN
        const float m = (float)ldexp(rstd, -e);
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          const int j = kChunk * (t + c * tpr), n = a.H - j;
          float o[kChunk];
#pragma unroll
          for (int i = 0; i < kChunk; ++i) o[i] = product_far(v[c][i], w[c][i], e) * m;
          if (n > 0) store8(static_cast<ACT*>(a.out) + row * a.ld_out + j, n, o);
        }
      }
    }
  }
}

// Rows of up to 512 elements take a wave each (8192 rows of 512, norm with all outputs: 10.8
// us, a workgroup each 21.4), of up to 4096 as many waves as hold them at a chunk a thread
// (4096 rows of 2048: 18.2 us, a wave of four chunks 23.5; 2048 rows of 2560: 14.8 us, eight
// waves of two chunks 20.6), longer ones 8 or 16 waves at two chunks a thread (2048 rows of
// 7168: 35.8 us, with one chunk a thread 36.6, with four 43, and on the seven waves that
// would hold them 42). The norm runs 16 waves a CU, which go on to further rows, their loads a
// row ahead (twice as many: 37.5 us; one row each: 43 before rows were loaded ahead). That is
// what the registers let on a CU for rows of more than 4096, about half of it for shorter ones,
// and twice of it for fp32 rows of 4097 to 8192, whose halves run one after the other (2048 rows
// of 7168, norm with the sum: 58 us, 4.0 TB/s). fp32 rows above 8192 spill 30 to 62 registers a
// lane (1024 rows of 16384: 106 us, 2.5 TB/s; 2048 of bf16, with codes, 74 us, 5.0 TB/s). The
// codes alone, with fewer registers, take one row each (2048 x 7168 rows: 8.9 us, 10.6 as the
// norm does).
template <typename ACT, bool NORM, int ADD>
void launch(const RowArgs& a, hipStream_t s) {
#define ROWS(WAVE, MAX, NC)                                                                                        \
  {                                                                                                                \
    const int block = WAVE || NC > 1 ? MAX : ((a.H - 1) / (64 * kChunk) + 1) * 64;                                 \
    const int all = WAVE ? (a.T - 1) / (MAX / 64) + 1 : a.T;                                                       \
    const int grid = NORM ? std::min(all, 128 * 2048 / block) : all;                                               \
    hipLaunchKernelGGL((k_rows<ACT, NORM, ADD, WAVE, MAX, NC>), dim3(grid), dim3(block), 0, s, a);                 \
  }
  if (a.H <= 512)
    ROWS(true, 256, 1)
  else if (a.H <= 4096)
    ROWS(false, 512, 1)
  else if (a.H <= 8192)
    ROWS(false, 512, 2)
  else
    ROWS(false, 1024, 2)
#undef ROWS
}

template <typename ACT>
void launch_norm(const RowArgs& a, hipStream_t s) {
  if (!a.add)
    launch<ACT, true, 0>(a, s);
  else if (a.add_f32 && sizeof(ACT) == 2)
    launch<ACT, true, 2>(a, s);
  else
    launch<ACT, true, 1>(a, s);
}

}  // namespace

void launch_rms_norm(const RowArgs& a, hipStream_t s) {
  if (a.act_bf16)
    launch_norm<uint16_t>(a, s);
  else
    launch_norm<float>(a, s);
}

void launch_quantize_rows(const RowArgs& a, hipStream_t s) {
  if (a.act_bf16)
    launch<uint16_t, false, 0>(a, s);
  else
    launch<float, false, 0>(a, s);
}

}  // namespace moe
