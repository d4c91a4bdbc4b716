// A whole routed layer for up to 64 tokens on experts of e4m3 codes with a scale for each
// 128 x 128 block: router, top-k, gate and up, silu, down, combine.
//
//   logits = x Wr + b (fp64 sums),  w = softmax of the k largest,  h_e = silu(Wg_e x) (Wu_e x)
//   y[t] = sum_e w[t][e] Wd_e h_e[t]
//
// The router's sums are in fp64, so that which experts a token takes does not turn on the
// order of the sums. A bf16 x fp8 product is exact in the bf16 MFMA (f8_dev.h); an fp32 value
// is the exact sum of three bf16 terms (8 bits of its mantissa each), so that fp32
// activations and the intermediate h, which stays in fp32, take three products.
//
// Every workgroup forms the routing's tables by itself, in LDS: a launch of its own would
// cost more.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "f8_dev.h"
#include "fp8.h"
#include "int8_out.h"
#include "wave.h"

namespace moe {
namespace {

constexpr int kMaxAssign = kF8LayerTokens * kF8LayerTopK;
constexpr int kTileTokens = 16;  // columns of the MFMA

// ----------------------------------------------------------------------------- router

struct __attribute__((packed, aligned(2))) Bf16x8u {
  uint32_t v[4];
};
struct __attribute__((packed, aligned(4))) F32x8u {
  float v[8];
};
__device__ __forceinline__ void values8(const uint16_t* p, float* v) {
  const Bf16x8u w = *reinterpret_cast<const Bf16x8u*>(p);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w.v[i] << 16);
    v[2 * i + 1] = __uint_as_float(w.v[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void values8(const float* p, float* v) {
  const F32x8u w = *reinterpret_cast<const F32x8u*>(p);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = w.v[i];
}

template <int CTRL, int ROWS>
__device__ __forceinline__ double dppd(double v) {  // a lane left out of ROWS adds 0
  const uint64_t u = __double_as_longlong(v);
  const uint32_t lo = dpp<CTRL, ROWS>(0, (int)(uint32_t)u), hi = dpp<CTRL, ROWS>(0, (int)(uint32_t)(u >> 32));
  return __longlong_as_double((int64_t)((uint64_t)hi << 32 | lo));
}
// the sum in lane 63
__device__ __forceinline__ double wave_sum_63(double v) {
  v += dppd<kDppXor1, 0xF>(v);
  v += dppd<kDppXor2, 0xF>(v);
  v += dppd<kDppHalfMirror, 0xF>(v);
  v += dppd<kDppMirror, 0xF>(v);
  v += dppd<kDppBcast15, 0xA>(v);
  v += dppd<kDppBcast31, 0xC>(v);
  return v;
}

// An expert's row a workgroup; its waves take eight neighbours a lane in turn. Also clears
// the counters of the launch that follows.
constexpr int kRouterWaves = 4;
template <typename ACT>
__global__ __launch_bounds__(64 * kRouterWaves) void k_f8_router(Fp8LayerArgs a) {
  __shared__ double part[kRouterWaves][kF8LayerTokens];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, e = blockIdx.x;
  if (e == 0 && threadIdx.x < 64) a.counters[threadIdx.x] = 0u;
  if (a.logits_in) {  // one workgroup for each token then
    if (a.logits)
      for (int i = threadIdx.x; i < a.E; i += 64 * kRouterWaves) a.logits[(int64_t)e * a.E + i] = a.logits_in[(int64_t)e * a.E + i];
    return;
  }
  const ACT* w = static_cast<const ACT*>(a.router_w) + e * a.ld_router;
  for (int t = 0; t < a.T; ++t) {
    const ACT* x = static_cast<const ACT*>(a.x) + t * a.ld_x;
    double sum = 0.0;
    for (int j = 8 * threadIdx.x; j < a.H; j += 8 * 64 * kRouterWaves) {  // H is a multiple of 16
      float wv[8], xv[8];
      values8(w + j, wv);
      values8(x + j, xv);
#pragma unroll
      for (int i = 0; i < 8; ++i) sum = fma((double)wv[i], (double)xv[i], sum);
    }
    sum = wave_sum_63(sum);
    if (lane == 63) part[wave][t] = sum;
  }
  __syncthreads();
  for (int t = threadIdx.x; t < a.T; t += 64 * kRouterWaves) {
    double v = a.router_b ? (double)a.router_b[e] : 0.0;
#pragma unroll
    for (int k = 0; k < kRouterWaves; ++k) v += part[k][t];
    a.logits[(int64_t)t * a.E + e] = (float)v;
  }
}

// ----------------------------------------------------------------------------- routing tables

// Assignments grouped by expert, in ascending order of experts and tokens. Those of weight
// 0 are left out.
struct Route {
  uint64_t mask[kF8LayerExperts];     // the expert's tokens
  float gate[kMaxAssign];             // weights, in grouped order
  uint16_t at[kF8LayerExperts];       // the expert's first place in that order
  uint16_t expert[kF8LayerExperts];   // experts with tokens
  uint16_t tile_expert[kMaxAssign];   // tiles of up to 16 tokens of one expert
  uint8_t tile_first[kMaxAssign];     // the tile's first among its expert's tokens
  uint8_t token[kMaxAssign];          // token of a place
  int experts, tiles;
};

// Orders as the logits do, with NaN before every number; over 0.
__device__ __forceinline__ uint32_t logit_key(float f) {
  const uint32_t u = f == 0.f ? 0u : __float_as_uint(f);
  if (f != f) return ~0u;
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// The k experts of one token by one wave: k rounds of the wave's maximum and the lowest
// expert that has it. Lane l holds experts l, l + 64, ...; lane j ends with slot j.
template <int NV>
__device__ __forceinline__ void choose(const float* logits, int E, int k, int& id, float& w) {
  const int lane = threadIdx.x & 63;
  float f[NV];
  uint32_t key[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    f[i] = logits[min(lane + 64 * i, E - 1)];
    key[i] = lane + 64 * i < E ? logit_key(f[i]) : 0u;
  }
  float mine = 0.f;
  id = 0;
  for (int j = 0; j < k; ++j) {
    uint32_t m = key[0];
#pragma unroll
    for (int i = 1; i < NV; ++i) m = max(m, key[i]);
    m = wave_max_u(m);
    int win = -1;
    float v = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const unsigned long long b = __ballot(key[i] == m);
      if (win < 0 && b != 0ull) {
        win = 64 * i + (int)__builtin_ctzll(b);
        v = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(f[i]), win & 63));
        if ((win & 63) == lane) key[i] = 0u;
      }
    }
    mine = lane == j ? v : mine;
    id = lane == j ? win : id;
  }
  const float top = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(mine), 0));
  const float p = lane < k && mine != -INFINITY ? expf(mine - top) : 0.f;
  const float sum = wave_sum(p);
  w = sum == 0.f ? 0.f : p / sum;  // every logit -infinity: nothing
}

__device__ __forceinline__ void route(const Fp8LayerArgs& a, Route& r, bool writes) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
  const float* logits = a.logits ? a.logits : a.logits_in;
  for (int e = threadIdx.x; e < a.E; e += blockDim.x) r.mask[e] = 0;
  __syncthreads();
  // the slots wait in the tables' arrays, which are filled later: ids in tile_expert, weights in
  // gate, by assignment
  for (int t = wave; t < a.T; t += waves) {
    int id;
    float w;
    const float* row = logits + (int64_t)t * a.E;
    const int nv = (a.E + 63) / 64;
    if (nv <= 2)
      choose<2>(row, a.E, a.k, id, w);
    else if (nv <= 6)
      choose<6>(row, a.E, a.k, id, w);
    else
      choose<16>(row, a.E, a.k, id, w);
    if (lane < a.k) {
      if (w != 0.f) atomicOr(reinterpret_cast<unsigned long long*>(&r.mask[id]), 1ull << t);
      r.tile_expert[t * a.k + lane] = (uint16_t)id;
      r.gate[t * a.k + lane] = w;
      if (writes) {
        if (a.ids) a.ids[t * a.k + lane] = id;
        if (a.gate) a.gate[t * a.k + lane] = w;
      }
    }
  }
  __syncthreads();
  // this thread's assignments, out of the arrays that they wait in
  constexpr int kMine = kMaxAssign / 256;  // of 256 threads and more
  int id[kMine];
  float w[kMine];
  const int n = a.T * a.k;
#pragma unroll
  for (int i = 0; i < kMine; ++i) {
    const int s = threadIdx.x + i * blockDim.x;
    id[i] = s < n ? r.tile_expert[s] : 0;
    w[i] = s < n ? r.gate[s] : 0.f;
  }
  __syncthreads();
  if (wave == 0) {
    int experts = 0, places = 0, tiles = 0;
    for (int e0 = 0; e0 < a.E; e0 += 64) {
      const int e = e0 + lane, c = e < a.E ? __popcll(r.mask[e]) : 0;
      const uint64_t some = __ballot(c > 0);
      const int tc = (c + kTileTokens - 1) / kTileTokens;
      const int incl = wave_incl_scan(c), tincl = wave_incl_scan(tc);
      if (c > 0) {
        r.at[e] = (uint16_t)(places + incl - c);
        r.expert[experts + __popcll(some & ((1ull << lane) - 1))] = (uint16_t)e;
        for (int i = 0; i < tc; ++i) {
          r.tile_expert[tiles + tincl - tc + i] = (uint16_t)e;
          r.tile_first[tiles + tincl - tc + i] = (uint8_t)(kTileTokens * i);
        }
      }
      experts += __popcll(some);
      places += __builtin_amdgcn_readlane(incl, 63);
      tiles += __builtin_amdgcn_readlane(tincl, 63);
    }
    if (lane == 0) {
      r.experts = experts;
      r.tiles = tiles;
    }
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kMine; ++i) {
    if (w[i] == 0.f) continue;
    const int t = (threadIdx.x + i * blockDim.x) / a.k;
    const int p = r.at[id[i]] + __popcll(r.mask[id[i]] & ((1ull << t) - 1));
    r.gate[p] = w[i];
    r.token[p] = (uint8_t)t;
  }
  __syncthreads();
}

// ----------------------------------------------------------------------------- products

// Eight values as NT bf16 terms whose sum they are.
template <typename ACT>
struct Terms;
template <>
struct Terms<uint16_t> {
  static constexpr int N = 1;
  __device__ __forceinline__ static void load(const uint16_t* p, bf16x8v* t) {
    const Bf16x8u w = *reinterpret_cast<const Bf16x8u*>(p);
    t[0] = __builtin_bit_cast(bf16x8v, u32x4v{w.v[0], w.v[1], w.v[2], w.v[3]});
  }
};
__device__ __forceinline__ uint16_t bf16_bits(float f) { return OutElem<true>::rounded(f); }
// f as three terms: 8 bits each, the last one exact; an infinity or a NaN stays whole in the first
__device__ __forceinline__ void three_terms(float f, uint16_t* t) {
  t[0] = bf16_bits(f);
  const float r = f - OutElem<true>::load(t[0]);
  t[1] = fabsf(f) < INFINITY ? bf16_bits(r) : 0;
  t[2] = fabsf(f) < INFINITY ? bf16_bits(r - OutElem<true>::load(t[1])) : 0;
}
template <>
struct Terms<float> {
  static constexpr int N = 3;
  __device__ __forceinline__ static void load(const float* p, bf16x8v* t) {
    float v[8];
    values8(p, v);
    uint32_t w[3][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint16_t a[3], b[3];
      three_terms(v[2 * i], a);
      three_terms(v[2 * i + 1], b);
#pragma unroll
      for (int k = 0; k < 3; ++k) w[k][i] = (uint32_t)a[k] | (uint32_t)b[k] << 16;
    }
#pragma unroll
    for (int k = 0; k < 3; ++k) t[k] = __builtin_bit_cast(bf16x8v, u32x4v{w[k][0], w[k][1], w[k][2], w[k][3]});
  }
};

constexpr int kWaves = 8;

// One item of the first half: 8 gate rows and their 8 up rows x a tile of up to 16 tokens.
template <typename ACT>
__device__ __forceinline__ void gate_up(const Fp8LayerArgs& a, const Route& r, int tile, int rb, f32x4 (*part)[64]) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, i = lane & 15, q = lane >> 4;
  const int e = r.tile_expert[tile], first = r.at[e] + r.tile_first[tile];
  const int tokens = min(kTileTokens, __popcll(r.mask[e]) - r.tile_first[tile]);
  const int HB = f8_blocks(a.H), IB = f8_blocks(a.I), pieces = a.H / 16;
  const int row = min(rb * 8 + (i & 7), a.I - 1) + (i >= 8 ? a.I : 0);
  g_f8i4* w = (g_f8i4*)(a.q_gu + ((int64_t)e * 2 * a.I + row) * a.H);
  // rows 4q .. of the result: gate's for q < 2, up's else
  const float* s = a.s_gu + (((int64_t)e * 2 + (q >> 1)) * IB + rb * 8 / kF8Block) * HB;
  const bool mine = i < tokens;
  const ACT* x = static_cast<const ACT*>(a.x) + (mine ? r.token[first + i] : 0) * a.ld_x;
  f32x4 acc = {0.f, 0.f, 0.f, 0.f};
  for (int b = wave; b < HB; b += kWaves) {
    f32x4 sum = {0.f, 0.f, 0.f, 0.f};
    const float scale = s[b];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int p = b * 8 + 4 * h + q;
      f8i4 wv = w[min(p, pieces - 1)];
      if (p >= pieces) wv = f8i4{0, 0, 0, 0};
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        bf16x8v t[Terms<ACT>::N] = {};
        if (mine && p < pieces) Terms<ACT>::load(x + p * 16 + 8 * c, t);
        const bf16x8v wb = f8_to_bf16(wv[2 * c], wv[2 * c + 1]);
#pragma unroll
        for (int k = 0; k < Terms<ACT>::N; ++k) sum = mfma_bf16(wb, t[k], sum);
      }
    }
#pragma unroll
    for (int v = 0; v < 4; ++v) acc[v] = fmaf(scale, sum[v], acc[v]);
  }
  part[wave][lane] = acc;
  __syncthreads();
  const int c = threadIdx.x / 8, j = threadIdx.x % 8;
  if (c < tokens && rb * 8 + j < a.I) {
    const float* p = reinterpret_cast<const float*>(&part[0][16 * (j / 4) + c]) + j % 4;
    float g = 0.f, u = 0.f;
#pragma unroll
    for (int k = 0; k < kWaves; ++k) {
      g += p[k * 64 * 4];
      u += p[k * 64 * 4 + 32 * 4];  // up's rows are 8 on
    }
    uint16_t t[3];
    three_terms(g / (1.f + expf(-g)) * u, t);
    const int64_t at = (int64_t)(first + c) * a.I + rb * 8 + j, plane = (int64_t)a.T * a.k * a.I;
#pragma unroll
    for (int k = 0; k < 3; ++k) a.h[k * plane + at] = t[k];
  }
  __syncthreads();
}

template <typename ACT>
__global__ __launch_bounds__(64 * kWaves) void k_f8_gate_up(Fp8LayerArgs a) {
  __shared__ Route r;
  __shared__ f32x4 part[kWaves][64];
  route(a, r, blockIdx.x == 0);
  const int per = (a.I - 1) / 8 + 1;
  for (int item = blockIdx.x; item < r.tiles * per; item += gridDim.x) gate_up<ACT>(a, r, item / per, item % per, part);
}

// One item of the second half: 16 rows of down x every token, over all experts. Column i of
// group g is token 16 g + i; an expert's products are added with its weight, those of
// tokens that did not choose it are left out.
template <typename ACT, int G>
__device__ __forceinline__ void down(const Fp8LayerArgs& a, const Route& r, int rb, f32x4 (*part)[G][64]) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, i = lane & 15, q = lane >> 4;
  const int HB = f8_blocks(a.H), IB = f8_blocks(a.I), pieces = a.I / 16, n0 = rb * 16;
  const int64_t plane = (int64_t)a.T * a.k * a.I;
  f32x4 acc[G];
#pragma unroll
  for (int g = 0; g < G; ++g) acc[g] = f32x4{0.f, 0.f, 0.f, 0.f};
  for (int n = 0; n < r.experts; ++n) {
    const int e = r.expert[n];
    const uint64_t mask = r.mask[e];
    g_f8i4* w = (g_f8i4*)(a.q_dn + ((int64_t)e * a.H + min(n0 + i, a.H - 1)) * a.I);
    const float* s = a.s_dn + ((int64_t)e * HB + n0 / kF8Block) * IB;
    for (int b = wave; b < IB; b += kWaves) {
      f8i4 wv[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int p = b * 8 + 4 * h + q;
        wv[h] = w[min(p, pieces - 1)];
        if (p >= pieces) wv[h] = f8i4{0, 0, 0, 0};
      }
      const float scale = s[b];
#pragma unroll
      for (int g = 0; g < G; ++g) {
        if (((mask >> (16 * g)) & 0xFFFF) == 0) continue;
        const int t = 16 * g + i;
        const bool mine = (mask >> t) & 1;
        const int at = mine ? r.at[e] + __popcll(mask & ((1ull << t) - 1)) : 0;
        const uint16_t* hp = a.h + (int64_t)at * a.I;
        f32x4 sum = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int p = b * 8 + 4 * h + q;
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const bf16x8v wb = f8_to_bf16(wv[h][2 * c], wv[h][2 * c + 1]);
#pragma unroll
            for (int k = 0; k < 3; ++k) {
              bf16x8v v = {};
              if (mine && p < pieces) v = *reinterpret_cast<const bf16x8v*>(hp + k * plane + p * 16 + 8 * c);
              sum = mfma_bf16(wb, v, sum);
            }
          }
        }
        const float ws = mine ? r.gate[at] * scale : 0.f;
#pragma unroll
        for (int v = 0; v < 4; ++v) acc[g][v] = mine ? fmaf(ws, sum[v], acc[g][v]) : acc[g][v];
      }
    }
  }
#pragma unroll
  for (int g = 0; g < G; ++g) part[wave][g][lane] = acc[g];
  __syncthreads();
  for (int o = threadIdx.x; o < 16 * a.T; o += 64 * kWaves) {
    const int t = o / 16, j = o % 16, n = n0 + j;
    const float* p = reinterpret_cast<const float*>(&part[0][t / 16][16 * (j / 4) + t % 16]) + j % 4;
    float v = 0.f;
#pragma unroll
    for (int k = 0; k < kWaves; ++k) v += p[k * G * 64 * 4];
    if (n >= a.H) continue;
    a.y[t * a.ld_y + n] = v;
    if (a.x_out) {
      typedef OutElem<sizeof(ACT) == 2> Out;
      const float s = Out::load(static_cast<const ACT*>(a.x)[t * a.ld_x + n]) + v;
      static_cast<ACT*>(a.x_out)[t * a.ld_x_out + n] = Out::rounded(s);
    }
  }
  __syncthreads();
}

template <typename ACT, int G>
__global__ __launch_bounds__(64 * kWaves) void k_f8_down(Fp8LayerArgs a) {
  __shared__ Route r;
  __shared__ f32x4 part[kWaves][G][64];
  route(a, r, false);
  for (int rb = blockIdx.x; rb < (a.H - 1) / 16 + 1; rb += gridDim.x) down<ACT, G>(a, r, rb, part);
}

template <typename ACT>
void layer(const Fp8LayerArgs& a, hipStream_t s) {
  hipLaunchKernelGGL((k_f8_router<ACT>), dim3(a.logits_in ? a.T : a.E), dim3(64 * kRouterWaves), 0, s, a);
  const int64_t items = (int64_t)a.T * a.k * ((a.I - 1) / 8 + 1);
  hipLaunchKernelGGL((k_f8_gate_up<ACT>), dim3((unsigned)std::min<int64_t>(items, 1024)), dim3(64 * kWaves), 0, s, a);
  const int rows = (a.H - 1) / 16 + 1, grid = std::min(rows, 1024);
  if (a.T <= 16)
    hipLaunchKernelGGL((k_f8_down<ACT, 1>), dim3(grid), dim3(64 * kWaves), 0, s, a);
  else if (a.T <= 32)
    hipLaunchKernelGGL((k_f8_down<ACT, 2>), dim3(grid), dim3(64 * kWaves), 0, s, a);
  else
    hipLaunchKernelGGL((k_f8_down<ACT, 4>), dim3(grid), dim3(64 * kWaves), 0, s, a);
}

}  // namespace

void launch_fp8_layer(const Fp8LayerArgs& a, bool act_bf16, hipStream_t s) {
  if (act_bf16)
    layer<uint16_t>(a, s);
  else
    layer<float>(a, s);
}

}  // namespace moe
