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

// f as three bf16 terms: 8 bits each, the last one exact; an infinity or a NaN stays whole in the first.
__device__ __forceinline__ void three_terms(float f, uint16_t* t) {
  typedef OutElem<true> Bf;
  t[0] = Bf::rounded(f);
  const bool finite = fabsf(f) < INFINITY;
  const float r = f - Bf::load(t[0]);
  t[1] = finite ? Bf::rounded(r) : 0;
  t[2] = finite ? Bf::rounded(r - Bf::load(t[1])) : 0;
}

// Workgroups 0 .. E - 1 take a row of the router each, H split over its threads, the others
// (fp32 activations) a token each, whose terms they write. With logits_in there are T
// workgroups, which copy a token's logits where they are wanted. Tokens are taken four at a
// time, their loads ahead of the sums.
constexpr int kRouterThreads = 256, kRouterTokens = 4;
template <typename ACT>
__global__ __launch_bounds__(kRouterThreads) void k_f8_router(Fp8LayerArgs a, int rows) {
  __shared__ double part[kRouterThreads / 64][kF8LayerTokens];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  if ((int)blockIdx.x >= rows) {
    const int t = blockIdx.x - rows;
    if (a.logits_in && a.logits)
      for (int i = threadIdx.x; i < a.E; i += kRouterThreads) a.logits[(int64_t)t * a.E + i] = a.logits_in[(int64_t)t * a.E + i];
    if (sizeof(ACT) == 4) {
      const float* x = static_cast<const float*>(a.x) + t * a.ld_x;
      for (int i = threadIdx.x; i < a.H; i += kRouterThreads) {
        uint16_t v[3];
        three_terms(x[i], v);
#pragma unroll
        for (int k = 0; k < 3; ++k) a.xt[((int64_t)k * a.T + t) * a.H + i] = v[k];
      }
    }
    return;
  }
  const int e = blockIdx.x;
  const ACT* w = static_cast<const ACT*>(a.router_w) + e * a.ld_router;
  for (int t0 = 0; t0 < a.T; t0 += kRouterTokens) {
    const ACT* x[kRouterTokens];
    double sum[kRouterTokens];
#pragma unroll
    for (int t = 0; t < kRouterTokens; ++t) {
      x[t] = static_cast<const ACT*>(a.x) + min(t0 + t, a.T - 1) * a.ld_x;
      sum[t] = 0.0;
    }
    for (int j = 8 * threadIdx.x; j < a.H; j += 8 * kRouterThreads) {  // H is a multiple of 16
      float wv[8], xv[kRouterTokens][8];
      values8(w + j, wv);
#pragma unroll
      for (int t = 0; t < kRouterTokens; ++t) values8(x[t] + j, xv[t]);
#pragma unroll
      for (int t = 0; t < kRouterTokens; ++t)
#pragma unroll
        for (int i = 0; i < 8; ++i) sum[t] = fma((double)wv[i], (double)xv[t][i], sum[t]);
    }
#pragma unroll
    for (int t = 0; t < kRouterTokens; ++t) {
      if (t0 + t >= a.T) break;
      sum[t] = wave_sum_63(sum[t]);
      if (lane == 63) part[wave][t0 + t] = sum[t];
    }
  }
  __syncthreads();
  for (int t = threadIdx.x; t < a.T; t += kRouterThreads) {
    double v = a.router_b ? (double)a.router_b[e] : 0.0;
#pragma unroll
    for (int k = 0; k < kRouterThreads / 64; ++k) v += part[k][t];
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
  uint16_t tile_expert[kMaxAssign];   // tiles: the expert, and the first of up to `tile` of its tokens
  uint8_t tile_first[kMaxAssign];
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

// `writes`: one workgroup of the launch, which also leaves the tables for the next launch.
template <int TILE>
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
      const int tc = (c + TILE - 1) / TILE;
      const int incl = wave_incl_scan(c), tincl = wave_incl_scan(tc);
      if (c > 0) {
        r.at[e] = (uint16_t)(places + incl - c);
        r.expert[experts + __popcll(some & ((1ull << lane) - 1))] = (uint16_t)e;
        for (int i = 0; i < tc; ++i) {
          r.tile_expert[tiles + tincl - tc + i] = (uint16_t)e;
          r.tile_first[tiles + tincl - tc + i] = (uint8_t)(TILE * i);
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
    if (writes) {
      a.tables->gate[p] = w[i];
      a.tables->token[p] = (uint8_t)t;
    }
  }
  if (writes) {
    for (int i = threadIdx.x; i < r.experts; i += blockDim.x) {
      const int e = r.expert[i];
      a.tables->expert[i] = Fp8Expert{(uint16_t)e, r.at[e], (uint16_t)__popcll(r.mask[e]), 0};
    }
    if (threadIdx.x == 0) a.tables->experts = r.experts;
  }
  __syncthreads();
}

// ----------------------------------------------------------------------------- products

constexpr int kWaves = 8;  // of a workgroup, taking blocks of 128 of K in turn

// Columns of the MFMA: 16 tokens of one term, or 5 tokens of three (column 3 c + k is token c's
// term k, the last column none's).
template <int TERMS>
struct Columns {
  static constexpr int kTokens = TERMS == 1 ? 16 : 5;
  static __device__ __forceinline__ int token(int column) { return TERMS == 1 ? column : column / 3; }
  static __device__ __forceinline__ int term(int column) { return TERMS == 1 ? 0 : column % 3; }
};

// the other terms' sums, from the two columns on; meant for a token's first column
__device__ __forceinline__ float add_terms(float v) {
  constexpr int kShl1 = 0x101, kShl2 = 0x102;  // row_shl: the lane 1 (2) on in the row of 16
  return v + (dppf<kShl1, 0xF>(0.f, v) + dppf<kShl2, 0xF>(0.f, v));
}

// Bytes 16 p .. of a row of codes, or the last of the row past its end.
__device__ __forceinline__ f8i4 piece(g_f8i4* row, int p, int pieces) { return row[min(p, pieces - 1)]; }
// The 16 bf16 at place 16 p of a row, as the two steps of piece p take them.
__device__ __forceinline__ void values(const uint16_t* row, int p, int pieces, bf16x8v* v) {
  const uint16_t* at = row + min(p, pieces - 1) * 16;
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    const Bf16x8u w = reinterpret_cast<const Bf16x8u*>(at)[c];
    v[c] = __builtin_bit_cast(bf16x8v, u32x4v{w.v[0], w.v[1], w.v[2], w.v[3]});
  }
}

__device__ __forceinline__ f32x4 times(const f8i4* w, const bf16x8v* v) {
  f32x4 sum = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int c = 0; c < 2; ++c) sum = mfma_bf16(f8_to_bf16(w[h][2 * c], w[h][2 * c + 1]), v[2 * h + c], sum);
  return sum;
}

// First half: an item is 16 gate rows and their 16 up rows x a tile of an expert's tokens.
// A wave's blocks of K over all of the workgroup's items are one sequence, of which it has
// kAhead under way.
template <int TERMS>
__global__ __launch_bounds__(64 * kWaves, 4) void k_f8_gate_up(Fp8LayerArgs a) {
  typedef Columns<TERMS> Cols;
  constexpr int kAhead = 2;
  __shared__ Route r;
  __shared__ f32x4 part[2][2][kWaves][64];
  route<Cols::kTokens>(a, r, blockIdx.x == 0);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), i = lane & 15, q = lane >> 4;
  const int HB = f8_blocks(a.H), IB = f8_blocks(a.I), pieces = a.H / 16, per = a.I / 16;
  const int steps = (HB + kWaves - 1) / kWaves, items = r.tiles * per;
  const uint16_t* xs = TERMS == 1 ? static_cast<const uint16_t*>(a.x) : a.xt + (int64_t)Cols::term(i) * a.T * a.H;
  const int64_t ld = TERMS == 1 ? a.ld_x : a.H;

  struct Unit {
    f8i4 g[2], u[2];
    bf16x8v x[4];
    float sg, su;
  };
  // what the loads are at
  int item = blockIdx.x, step = 0;
  g_f8i4 *wg = nullptr, *wu = nullptr;
  const uint16_t* x = nullptr;
  const float* s = nullptr;
  auto load = [&](Unit& f) {
    if (item >= items) return;
    if (step == 0) {
      const int tile = item / per, rb = item % per, e = r.tile_expert[tile], first = r.tile_first[tile];
      const int tokens = min(Cols::kTokens, __popcll(r.mask[e]) - first);
      wg = (g_f8i4*)(a.q_gu + ((int64_t)e * 2 * a.I + rb * 16 + i) * a.H);
      wu = (g_f8i4*)(a.q_gu + ((int64_t)e * 2 * a.I + a.I + rb * 16 + i) * a.H);
      s = a.s_gu + ((int64_t)e * 2 * IB + rb * 16 / kF8Block) * HB;
      // columns past the tile's are the first one's again, and not stored
      const int c = Cols::token(i);
      x = xs + r.token[r.at[e] + first + (c < tokens ? c : 0)] * ld;
    }
    const int b = min(wave + step * kWaves, HB - 1);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      f.g[h] = piece(wg, b * 8 + 4 * h + q, pieces);
      f.u[h] = piece(wu, b * 8 + 4 * h + q, pieces);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) values(x, b * 8 + 4 * h + q, pieces, f.x + 2 * h);
    f.sg = s[b];
    f.su = s[(int64_t)IB * HB + b];
    if (++step == steps) {
      step = 0;
      item += gridDim.x;
    }
  };
  // what the sums are at
  int at = blockIdx.x, done = 0, turn = 0;
  f32x4 gate = {0.f, 0.f, 0.f, 0.f}, up = gate;
  auto products = [&](Unit& f) {
    const int b = wave + done * kWaves;
    if (b < HB) {
      if (b * 8 + 8 > pieces) {  // K ends inside the block
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if (b * 8 + 4 * h + q >= pieces) {
            f.g[h] = f.u[h] = f8i4{0, 0, 0, 0};
            f.x[2 * h] = f.x[2 * h + 1] = bf16x8v{};
          }
      }
      const f32x4 pg = times(f.g, f.x), pu = times(f.u, f.x);
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        gate[v] = fmaf(f.sg, pg[v], gate[v]);
        up[v] = fmaf(f.su, pu[v], up[v]);
      }
    }
    if (++done < steps) return;
    // the item's sums meet; another buffer each time, so that one barrier does
    if (TERMS > 1) {
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        gate[v] = add_terms(gate[v]);
        up[v] = add_terms(up[v]);
      }
    }
    part[turn][0][wave][lane] = gate;
    part[turn][1][wave][lane] = up;
    __syncthreads();
    const int tile = at / per, rb = at % per, e = r.tile_expert[tile], first = r.tile_first[tile];
    const int tokens = min(Cols::kTokens, __popcll(r.mask[e]) - first);
    const int c = threadIdx.x / 16, j = threadIdx.x % 16;
    if (c < tokens) {
      const int column = TERMS == 1 ? c : 3 * c;
      const float* p = reinterpret_cast<const float*>(&part[turn][0][0][16 * (j / 4) + column]) + j % 4;
      float gs = 0.f, us = 0.f;
#pragma unroll
      for (int k = 0; k < kWaves; ++k) {
        gs += p[k * 64 * 4];
        us += p[(kWaves + k) * 64 * 4];
      }
      uint16_t t[3];
      three_terms(gs / (1.f + expf(-gs)) * us, t);
      const int64_t to = (int64_t)(r.at[e] + first + c) * a.I + rb * 16 + j, plane = (int64_t)a.T * a.k * a.I;
#pragma unroll
      for (int k = 0; k < 3; ++k) a.h[k * plane + to] = t[k];
    }
    gate = up = f32x4{0.f, 0.f, 0.f, 0.f};
    done = 0;
    turn ^= 1;
    at += gridDim.x;
  };
  Unit f[kAhead];
#pragma unroll
  for (int k = 0; k < kAhead; ++k) load(f[k]);
  while (at < items) {
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      if (at < items) {
        products(f[k]);
        load(f[k]);
      }
    }
  }
}

// Second half: 16 rows of down x every token, over all experts. A wave's blocks of K over the
// experts are one sequence, of which it has kAhead under way, with the first tile of the
// expert's tokens. What a block gives a token is added, with the token's weight for the
// expert, to the wave's sums in LDS; the waves' sums meet at the end.
template <typename ACT>
__global__ __launch_bounds__(64 * kWaves, 4) void k_f8_down(Fp8LayerArgs a) {
  typedef Columns<3> Cols;
  constexpr int kAhead = 3;
  extern __shared__ __attribute__((aligned(16))) float sums[];  // [kWaves][T][16]
  __shared__ Fp8Expert experts[kF8LayerExperts];
  __shared__ float gates[kMaxAssign];
  __shared__ uint8_t tokens[kMaxAssign];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), i = lane & 15, q = lane >> 4;
  const int HB = f8_blocks(a.H), IB = f8_blocks(a.I), pieces = a.I / 16, n0 = blockIdx.x * 16;
  const int n_experts = a.tables->experts;
  for (int k = threadIdx.x; k < n_experts; k += 64 * kWaves) experts[k] = a.tables->expert[k];
  for (int k = threadIdx.x; k < a.T * a.k; k += 64 * kWaves) {
    gates[k] = a.tables->gate[k];
    tokens[k] = a.tables->token[k];
  }
  for (int k = threadIdx.x; k < kWaves * a.T * 16; k += 64 * kWaves) sums[k] = 0.f;
  __syncthreads();
  const int steps = (IB + kWaves - 1) / kWaves;
  const uint16_t* hs = a.h + (int64_t)Cols::term(i) * a.T * a.k * a.I;
  const int c = Cols::token(i);

  struct Unit {
    f8i4 w[2];
    bf16x8v h[4];
    float s;
  };
  auto load_h = [&](bf16x8v* h, const Fp8Expert& e, int first, int b) {
    // columns past the tile's are the first one's again, and not used
    const uint16_t* row = hs + (int64_t)(e.at + first + (first + c < e.count ? c : 0)) * a.I;
#pragma unroll
    for (int k = 0; k < 2; ++k) values(row, b * 8 + 4 * k + q, pieces, h + 2 * k);
  };
  int n = 0, step = 0;
  auto load = [&](Unit& f) {
    if (n >= n_experts) return;
    const Fp8Expert e = experts[n];
    const int b = min(wave + step * kWaves, IB - 1);
    g_f8i4* w = (g_f8i4*)(a.q_dn + ((int64_t)e.expert * a.H + n0 + i) * a.I);
#pragma unroll
    for (int k = 0; k < 2; ++k) f.w[k] = piece(w, b * 8 + 4 * k + q, pieces);
    load_h(f.h, e, 0, b);
    f.s = a.s_dn[((int64_t)e.expert * HB + n0 / kF8Block) * IB + b];
    if (++step == steps) {
      step = 0;
      ++n;
    }
  };
  int at = 0, done = 0;
  auto products = [&](Unit& f) {
    const int b = wave + done * kWaves;
    const Fp8Expert e = experts[at];
    if (b < IB) {
      const bool ends = b * 8 + 8 > pieces;  // K ends inside the block
      if (ends) {
#pragma unroll
        for (int k = 0; k < 2; ++k)
          if (b * 8 + 4 * k + q >= pieces) f.w[k] = f8i4{0, 0, 0, 0};
      }
      for (int first = 0; first < e.count; first += Cols::kTokens) {
        if (first > 0) load_h(f.h, e, first, b);
        if (ends) {
#pragma unroll
          for (int k = 0; k < 2; ++k)
            if (b * 8 + 4 * k + q >= pieces) f.h[2 * k] = f.h[2 * k + 1] = bf16x8v{};
        }
        f32x4 sum = times(f.w, f.h);
#pragma unroll
        for (int v = 0; v < 4; ++v) sum[v] = add_terms(sum[v]);
        if (Cols::term(i) == 0 && first + c < e.count && c < Cols::kTokens) {
          const float scale = gates[e.at + first + c] * f.s;
          f32x4* to = reinterpret_cast<f32x4*>(&sums[(wave * a.T + tokens[e.at + first + c]) * 16 + 4 * q]);
          f32x4 v = *to;
#pragma unroll
          for (int k = 0; k < 4; ++k) v[k] = fmaf(scale, sum[k], v[k]);
          *to = v;
        }
      }
    }
    if (++done == steps) {
      done = 0;
      ++at;
    }
  };
  Unit f[kAhead];
#pragma unroll
  for (int k = 0; k < kAhead; ++k) load(f[k]);
  while (at < n_experts) {
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      if (at < n_experts) {
        products(f[k]);
        load(f[k]);
      }
    }
  }
  __syncthreads();
  for (int o = threadIdx.x; o < 16 * a.T; o += 64 * kWaves) {
    const int t = o / 16, col = n0 + o % 16;
    float v = 0.f;
#pragma unroll
    for (int k = 0; k < kWaves; ++k) v += sums[k * a.T * 16 + o];
    a.y[t * a.ld_y + col] = v;
    if (a.x_out) {
      typedef OutElem<sizeof(ACT) == 2> Out;
      const float x = Out::load(static_cast<const ACT*>(a.x)[t * a.ld_x + col]) + v;
      static_cast<ACT*>(a.x_out)[t * a.ld_x_out + col] = Out::rounded(x);
    }
  }
}

template <typename ACT>
void layer(const Fp8LayerArgs& a, hipStream_t s) {
  constexpr int kTerms = sizeof(ACT) == 2 ? 1 : 3;
  const int rows = a.logits_in ? 0 : a.E, more = a.logits_in || kTerms == 3 ? a.T : 0;
  hipLaunchKernelGGL((k_f8_router<ACT>), dim3(rows + more), dim3(kRouterThreads), 0, s, a, rows);
  const int64_t items = (int64_t)a.T * a.k * (a.I / 16);
  hipLaunchKernelGGL((k_f8_gate_up<kTerms>), dim3((unsigned)std::min<int64_t>(items, 512)), dim3(64 * kWaves), 0, s, a);
  hipLaunchKernelGGL((k_f8_down<ACT>), dim3(a.H / 16), dim3(64 * kWaves), sizeof(float) * kWaves * 16 * a.T, s, a);
}

}  // namespace

void launch_fp8_layer(const Fp8LayerArgs& a, bool act_bf16, hipStream_t s) {
  if (act_bf16)
    layer<uint16_t>(a, s);
  else
    layer<float>(a, s);
}

}  // namespace moe
