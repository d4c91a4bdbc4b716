// A whole routed layer for up to 64 tokens on experts of e4m3 codes with a scale for each
// 128 x 128 block: router, top-k, gate and up, silu, down, combine.
//
//   logits = x Wr + b (fp64 sums),  w = softmax of the k largest,  h_e = silu(Wg_e x) (Wu_e x)
//   y[t] = sum_e w[t][e] Wd_e h_e[t]
//
// The router's sums are in fp64, so that which experts a token takes does not turn on the
// order of the sums. A bf16 x fp8 product is exact in the bf16 MFMA (f8_dev.h); an fp32 value
// is the exact sum of three bf16 terms (8 bits of its mantissa each) with powers of two, so that
// fp32 activations and the intermediate h, which stays in fp32, take three products.
//
// Three launches: the router (which also lays out x as the products read it), the first half, the
// second half. Every workgroup of the first half forms the routing's tables by itself, in LDS
// (2.5 us for one token), instead of a launch of its own; one leaves them for the second half.
//
// What bounds it: a token on 6 experts of 7168 / 2048 (264 MB) takes 61 us, of which gate and up
// 31 (5.7 TB/s), down 18 (4.9), the router 6; a token on 8 of 2048 / 768 (38 MB) 19 us, of which
// 3 + 9 + 6: there the starts of three short bursts count, not the bytes (7.5 us). 16 tokens take 71 us on
// 2048 / 768 (48 experts: gate and up 4.2 TB/s, down 2.6) and 382 on 7168 / 2048 (37: 5.5, 3.5). 64 tokens on one
// expert of 2048 / 768 take 42: the router, with a workgroup for each expert, 18, down, which loads the weights
// again for every two tokens, 13.
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

// f as three bf16 terms, f = t0 + 2^-7 t1 + 2^-16 t2 for every finite f: its first 8 bits, cut; what that
// leaves, under 2^-7 of f's binade and held 2^7 fold, rounded; what that leaves, held 2^9 fold again. So
// none is larger than f (than 2^-125, of the smallest f, whose terms are bf16 numbers too), and the
// sums of none leave fp32 where f's own do not. An infinity or a NaN stays whole in the first.
constexpr float kSecond = 0x1p-7f, kThird = 0x1p-9f;  // the second to the first, the third to the second
__device__ __forceinline__ void three_terms(float f, uint16_t* t) {
  typedef OutElem<true> Bf;
  const bool finite = fabsf(f) < INFINITY;
  const uint32_t u = __float_as_uint(f);
  const float r = finite ? (f - __uint_as_float(u & 0xFFFF0000u)) * (1.f / kSecond) : 0.f;
  t[0] = finite ? (uint16_t)(u >> 16) : Bf::rounded(f);
  t[1] = Bf::rounded(r);
  t[2] = (uint16_t)(__float_as_uint((r - Bf::load(t[1])) * (1.f / kThird)) >> 16);
}

// The first `rows` workgroups take a row of the router each, H split over their threads, the
// others a token each, whose values or terms they write where the products read them (and its
// given logits, where they are wanted). Tokens are taken four at a time, their loads ahead of
// the sums.
constexpr int kRouterThreads = 256, kRouterTokens = 4;
template <typename ACT>
__global__ __launch_bounds__(kRouterThreads) void k_f8_router(Fp8LayerArgs a, int rows) {
  __shared__ double part[kRouterThreads / 64][kF8LayerTokens];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  if ((int)blockIdx.x >= rows) {
    const int t = blockIdx.x - rows;
    if (a.logits_in && a.logits)
      for (int i = threadIdx.x; i < a.E; i += kRouterThreads) a.logits[(int64_t)t * a.E + i] = a.logits_in[(int64_t)t * a.E + i];
    const ACT* x = static_cast<const ACT*>(a.x) + t * a.ld_x;
    for (int i = threadIdx.x; i < a.Hp; i += kRouterThreads) {
      if (sizeof(ACT) == 2) {
        a.xt[(int64_t)t * a.Hp + i] = i < a.H ? x[i] : 0;
      } else {
        uint16_t v[3];
        three_terms(i < a.H ? x[i] : 0.f, v);
#pragma unroll
        for (int k = 0; k < 3; ++k) a.xt[((int64_t)k * a.T + t) * a.Hp + i] = v[k];
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
  uint64_t mask[kF8LayerExperts];  // the expert's tokens
  Fp8Tile tile[kMaxAssign];
  float gate[kMaxAssign];          // weights, in grouped order
  uint16_t at[kF8LayerExperts];    // the expert's first place in that order
  uint8_t token[kMaxAssign];       // token of a place
  int tiles;
};
constexpr int kDownTokens = 2;  // of a tile of the second half

// Orders as the logits do, with NaN before every number; over 0.
__device__ __forceinline__ uint32_t logit_key(float f) {
  const uint32_t u = f == 0.f ? 0u : __float_as_uint(f);
  if (f != f) return ~0u;
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ float logit_of(uint32_t key) {
  if (key == ~0u) return __uint_as_float(0x7FC00000u);
  return __uint_as_float(key & 0x80000000u ? key & 0x7FFFFFFFu : ~key);
}

// The k experts of one token by one wave: k rounds of the wave's maximum and the lowest
// expert that has it. Lane l holds experts l, l + 64, ...; lane j ends with slot j, and its
// rank among the token's experts of any weight.
template <int NV>
__device__ __forceinline__ void choose_of(const float* logits, int E, int k, int& id, float& w, int& rank) {
  const int lane = threadIdx.x & 63;
  uint32_t key[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const float f = logits[min(lane + 64 * i, E - 1)];
    key[i] = lane + 64 * i < E ? logit_key(f) : 0u;
  }
  uint32_t mine = 0u;
  id = 0;
  for (int j = 0; j < k; ++j) {
    uint32_t m = key[0];
#pragma unroll
    for (int i = 1; i < NV; ++i) m = max(m, key[i]);
    m = wave_max_u(m);
    int win = 0;
#pragma unroll
    for (int i = NV - 1; i >= 0; --i) {
      const unsigned long long b = __ballot(key[i] == m);
      win = b != 0ull ? 64 * i + (int)__builtin_ctzll(b) : win;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) key[i] = lane + 64 * i == win ? 0u : key[i];
    mine = lane == j ? m : mine;
    id = lane == j ? win : id;
  }
  const float v = logit_of(mine), top = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 0));
  const bool counts = lane < k && v != -INFINITY;
  const float p = counts ? expf(v - top) : 0.f;
  const float sum = wave_sum(p);
  w = counts ? p / sum : 0.f;  // 0 also where the sum is NaN, for another logit's sake, or 0
  const uint64_t some = __ballot(w != 0.f);
  rank = 0;
  for (int j = 0; j < k; ++j) rank += (some >> j & 1) && __builtin_amdgcn_readlane(id, j) < id;
}
// A lane's experts are searched whether they are there or not, in every round: 128 experts in the form for 128
// a token's layer of 2048 / 256 14.9 us (for 384: 15.7, for 1024: 17.7), 16 tokens' 38.3 (39.9, 44.2); 256 in that for
// 384 16.5 and 41.9 (for 1024: 18.4, 46.1).
__device__ __forceinline__ void choose(const float* logits, int E, int k, int& id, float& w, int& rank) {
  const int nv = (E + 63) / 64;
  if (nv <= 2)
    choose_of<2>(logits, E, k, id, w, rank);
  else if (nv <= 6)
    choose_of<6>(logits, E, k, id, w, rank);
  else
    choose_of<16>(logits, E, k, id, w, rank);
}

// Tiles of up to TILE tokens for this launch; the workgroup that `writes` also leaves the outputs,
// and the tables for the next launch.
template <int TILE>
__device__ __forceinline__ void route(const Fp8LayerArgs& a, Route& r, bool writes) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
  const float* logits = a.logits ? a.logits : a.logits_in;
  if (a.T == 1) {  // a token's experts are its tiles: no grouping (route of 2048 / 128 / 8: 2.5 us, 3.8 with it)
    if (wave == 0) {
      int id, rank;
      float w;
      choose(logits, a.E, a.k, id, w, rank);
      const bool is = lane < a.k && w != 0.f;
      const int n = __popcll(__ballot(is));
      if (is) {
        r.tile[rank] = Fp8Tile{(uint16_t)id, (uint16_t)rank, 1, 0};
        r.token[rank] = 0;
      }
      if (lane == 0) r.tiles = n;
      if (writes) {
        if (is) {
          a.tables->tile[rank] = Fp8Tile{(uint16_t)id, (uint16_t)rank, 1, 0};
          a.tables->gate[rank] = w;
        }
        if (lane < a.k) {
          a.tables->place[lane] = lane < n ? (uint32_t)lane | (uint32_t)lane << 16 : kF8NoPlace;
          if (a.ids) a.ids[lane] = id;
          if (a.gate) a.gate[lane] = w;
        }
        if (lane == 0) a.tables->tiles = a.tables->places = n;
      }
    }
    __syncthreads();
    return;
  }
  uint32_t* slot = reinterpret_cast<uint32_t*>(r.tile);  // id and rank of an assignment, until the tiles are made
  for (int e = threadIdx.x; e < a.E; e += blockDim.x) r.mask[e] = 0;
  __syncthreads();
  for (int t = wave; t < a.T; t += waves) {
    int id, rank;
    float w;
    choose(logits + (int64_t)t * a.E, a.E, a.k, id, w, rank);
    if (lane < a.k) {
      const int s = t * a.k + lane;
      if (w != 0.f) atomicOr(reinterpret_cast<unsigned long long*>(&r.mask[id]), 1ull << t);
      slot[s] = (uint32_t)id | (uint32_t)rank << 16;
      r.gate[s] = w;
      if (writes) {
        a.tables->place[s] = kF8NoPlace;
        if (a.ids) a.ids[s] = id;
        if (a.gate) a.gate[s] = w;
      }
    }
  }
  __syncthreads();
  constexpr int kMine = kMaxAssign / 512;  // a thread's assignments
  uint32_t mine[kMine];
  float w[kMine];
  const int n = a.T * a.k;
#pragma unroll
  for (int i = 0; i < kMine; ++i) {
    const int s = threadIdx.x + i * 512;
    mine[i] = s < n ? slot[s] : 0;
    w[i] = s < n ? r.gate[s] : 0.f;
  }
  __syncthreads();
  if (wave == 0) {
    int places = 0, tiles = 0, down = 0;
    for (int e0 = 0; e0 < a.E; e0 += 64) {
      const int e = e0 + lane, c = e < a.E ? __popcll(r.mask[e]) : 0;
      if (__ballot(c > 0) == 0) continue;
      const int tc = (c + TILE - 1) / TILE, dc = (c + kDownTokens - 1) / kDownTokens;
      const int incl = wave_incl_scan(c), tincl = wave_incl_scan(tc), dincl = wave_incl_scan(dc);
      if (c > 0) {
        const int at = places + incl - c;
        r.at[e] = (uint16_t)at;
        for (int i = 0; i < tc; ++i)
          r.tile[tiles + tincl - tc + i] = Fp8Tile{(uint16_t)e, (uint16_t)(at + TILE * i), (uint16_t)min(TILE, c - TILE * i), 0};
        if (writes)
          for (int i = 0; i < dc; ++i)
            a.tables->tile[down + dincl - dc + i] =
                Fp8Tile{(uint16_t)e, (uint16_t)(at + kDownTokens * i), (uint16_t)min(kDownTokens, c - kDownTokens * i), 0};
      }
      places += __builtin_amdgcn_readlane(incl, 63);
      tiles += __builtin_amdgcn_readlane(tincl, 63);
      down += __builtin_amdgcn_readlane(dincl, 63);
    }
    if (lane == 0) {
      r.tiles = tiles;
      if (writes) {
        a.tables->tiles = down;
        a.tables->places = places;
      }
    }
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kMine; ++i) {
    if (w[i] == 0.f) continue;
    const int t = (threadIdx.x + i * 512) / a.k, id = mine[i] & 0xFFFF;
    const int within = __popcll(r.mask[id] & ((1ull << t) - 1)), p = r.at[id] + within;
    r.token[p] = (uint8_t)t;
    if (writes) {
      a.tables->gate[p] = w[i];
      a.tables->place[t * a.k + (mine[i] >> 16)] = (uint32_t)p | (uint32_t)(p - within % kDownTokens) << 16;  // behind the barriers since its first value
    }
  }
  __syncthreads();
}

// ----------------------------------------------------------------------------- products
//
// Operands are of 8 rows and 8 vectors, at two parities of the pieces of K (f8_dev.h).

constexpr int kWaves = 8;  // of a workgroup, taking blocks of 128 of K in turn
constexpr int kRows = 8;   // of weights in an operand
constexpr int kCus = 256;

// Vectors: 8 tokens of one term, or 2 tokens of three (vector 3 c + k is token c's term k).
template <int TERMS>
struct Vectors {
  static constexpr int kTokens = TERMS == 1 ? 8 : 2;
  static __device__ __forceinline__ int token(int v) { return TERMS == 1 ? v : v / 3; }
  static __device__ __forceinline__ int term(int v) { return TERMS == 1 ? 0 : v % 3; }
  // the sum over the parities, and over the terms with their sizes; in the first lane of a token's
  static __device__ __forceinline__ float whole(float v) {
    constexpr int kShl2 = 0x102, kShl4 = 0x104;  // row_shl: the lane 2 (4) on in the row of 16
    v += dppf<kDppXor1, 0xF>(0.f, v);
    return TERMS == 1 ? v : fmaf(fmaf(dppf<kShl4, 0xF>(0.f, v), kThird, dppf<kShl2, 0xF>(0.f, v)), kSecond, v);
  }
  static __device__ __forceinline__ int lane_of(int token) { return TERMS == 1 ? 2 * token : 6 * token; }
  static __device__ __forceinline__ bool is_first(int column) { return TERMS == 1 ? column % 2 == 0 : column == 0 || column == 6; }
};

// A lane's 16 values of a vector, as two steps of the MFMA take them.
struct Values {
  bf16x8v v[2];
};
__device__ __forceinline__ Values load_values(__amdgpu_buffer_rsrc_t from, uint32_t at) {
  return Values{{__builtin_bit_cast(bf16x8v, __builtin_amdgcn_raw_buffer_load_b128(from, at, 0, 0)),
                 __builtin_bit_cast(bf16x8v, __builtin_amdgcn_raw_buffer_load_b128(from, at + 16, 0, 0))}};
}
// The workspace's bf16 values as a buffer of under 2^30 bytes: a lane whose vector is none reads past its
// end, which gives zeros and asks no memory for anything. (Vectors that repeat another's instead
// take as much of the CU's room for loads under way as the weights do: 128 CUs then stream
// 2.8 TB/s of weights, and 5.5 without vectors.)
__device__ __forceinline__ __amdgpu_buffer_rsrc_t values_buffer(const uint16_t* p, int64_t n) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t*>(p), 0, (uint32_t)(2 * n), 0x00020000);
}
constexpr uint32_t kNoVector = 1u << 30;

// A block's scale as a power of two from 2^-100 to 2^100, which the codes' conversion takes, and
// the rest, of size 1 to 2 where the scale is in that range. So what is summed has the size of the
// weights, not of their codes, and leaves fp32 only where the weights' own sum does; no bit of
// a sum that stays inside changes.
struct BlockScale {
  float power, rest;
  __device__ __forceinline__ explicit BlockScale(float s) {
    constexpr uint32_t kLeast = (127u - 100) << 23, kMost = (127u + 100) << 23;
    const uint32_t e = min(max(__float_as_uint(s) & 0x7F800000u, kLeast), kMost);
    power = __uint_as_float(e);
    rest = s * __uint_as_float((254u << 23) - e);
  }
};

// The sums of 8 rows with a block's values, all parities: added, scaled, to s.
__device__ __forceinline__ void add_products(const f8i4& w, const Values& x, const BlockScale& scale, f32x4& s) {
  f32x4 p = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int c = 0; c < 2; ++c) p = mfma_bf16(f8_to_bf16(w[2 * c], w[2 * c + 1], scale.power), x.v[c], p);
#pragma unroll
  for (int v = 0; v < 4; ++v) s[v] = fmaf(scale.rest, p[v], s[v]);
}

__device__ __forceinline__ Fp8Tile uniform(const Fp8Tile* tile) {
  const uint64_t u = *reinterpret_cast<const uint64_t*>(tile);
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)u), hi = __builtin_amdgcn_readfirstlane((uint32_t)(u >> 32));
  return Fp8Tile{(uint16_t)lo, (uint16_t)(lo >> 16), (uint16_t)hi, 0};
}

// First half: an item is 16 gate rows and their 16 up rows x a tile of an expert's tokens. A
// workgroup keeps to its rows and takes every gridDim.y'th tile. A wave's blocks of K over all of
// its items are one sequence, of which it has kAhead under way. A turn but the last loads as
// many, past the end the last tile's again: a load that a branch leaves out would make every
// wait one for all loads.
template <int TERMS>
__global__ __launch_bounds__(64 * kWaves, 4) void k_f8_gate_up(Fp8LayerArgs a) {
  typedef Vectors<TERMS> Vec;
  // With three, a token on 2048 / 768 takes 18.7 us (17.7), on 4096 / 768 27.8 (26.5), on 7168 / 2048 55.1 (54.2), 16 tokens
  // 73.9 (72.8), 98.2 (96.9) and 355 (356); the most that a third wins is 3%, a token on 2560 / 2048 21.8 (22.5).
  constexpr int kAhead = 2;
  __shared__ Route r;
  __shared__ float part[2][kWaves][4][2][64];  // [turn][wave][operand][row of the lane's two][lane]
  route<Vec::kTokens>(a, r, blockIdx.x + blockIdx.y == 0);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), i = lane & 15, q = lane >> 4;
  const int HB = f8_blocks(a.H), IB = f8_blocks(a.I), pieces = a.H / 16, rb = blockIdx.x;
  const int steps = (HB + kWaves - 1) / kWaves, own = 2 * q + (i & 1);  // own: piece of a block
  const int tiles = r.tiles, zero = lane_zero();
  if ((int)blockIdx.y >= tiles) return;
  const __amdgpu_buffer_rsrc_t xs = values_buffer(a.xt, (int64_t)TERMS * a.T * a.Hp);
  const uint32_t own_x = 2 * (Vec::term(i / 2) * a.T * a.Hp + own * 16);
  const int row = (i / 2) * a.H, eight = kRows * a.H;  // within the item's 16 rows
  const int c = Vec::token(i / 2);

  struct Unit {
    f8i4 w[4];  // gate's rows 0 - 7 and 8 - 15, up's
    Values x;
    float sg, su;
  };
  // what the loads are at
  int tile = blockIdx.y, step = 0;
  const uint8_t *wg = nullptr, *wu = nullptr;
  uint32_t x = 0;
  const float* s = nullptr;
  auto load = [&](Unit& f) {
    if (step == 0) {
      const Fp8Tile t = uniform(&r.tile[min(tile, tiles - 1)]);
      wg = a.q_gu + ((int64_t)t.expert * 2 * a.I + rb * 16) * a.H;
      wu = wg + (int64_t)a.I * a.H;
      s = a.s_gu + ((int64_t)t.expert * 2 * IB + rb * 16 / kF8Block) * HB;
      x = c < t.tokens ? own_x + 2 * r.token[t.at + c] * a.Hp : kNoVector;
    }
    const int b = min(wave + step * kWaves, HB - 1), at = row + 16 * min(b * 8 + own, pieces - 1);
    f.w[0] = *(g_f8i4*)(wg + at);
    f.w[1] = *(g_f8i4*)(wg + at + eight);
    f.w[2] = *(g_f8i4*)(wu + at);
    f.w[3] = *(g_f8i4*)(wu + at + eight);
    f.x = load_values(xs, x + 2 * b * kF8Block);
    f.sg = s[b + zero];
    f.su = s[IB * HB + b + zero];
    if (++step == steps) {
      step = 0;
      tile += gridDim.y;
    }
  };
  // what the sums are at
  int at = blockIdx.y, done = 0, turn = 0;
  f32x4 sum[4] = {};
  auto products = [&](const Unit& f) {
    if (wave + done * kWaves < HB) {
      const BlockScale sg(f.sg), su(f.su);
      add_products(f.w[0], f.x, sg, sum[0]);
      add_products(f.w[1], f.x, sg, sum[1]);
      add_products(f.w[2], f.x, su, sum[2]);
      add_products(f.w[3], f.x, su, sum[3]);
    }
    if (++done < steps) return;
    done = 0;
    // the item's sums meet; another buffer each time, so that one barrier does
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      part[turn][wave][k][0][lane] = Vec::whole(of_parity(sum[k][0], sum[k][1]));
      part[turn][wave][k][1][lane] = Vec::whole(of_parity(sum[k][2], sum[k][3]));
      sum[k] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
    meet();
    const Fp8Tile t = uniform(&r.tile[at]);
    const int ct = threadIdx.x / 16, j = threadIdx.x % 16;
    if (ct < t.tokens) {
      const float* from = &part[turn][0][j / 8][j % 2][16 * (j % 8 / 2) + Vec::lane_of(ct)];
      float g = 0.f, u = 0.f;
#pragma unroll
      for (int k = 0; k < kWaves; ++k) {
        g += from[k * 4 * 2 * 64];
        u += from[k * 4 * 2 * 64 + 2 * 2 * 64];
      }
      uint16_t v[3];
      three_terms(g / (1.f + expf(-g)) * u, v);
      uint16_t* to = a.h + (int64_t)(t.at + ct) * a.Ip + rb * 16 + j;
      const int64_t plane = (int64_t)a.T * a.k * a.Ip;
#pragma unroll
      for (int k = 0; k < 3; ++k) to[k * plane] = v[k];
      if (rb == (int)gridDim.x - 1)
        for (int z = 16; rb * 16 + z < a.Ip; z += 16)
#pragma unroll
          for (int k = 0; k < 3; ++k) to[k * plane + z] = 0;
    }
    turn ^= 1;
    at += gridDim.y;
  };
  Unit f[kAhead];
#pragma unroll
  for (int k = 0; k < kAhead; ++k) load(f[k]);
  int left = ((tiles - 1 - (int)blockIdx.y) / (int)gridDim.y + 1) * steps;  // blocks of K
  for (; left > kAhead; left -= kAhead) {
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      products(f[k]);
      load(f[k]);
    }
  }
#pragma unroll
  for (int k = 0; k < kAhead; ++k)
    if (k < left) products(f[k]);
}

// Second half: 8 OPS rows of down x every token, over all tiles. Waves are KS x NG: wave (s, g)
// takes the blocks s, s + KS, ... of K of the tiles g, g + NG, ..., one sequence of which it has
// kAhead under way. What they give an assignment goes to LDS, one place for each assignment
// and s, and is added there with the assignments' weights in the order of the experts: so a
// token's sums do not turn on which others there are. Where LDS does not hold all places, they
// go in windows of `window`, which the last tile of one may run over.
struct DownShape {
  int ks, slots, window;
};

template <typename ACT, int WAVES, int OPS>
__global__ __launch_bounds__(64 * WAVES, 4) void k_f8_down(Fp8LayerArgs a, DownShape d) {
  typedef Vectors<3> Vec;
  static_assert(Vec::kTokens == kDownTokens, "the tables' tiles");
  constexpr int kAhead = 3;  // six or four: a token on 2048 / 768 20.1 us (18.8), the others the same
  constexpr int kOf = kRows * OPS;                                     // rows of the workgroup
  constexpr int kOut = (kF8LayerTokens * kOf - 1) / (64 * WAVES) + 1;  // outputs of a thread
  extern __shared__ __attribute__((aligned(16))) float acc[];  // [ks][slots][kOf]
  const int n = a.T * a.k;
  Fp8Tile* tile = reinterpret_cast<Fp8Tile*>(acc + d.ks * d.slots * kOf);
  float* gates = reinterpret_cast<float*>(tile + n);
  uint32_t* place = reinterpret_cast<uint32_t*>(gates + n);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), i = lane & 15, q = lane >> 4;
  const int HB = f8_blocks(a.H), IB = f8_blocks(a.I), pieces = a.I / 16, n0 = blockIdx.x * kOf;
  for (int k = threadIdx.x; k < n; k += 64 * WAVES) {
    tile[k] = a.tables->tile[k];
    gates[k] = a.tables->gate[k];
    place[k] = a.tables->place[k];
  }
  const int tiles = __builtin_amdgcn_readfirstlane(a.tables->tiles), places = __builtin_amdgcn_readfirstlane(a.tables->places);
  __syncthreads();
  const int ks = wave % d.ks, g = wave / d.ks, groups = WAVES / d.ks, steps = (IB + d.ks - 1) / d.ks;
  const int own = 2 * q + (i & 1), c = Vec::token(i / 2), zero = lane_zero();  // own: piece of a block
  const __amdgpu_buffer_rsrc_t hs = values_buffer(a.h, (int64_t)3 * n * a.Ip);
  const uint32_t own_h = 2 * (Vec::term(i / 2) * n * a.Ip + own * 16);
  const int row = (i / 2) * a.I;  // within eight rows

  struct Unit {
    f8i4 w[OPS];
    Values h;
    float s;
  };
  float y[kOut] = {};
  int end = 0;
  for (int base = 0; base < places; base += d.window) {
    const int begin = end;  // the window's tiles
    end = tiles;
    if (base + d.window < places) {
      int lo = begin;
      while (lo < end) {  // the first tile past the window
        const int mid = (lo + end) / 2;
        if (tile[mid].at < base + d.window)
          lo = mid + 1;
        else
          end = mid;
      }
      end = __builtin_amdgcn_readfirstlane(end);
    }
    int next = begin + g, step = 0;  // what the loads are at
    const uint8_t* w = nullptr;
    uint32_t h = 0;
    const float* s = nullptr;
    auto load = [&](Unit& f) {
      if (step == 0) {
        const Fp8Tile t = uniform(&tile[min(next, tiles - 1)]);
        w = a.q_dn + ((int64_t)t.expert * a.H + n0) * a.I;
        s = a.s_dn + ((int64_t)t.expert * HB + n0 / kF8Block) * IB;
        h = c < t.tokens ? own_h + 2 * (t.at + c) * a.Ip : kNoVector;
      }
      const int b = min(ks + step * d.ks, IB - 1), at = row + 16 * min(b * 8 + own, pieces - 1);
#pragma unroll
      for (int k = 0; k < OPS; ++k) f.w[k] = *(g_f8i4*)(w + at + k * kRows * a.I);
      f.h = load_values(hs, h + 2 * b * kF8Block);
      f.s = s[b + zero];
      if (++step == steps) {
        step = 0;
        next += groups;
      }
    };
    int at = begin + g, done = 0;  // what the sums are at
    f32x4 sum[OPS] = {};           // rows 2 q and 2 q + 1 of each eight
    auto products = [&](const Unit& f) {
      if (ks + done * d.ks < IB) {
        const BlockScale scale(f.s);
#pragma unroll
        for (int k = 0; k < OPS; ++k) add_products(f.w[k], f.h, scale, sum[k]);
      }
      if (++done < steps) return;
      done = 0;
      const Fp8Tile t = uniform(&tile[at]);
#pragma unroll
      for (int k = 0; k < OPS; ++k) {
        const float v0 = Vec::whole(of_parity(sum[k][0], sum[k][1])), v1 = Vec::whole(of_parity(sum[k][2], sum[k][3]));
        sum[k] = f32x4{0.f, 0.f, 0.f, 0.f};
        if (Vec::is_first(i) && c < t.tokens) {
          float* to = &acc[(ks * d.slots + t.at + c - base) * kOf + 8 * k + 2 * q];
          to[0] = v0;
          to[1] = v1;
        }
      }
      at += groups;
    };
    Unit f[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) load(f[k]);
    int left = at < end ? ((end - 1 - at) / groups + 1) * steps : 0;  // blocks of K
    for (; left > kAhead; left -= kAhead) {
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        products(f[k]);
        load(f[k]);
      }
    }
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
      if (k < left) products(f[k]);
    meet();
#pragma unroll
    for (int o = 0; o < kOut; ++o) {
      const int out = threadIdx.x + o * 64 * WAVES, t = out / kOf, r = out % kOf;
      if (t >= a.T) break;
      constexpr int kAt = 4;  // assignments at once
      for (int j = 0; j < a.k; j += kAt) {
        const float* from[kAt];
        float gate[kAt], v[kAt];
        bool is[kAt];
#pragma unroll
        for (int u = 0; u < kAt; ++u) {
          const uint32_t at = place[t * a.k + min(j + u, a.k - 1)];
          const int p = at & 0xFFFF, first = at >> 16;
          is[u] = j + u < a.k && first >= base && first < base + d.window;
          from[u] = acc + (is[u] ? p - base : 0) * kOf + r;
          gate[u] = gates[is[u] ? p : 0];
          v[u] = 0.f;
        }
        for (int k = 0; k < d.ks; ++k)
#pragma unroll
          for (int u = 0; u < kAt; ++u) v[u] += from[u][k * d.slots * kOf];
#pragma unroll
        for (int u = 0; u < kAt; ++u) y[o] = is[u] ? fmaf(gate[u], v[u], y[o]) : y[o];
      }
    }
    meet();
  }
#pragma unroll
  for (int o = 0; o < kOut; ++o) {
    const int out = threadIdx.x + o * 64 * WAVES, t = out / kOf, col = n0 + out % kOf;
    if (t >= a.T) break;
    a.y[t * a.ld_y + col] = y[o];
    if (a.x_out) {
      typedef OutElem<sizeof(ACT) == 2> Out;
      const float x = Out::load(static_cast<const ACT*>(a.x)[t * a.ld_x + col]) + y[o];
      static_cast<ACT*>(a.x_out)[t * a.ld_x_out + col] = Out::rounded(x);
    }
  }
}

template <typename ACT, int WAVES, int OPS>
void down(const Fp8LayerArgs& a, hipStream_t s) {
  const int IB = f8_blocks(a.I), n = a.T * a.k;
  // K in two parts from 4 blocks on and in four from 16, where that leaves a wave at most an eighth of its steps
  // without a block: fewer tiles then have to be at hand for every wave to have work, but the sums of more parts
  // meet in LDS. A token (16 tokens) on H = 2048, in 1 / 2 / 4 / 8 parts, us: I = 256 13.8 / 14.5 / 15.1 / - (30.3 /
  // 31.2 / 38.0), 512 13.0 / 12.8 / 13.6 / 14.1 (32.4 / 33.2 / 34.2 / 40.4), 768 17.8 / 17.3 / 18.7 / 19.9 (57.0 / 57.6 /
  // 63.8 / 67.6), 2048 18.9 / 18.6 / 18.7 / 19.1 (76.7 / 77.2 / 78.2 / 78.9), 4096 20.2 / 18.5 / 18.2 / 18.3 (76.0 / 75.6 /
  // 76.8 / 77.5); as many parts as waves 20.1 (81.4) on 2048.
  int ks = 1;
  for (int p : {2, 4})
    if (IB >= p * p && (IB + p - 1) / p * p * 7 <= IB * 8) ks = p;
  constexpr int kRoom = WAVES == 8 ? 48 << 10 : 96 << 10;  // LDS for the sums: two workgroups a CU, or one
  const int place = kRows * OPS * (int)sizeof(float), room = kRoom / (ks * place);
  DownShape d;
  d.ks = ks;
  d.slots = std::min(n, room);
  d.window = n <= room ? n : room - (kDownTokens - 1);
  const size_t lds = (size_t)ks * d.slots * place + (sizeof(Fp8Tile) + sizeof(float) + sizeof(uint32_t)) * n;
  hipLaunchKernelGGL((k_f8_down<ACT, WAVES, OPS>), dim3(a.H / (kRows * OPS)), dim3(64 * WAVES), lds, s, a, d);
}

template <typename ACT>
void layer(const Fp8LayerArgs& a, hipStream_t s) {
  constexpr int kTerms = sizeof(ACT) == 2 ? 1 : 3;
  const int rows = a.logits_in ? 0 : a.E;
  hipLaunchKernelGGL((k_f8_router<ACT>), dim3(rows + a.T), dim3(kRouterThreads), 0, s, a, rows);
  // blocks of rows; tiles, shared by as many workgroups as the CUs hold at two each: 16 tokens on 2048 / 768, 8 of
  // 128 experts, 71.5 us (one each: 70.6, four: 75.6, half as many as CUs: 95.7), 64 tokens 183 (183, 197, 245), 16 on
  // 7168 / 2048 341 (336, 339, 417), on 4096 / 256 55.7 (55.1, 61.1, 61.0), 40 on 1024 / 4096 185 (187, 194, 187)
  const int per = a.I / 16, most = a.T * a.k;
  const dim3 grid(per, std::min(most, std::max(1, 2 * kCus / per)));
  hipLaunchKernelGGL((k_f8_gate_up<kTerms>), grid, dim3(64 * kWaves), 0, s, a);
  // 8 rows and twice the waves a workgroup, which takes a CU to itself, while one round of the CUs holds them:
  // H = 2048 17.5 us for a token and 66 for 16 (8 of 64 experts, I = 768; 16 rows: 18.2 and 74). Above, two
  // workgroups of 16 rows a CU, which read each vector half as often: H = 2064 19.4 and 82 (8 rows: 21.9 and
  // 94), 4096 27 and 97 (30 and 111), 7168 39 and 172 (47 and 198).
  if (a.H / kRows <= kCus)
    down<ACT, 16, 1>(a, s);
  else
    down<ACT, 8, 2>(a, s);
}

}  // namespace

void launch_fp8_layer(const Fp8LayerArgs& a, bool act_bf16, hipStream_t s) {
  if (act_bf16)
    layer<uint16_t>(a, s);
  else
    layer<float>(a, s);
}

}  // namespace moe
