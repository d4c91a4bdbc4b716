// Internal interface of the operators on e4m3 codes with a scale for each block of 128.
// Every leading dimension is in elements; the entry points have checked every argument.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

namespace moe {

constexpr int kF8Block = 128;
__host__ __device__ constexpr int f8_blocks(int n) { return (n + kF8Block - 1) / kF8Block; }

struct Fp8QuantArgs {
  const void* x;  // [T][H] act
  uint8_t* q;     // [T][H]
  float* s;       // [ceil(T / rows)][ceil(H / 128)]
  int64_t ld_x, ld_q, ld_s;
  int T, H;
};
void launch_fp8_quantize(const Fp8QuantArgs& a, bool act_bf16, int block_rows, hipStream_t s);

// What the product adds and writes: out = act(sum + bias + y + res).
struct Fp8Out {
  const float* bias;  // [N] or null
  const float* y;     // [T][N] or null
  const void* res;    // [T][N] of out's type, or null
  void* out;          // [T][N]
  int64_t ld_y, ld_res, ld_out;
};

struct Fp8Args {
  const uint8_t* x;  // [T][K]
  const uint8_t* w;  // [N][K]
  const float* sx;   // [T][ceil(K/128)]
  const float* sw;   // [ceil(N/128)][ceil(K/128)]
  int64_t ld_x, ld_w, ld_sx, ld_sw;
  int T, N, K;
  Fp8Out o;
};
void launch_fp8_matmul(const Fp8Args& a, bool out_bf16, hipStream_t s);
// for many rows
void launch_fp8_gemm(const Fp8Args& a, bool out_bf16, hipStream_t s);

constexpr int kF8LayerTokens = 64, kF8LayerExperts = 1024, kF8LayerTopK = 32;

// Up to a few tokens of one expert: the expert, the first one's place among the assignments
// (grouped by expert, in ascending order of experts and tokens) and how many they are.
struct Fp8Tile {
  uint16_t expert, at, tokens, none;
};
struct Fp8Tables {
  Fp8Tile tile[kF8LayerTokens * kF8LayerTopK];
  float gate[kF8LayerTokens * kF8LayerTopK];  // by place
  // [T][k]: a token's places, ascending, each with its tile's first one in the upper half, then kF8NoPlace
  uint32_t place[kF8LayerTokens * kF8LayerTopK];
  int tiles, places;
};
constexpr uint32_t kF8NoPlace = ~0u;

struct Fp8LayerArgs {
  const void* x;          // [T][H] act
  const void* router_w;   // [E][H] act
  const float* router_b;  // [E] or null
  const float* logits_in; // [T][E] or null
  const uint8_t* q_gu;
  const float* s_gu;
  const uint8_t* q_dn;
  const float* s_dn;
  float* y;
  void* x_out;            // or null
  float* logits;          // [T][E]: the caller's, or the workspace's; null with logits_in alone
  int32_t* ids;           // [T][k] or null
  float* gate;            // [T][k] or null
  uint16_t* h;            // workspace: the intermediate's three bf16 terms, [3][T k][Ip]
  uint16_t* xt;           // workspace: x, or its three bf16 terms, [terms][T][Hp]
  Fp8Tables* tables;      // workspace
  int64_t ld_x, ld_router, ld_y, ld_x_out;
  int T, H, I, E, k;
  int Hp, Ip;             // H and I up to whole blocks, the rest zeros
};
void launch_fp8_layer(const Fp8LayerArgs& a, bool act_bf16, hipStream_t s);

}  // namespace moe
