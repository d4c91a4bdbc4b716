// Internal interface of the dense operators beside the routed layer: the row
// kernels (norm, 8-bit codes of rows) and the 8-bit matrix products. Every leading
// dimension is in elements; the entry points have checked every argument.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>
#include <string>

#include "moe_offload.h"

namespace moe {

// Sets the calling thread's moe_last_error() message and returns `s`.
moe_status report_error(moe_status s, const char* msg) noexcept;

// Largest row of the row kernels, which hold a row in registers.
constexpr int kRowMax = 16384;

struct RowArgs {
  const void* x;       // [T][H] act
  const void* add;     // [T][H] act or fp32, or null (norm only)
  const void* weight;  // [H] act (norm only)
  void* x_out;         // [T][H] act, or null: act(x + add)
  void* out;           // [T][H] act, or null: the norm
  int8_t* q;           // [T][H] codes, or null
  float* s;            // [T] scales of the codes
  int64_t ld_x, ld_add, ld_x_out, ld_out, ld_q;
  int T, H;
  int act_bf16, add_f32;
  float eps;
};
void launch_rms_norm(const RowArgs& a, hipStream_t s);
void launch_quantize_rows(const RowArgs& a, hipStream_t s);

// What the product's epilogue reads and writes: out = act(acc sx sw + bias + y + res).
struct Int8Out {
  const float* sx;    // [T]
  const float* sw;    // [N]
  const float* bias;  // [N] or null
  const float* y;     // [T][N] or null
  const void* res;    // [T][N] of out's type, or null
  void* out;          // [T][N]
  int64_t ld_y, ld_res, ld_out;
};

struct Int8Args {
  const int8_t* x;  // [T][K] codes
  const int8_t* w;  // [N][K] codes; gated: [2N][K], gate rows, then up rows
  int64_t ld_x, ld_w;
  int T, N, K;
  Int8Out o;
};
// out = the product's epilogue, in bf16 or fp32
void launch_int8_matmul(const Int8Args& a, bool out_bf16, hipStream_t s);
// out = h [T][N] fp32 = silu(gate) * up
void launch_int8_gated(const Int8Args& a, hipStream_t s);
// The gated block's second half for a few tokens: the codes of h [T][K] fp32 and their
// product in one kernel (a.x and a.o.sx are not read); the same bits as launch_quantize_rows and
// launch_int8_matmul. Only where int8_down_fits.
bool int8_down_fits(int T, int K);
void launch_int8_down(const Int8Args& a, const float* h, bool out_bf16, hipStream_t s);
// the first two for many rows
void launch_int8_gemm(const Int8Args& a, bool out_bf16, hipStream_t s);
void launch_int8_gated_gemm(const Int8Args& a, hipStream_t s);

}  // namespace moe
