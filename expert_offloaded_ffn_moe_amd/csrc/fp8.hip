// Entry points of the operators on e4m3 codes with a scale for each block of 128: codes,
// the matrix product and the whole layer of a few tokens. Each checks its arguments and
// enqueues its kernels; none allocates, synchronises or keeps anything between calls.
#include "fp8.h"

#include <hip/hip_runtime.h>

#include "args.h"
#include "dense.h"

using namespace moe;

namespace {

constexpr int kMaxK = 131056;       // columns of a matrix that products read
constexpr int kMaxColumns = 1 << 20;  // of one that is coded
constexpr int kMaxI = 16384;

moe_status check_k(const char* name, int K, int most) {
  if (K < 16 || K > most || K % 16) return bad("%s must be a multiple of 16 in 16..%d", name, most);
  return MOE_OK;
}

moe_status check_layer_shape(int T, int H, int I, int E, int k) {
  if (T < 0 || T > kF8LayerTokens) return bad("T out of range 0..%d", kF8LayerTokens);
  CHECK(check_k("H", H, kMaxK));
  CHECK(check_k("I", I, kMaxI));
  if (E < 1 || E > kF8LayerExperts) return bad("E out of range 1..%d", kF8LayerExperts);
  if (k < 1 || k > E || k > kF8LayerTopK) return bad("k out of range 1..min(E, %d)", kF8LayerTopK);
  return MOE_OK;
}

// the layer's workspace: tables | logits [T][E] | bf16 terms of the activations [3][T][H] and of
// the intermediate [3][T k][I], H and I up to whole blocks
struct LayerSpace {
  size_t tables = 0, logits, x, h, bytes;
  LayerSpace(int64_t T, int64_t H, int64_t I, int64_t E, int64_t k) {
    logits = up256(sizeof(Fp8Tables));
    x = logits + up256(sizeof(float) * T * E);
    h = x + up256(3 * sizeof(uint16_t) * T * f8_blocks(H) * kF8Block);
    bytes = h + up256(3 * sizeof(uint16_t) * T * k * f8_blocks(I) * kF8Block);
  }
};

}  // namespace

extern "C" {

moe_status moe_fp8_quantize(const moe_fp8_quantize_args* a, moe_stream stream) {
  if (!a) return bad("args is null");
  if (a->T < 0 || a->T > kMaxRows) return bad("T out of range 0..%d", kMaxRows);
  if (a->H < 1 || a->H > kMaxColumns) return bad("H out of range 1..%d", kMaxColumns);
  CHECK(check_act("act_dtype", a->act_dtype));
  if (a->block_rows != 1 && a->block_rows != kF8Block) return bad("block_rows is neither 1 nor %d", kF8Block);
  if (a->T == 0) return MOE_OK;
  const int sz = act_size(a->act_dtype), T = a->T, H = a->H;
  Mat x{"x", a->x, T, H, a->ld_x, sz}, q{"q_out", a->q_out, T, H, a->ld_q, 1};
  Mat s{"s_out", a->s_out, (T - 1) / a->block_rows + 1, f8_blocks(H), a->ld_s, 4};
  CHECK(check_mat(x, true, sz));
  CHECK(check_mat(q, true, 1));
  CHECK(check_mat(s, true, 4));
  CHECK(apart(q, x));
  CHECK(apart(s, x));
  CHECK(apart(s, q));
  const Fp8QuantArgs r{a->x, a->q_out, a->s_out, x.ld, q.ld, s.ld, T, H};
  const hipStream_t st = static_cast<hipStream_t>(stream);
  const OnStreamDevice on(st);
  CHECK(on.ready());
  launch_fp8_quantize(r, a->act_dtype == MOE_ACT_BF16, a->block_rows, st);
  return launched("the blocks' codes");
}

moe_status moe_fp8_matmul(const moe_fp8_matmul_args* a, moe_stream stream) {
  if (!a) return bad("args is null");
  if (a->T < 0 || a->T > kMaxRows) return bad("T out of range 0..%d", kMaxRows);
  if (a->N < 1 || a->N > kMaxWidth) return bad("N out of range 1..%d", kMaxWidth);
  CHECK(check_k("K", a->K, kMaxK));
  CHECK(check_act("out_dtype", a->out_dtype));
  if (a->T == 0) return MOE_OK;
  const int T = a->T, N = a->N, K = a->K, sz = act_size(a->out_dtype), KB = f8_blocks(K);
  Mat x{"q_x", a->q_x, T, K, a->ld_x, 1}, w{"q_w", a->q_w, N, K, a->ld_w, 1};
  Mat sx{"s_x", a->s_x, T, KB, a->ld_sx, 4}, sw{"s_w", a->s_w, f8_blocks(N), KB, a->ld_sw, 4}, bias{"bias", a->bias, 1, N, N, 4};
  Epilogue e{{"y_in", a->y_in, T, N, a->ld_y, 4}, {"res", a->res, T, N, a->ld_res, sz}, {"out", a->out, T, N, a->ld_out, sz}};
  CHECK(check_mat(x, true, 16));
  CHECK(check_mat(w, true, 16));
  CHECK(check_mat(sx, true, 4));
  CHECK(check_mat(sw, true, 4));
  CHECK(check_mat(bias, false, 4));
  CHECK(check_epilogue(e));
  for (const Mat* in : {&x, &w, &sx, &sw, &bias}) CHECK(apart(e.out, *in));
  const Fp8Args g{a->q_x, a->q_w, a->s_x, a->s_w, x.ld, w.ld, sx.ld, sw.ld, T, N, K,
                  {a->bias, a->y_in, a->res, a->out, e.y.ld, e.res.ld, e.out.ld}};
  const hipStream_t st = static_cast<hipStream_t>(stream);
  const OnStreamDevice on(st);
  CHECK(on.ready());
  launch_fp8_matmul(g, a->out_dtype == MOE_ACT_BF16, st);
  return launched("the product of blocks");
}

moe_status moe_fp8_layer_workspace(int32_t T, int32_t H, int32_t I, int32_t E, int32_t k, size_t* bytes) {
  if (!bytes) return bad("bytes is null");
  *bytes = 0;
  CHECK(check_layer_shape(T, H, I, E, k));
  *bytes = LayerSpace(T, H, I, E, k).bytes;
  return MOE_OK;
}

moe_status moe_fp8_layer(const moe_fp8_layer_args* a, moe_stream stream) {
  if (!a) return bad("args is null");
  CHECK(check_layer_shape(a->T, a->H, a->I, a->E, a->k));
  CHECK(check_act("act_dtype", a->act_dtype));
  if (a->T == 0) return MOE_OK;
  const int T = a->T, H = a->H, I = a->I, E = a->E, k = a->k, sz = act_size(a->act_dtype);
  const int HB = f8_blocks(H), IB = f8_blocks(I);
  const LayerSpace f(T, H, I, E, k);
  const auto flat = [](const char* name, const void* p, int64_t n, int size) { return Mat{name, p, 1, n, n, size}; };
  Mat x{"x", a->x, T, H, a->ld_x, sz}, rw{"router_w", a->logits_in ? nullptr : a->router_w, E, H, a->ld_router, sz};
  Mat rb = flat("router_b", a->logits_in ? nullptr : a->router_b, E, 4), li = flat("logits_in", a->logits_in, (int64_t)T * E, 4);
  Mat gu = flat("q_gu", a->q_gu, (int64_t)E * 2 * I * H, 1), sgu = flat("s_gu", a->s_gu, (int64_t)E * 2 * IB * HB, 4);
  Mat dn = flat("q_dn", a->q_dn, (int64_t)E * H * I, 1), sdn = flat("s_dn", a->s_dn, (int64_t)E * HB * IB, 4);
  Mat y{"y", a->y, T, H, a->ld_y, 4}, xo{"x_out", a->x_out, T, H, a->ld_x_out, sz};
  Mat lo = flat("logits", a->logits, (int64_t)T * E, 4), ids = flat("topk_ids", a->topk_ids, T * k, 4);
  Mat w = flat("topk_w", a->topk_w, T * k, 4), ws = flat("workspace", a->workspace, (int64_t)f.bytes, 1);
  CHECK(check_mat(x, true, sz));
  CHECK(check_mat(rw, !a->logits_in, sz));
  CHECK(check_mat(rb, false, 4));
  CHECK(check_mat(li, false, 4));
  CHECK(check_mat(gu, true, 16));
  CHECK(check_mat(sgu, true, 4));
  CHECK(check_mat(dn, true, 16));
  CHECK(check_mat(sdn, true, 4));
  CHECK(check_mat(y, true, 4));
  CHECK(check_mat(xo, false, sz));
  CHECK(check_mat(lo, false, 4));
  CHECK(check_mat(ids, false, 4));
  CHECK(check_mat(w, false, 4));
  CHECK(check_mat(ws, true, 256));
  if (a->workspace_bytes < f.bytes)
    return bad("the workspace holds %zu bytes, %zu are needed (moe_fp8_layer_workspace)", a->workspace_bytes, f.bytes);
  const Mat* outs[] = {&y, &xo, &lo, &ids, &w, &ws};
  for (int i = 0; i < 6; ++i) {
    for (const Mat* in : {&rw, &rb, &li, &gu, &sgu, &dn, &sdn}) CHECK(apart(*outs[i], *in));
    CHECK(outs[i] == &xo ? apart_or_same(xo, x) : apart(*outs[i], x));
    for (int j = 0; j < i; ++j) CHECK(apart(*outs[i], *outs[j]));
  }
  uint8_t* base = static_cast<uint8_t*>(a->workspace);
  Fp8LayerArgs g{};
  g.x = a->x;
  g.router_w = a->router_w;
  g.router_b = a->router_b;
  g.logits_in = a->logits_in;
  g.q_gu = a->q_gu;
  g.s_gu = a->s_gu;
  g.q_dn = a->q_dn;
  g.s_dn = a->s_dn;
  g.y = a->y;
  g.x_out = a->x_out;
  g.logits = a->logits ? a->logits : a->logits_in ? nullptr : reinterpret_cast<float*>(base + f.logits);
  g.ids = a->topk_ids;
  g.gate = a->topk_w;
  g.h = reinterpret_cast<uint16_t*>(base + f.h);
  g.xt = reinterpret_cast<uint16_t*>(base + f.x);
  g.tables = reinterpret_cast<Fp8Tables*>(base + f.tables);
  g.ld_x = x.ld;
  g.ld_router = rw.ld;
  g.ld_y = y.ld;
  g.ld_x_out = xo.ld;
  g.T = T;
  g.H = H;
  g.I = I;
  g.E = E;
  g.k = k;
  g.Hp = HB * kF8Block;
  g.Ip = IB * kF8Block;
  const hipStream_t st = static_cast<hipStream_t>(stream);
  const OnStreamDevice on(st);
  CHECK(on.ready());
  launch_fp8_layer(g, a->act_dtype == MOE_ACT_BF16, st);
  return launched("the layer");
}

}  // extern "C"
