// Entry points of the dense operators beside the routed layer: norm, codes of rows,
// the 8-bit product and the gated block. Each checks its arguments and enqueues its
// kernels; none allocates, synchronises or keeps anything between calls.
#include "dense.h"

#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdarg>
#include <cstdio>

using namespace moe;

namespace {

constexpr int kMaxRows = 1 << 20;   // T
constexpr int kMaxWidth = 1 << 24;  // N
constexpr int kMaxK = 131056;       // 128 * 128 * K stays within int32

moe_status bad(const char* fmt, ...) {
  char msg[256];
  va_list ap;
  va_start(ap, fmt);
  std::vsnprintf(msg, sizeof(msg), fmt, ap);
  va_end(ap);
  return report_error(MOE_E_INVALID, msg);
}

// A matrix argument: rows x cols elements of `size` bytes, row stride `ld` elements.
struct Mat {
  const char* name;
  const void* p;
  int64_t rows, cols, ld;
  int size;
  const char* begin() const { return static_cast<const char*>(p); }
  const char* end() const { return begin() + ((rows - 1) * ld + cols) * size; }
};

// A required (or, if null is allowed, given) matrix with a sound stride and address;
// a stride of 0 stands for packed rows and is replaced.
moe_status check_mat(Mat& m, bool required, int align) {
  if (!m.p) return required ? bad("%s is required", m.name) : MOE_OK;
  if (m.ld == 0) m.ld = m.cols;
  // (a single row, such as a large workspace, has no stride that an address is formed with)
  if (m.ld < m.cols || (m.rows > 1 && m.ld > (int64_t(1) << 36))) return bad("%s: row stride %lld is under %lld or too large", m.name, (long long)m.ld, (long long)m.cols);
  if (reinterpret_cast<uintptr_t>(m.p) % align) return bad("%s must be %d-byte aligned", m.name, align);
  if (m.rows > 1 && m.ld * m.size % align) return bad("%s: rows must be %d-byte aligned", m.name, align);
  return MOE_OK;
}

// Whether two matrices share elements. Rows of one stride side by side, as in a fused
// projection's output, do not; rows of unlike strides are taken to where their extents meet.
bool overlap(const Mat& a, const Mat& b) {
  if (!a.p || !b.p || a.begin() >= b.end() || b.begin() >= a.end()) return false;
  const int64_t la = a.rows > 1 ? a.ld * a.size : 0, lb = b.rows > 1 ? b.ld * b.size : 0;
  const int64_t ld = la ? la : lb;  // a single row may stand beside the other's
  if (!ld || (la && lb && la != lb)) return true;
  // a's rows are at 0 .. of every ld bytes, b's at d ..
  const int64_t d = ((b.begin() - a.begin()) % ld + ld) % ld;
  return d < a.cols * a.size || d + b.cols * b.size > ld;
}
// the same elements at the same places: a row's reader may write them
bool same(const Mat& a, const Mat& b) {
  return a.p == b.p && a.size == b.size && a.rows == b.rows && a.cols == b.cols && (a.ld == b.ld || a.rows == 1);
}

moe_status apart(const Mat& out, const Mat& in) {
  return overlap(out, in) ? bad("%s overlaps %s", out.name, in.name) : MOE_OK;
}
moe_status apart_or_same(const Mat& out, const Mat& in) { return same(out, in) ? MOE_OK : apart(out, in); }

#define CHECK(expr)                   \
  do {                                \
    const moe_status _s = (expr);     \
    if (_s != MOE_OK) return _s;      \
  } while (0)

moe_status hip_failed(const char* what, hipError_t e) {
  char msg[256];
  std::snprintf(msg, sizeof(msg), "%s: %s", what, hipGetErrorString(e));
  return report_error(MOE_E_HIP, msg);
}

// Work is enqueued with the stream's device current, whichever the caller's is.
class OnStreamDevice {
 public:
  explicit OnStreamDevice(hipStream_t s) {
    hipDevice_t dev = 0;
    if (s && (error_ = hipGetDevice(&prev_)) == hipSuccess && (error_ = hipStreamGetDevice(s, &dev)) == hipSuccess && dev != prev_) {
      error_ = hipSetDevice(dev);
      changed_ = error_ == hipSuccess;
    }
    // launched() asks for the thread's last error: what the caller's own calls left there is
    // not a launch's
    (void)hipGetLastError();
  }
  ~OnStreamDevice() {
    if (changed_) (void)hipSetDevice(prev_);
  }
  moe_status ready() const { return error_ == hipSuccess ? MOE_OK : hip_failed("the stream's device", error_); }

 private:
  hipError_t error_ = hipSuccess;
  int prev_ = 0;
  bool changed_ = false;
};

moe_status launched(const char* what) {
  const hipError_t e = hipGetLastError();
  if (e == hipSuccess) return MOE_OK;
  char msg[64];
  std::snprintf(msg, sizeof(msg), "launching %s", what);
  return hip_failed(msg, e);
}

int act_size(int dtype) { return dtype == MOE_ACT_BF16 ? 2 : 4; }

moe_status check_act(const char* name, int dtype) {
  return dtype == MOE_ACT_BF16 || dtype == MOE_ACT_F32 ? MOE_OK : bad("%s is neither MOE_ACT_F32 nor MOE_ACT_BF16", name);
}

moe_status check_rows(int T, int H) {
  if (T < 0 || T > kMaxRows) return bad("T out of range 0..%d", kMaxRows);
  if (H < 1 || H > kRowMax) return bad("H out of range 1..%d", kRowMax);
  return MOE_OK;
}

moe_status check_k(const char* name, int K) {
  if (K < 16 || K > kMaxK || K % 16) return bad("%s must be a multiple of 16 in 16..%d", name, kMaxK);
  return MOE_OK;
}

// Codes are read in 16-byte pieces.
moe_status check_codes(Mat& m) { return check_mat(m, true, 16); }

struct Epilogue {
  Mat y, res, out;
};

moe_status check_epilogue(Epilogue& e) {
  CHECK(check_mat(e.out, true, e.out.size));
  CHECK(check_mat(e.y, false, 4));
  CHECK(check_mat(e.res, false, e.res.size));
  if (e.y.p) CHECK(apart_or_same(e.out, e.y));
  if (e.res.p) CHECK(apart_or_same(e.out, e.res));
  return MOE_OK;
}

size_t up256(size_t n) { return (n + 255) & ~size_t(255); }

// the block's workspace: h [T][I] fp32 | codes [T][I] | scales [T]
struct FfnSpace {
  size_t h = 0, q, s, bytes;
  FfnSpace(int64_t T, int64_t I) {
    q = up256(sizeof(float) * T * I);
    s = q + up256(T * I);
    bytes = s + up256(sizeof(float) * T);
  }
};

moe_status check_ffn_shape(int T, int H, int I) {
  if (T < 0 || T > kMaxRows) return bad("T out of range 0..%d", kMaxRows);
  CHECK(check_k("H", H));
  CHECK(check_k("I", I));
  if (I > kRowMax) return bad("I out of range 16..%d", kRowMax);
  return MOE_OK;
}

}  // namespace

extern "C" {

moe_status moe_rms_norm(const moe_rms_norm_args* a, moe_stream stream) {
  if (!a) return bad("args is null");
  CHECK(check_rows(a->T, a->H));
  CHECK(check_act("act_dtype", a->act_dtype));
  if (a->add) {
    CHECK(check_act("add_dtype", a->add_dtype));
    if (a->add_dtype == MOE_ACT_BF16 && a->act_dtype != MOE_ACT_BF16) return bad("add_dtype must be act_dtype or MOE_ACT_F32");
  }
  if (!(a->eps > 0.f) || !std::isfinite(a->eps)) return bad("eps must be positive and finite");
  if (a->T == 0) return MOE_OK;
  const int sz = act_size(a->act_dtype), T = a->T, H = a->H;
  Mat x{"x", a->x, T, H, a->ld_x, sz}, add{"add", a->add, T, H, a->ld_add, act_size(a->add_dtype)};
  Mat w{"weight", a->weight, 1, H, H, sz}, xo{"x_out", a->x_out, T, H, a->ld_x_out, sz};
  Mat out{"out", a->out, T, H, a->ld_out, sz}, q{"q_out", a->q_out, T, H, a->ld_q, 1}, s{"s_out", a->s_out, 1, T, T, 4};
  CHECK(check_mat(x, true, sz));
  CHECK(check_mat(add, false, add.size));
  CHECK(check_mat(w, true, sz));
  CHECK(check_mat(xo, false, sz));
  CHECK(check_mat(out, false, sz));
  CHECK(check_mat(q, false, 1));
  CHECK(check_mat(s, false, 4));
  if (!xo.p && !out.p && !q.p) return bad("no output is given");
  if (!q.p != !s.p) return bad("q_out and s_out are given together");
  if (xo.p && !add.p) return bad("x_out needs add");
  const Mat* outs[] = {&xo, &out, &q, &s};
  for (int i = 0; i < 4; ++i) {
    const bool may_be = i < 2;  // x_out and out may be x or add
    for (const Mat* in : {&x, &add}) CHECK(may_be ? apart_or_same(*outs[i], *in) : apart(*outs[i], *in));
    CHECK(apart(*outs[i], w));
    for (int j = 0; j < i; ++j) CHECK(apart(*outs[i], *outs[j]));
  }
  RowArgs r{x.p,  add.p, w.p,   a->x_out, a->out, a->q_out,
            a->s_out, x.ld, add.ld, xo.ld, out.ld, q.ld, T, H, a->act_dtype == MOE_ACT_BF16,
            a->add_dtype == MOE_ACT_F32, a->eps};
  const OnStreamDevice on(static_cast<hipStream_t>(stream));
  CHECK(on.ready());
  launch_rms_norm(r, static_cast<hipStream_t>(stream));
  return launched("the norm");
}

moe_status moe_quantize_rows(const moe_quantize_args* a, moe_stream stream) {
  if (!a) return bad("args is null");
  CHECK(check_rows(a->T, a->H));
  CHECK(check_act("act_dtype", a->act_dtype));
  if (a->T == 0) return MOE_OK;
  const int sz = act_size(a->act_dtype);
  Mat x{"x", a->x, a->T, a->H, a->ld_x, sz}, q{"q_out", a->q_out, a->T, a->H, a->ld_q, 1}, s{"s_out", a->s_out, 1, a->T, a->T, 4};
  CHECK(check_mat(x, true, sz));
  CHECK(check_mat(q, true, 1));
  CHECK(check_mat(s, true, 4));
  CHECK(apart(q, x));
  CHECK(apart(s, x));
  CHECK(apart(s, q));
  RowArgs r{};
  r.x = x.p;
  r.q = a->q_out;
  r.s = a->s_out;
  r.ld_x = x.ld;
  r.ld_q = q.ld;
  r.T = a->T;
  r.H = a->H;
  r.act_bf16 = a->act_dtype == MOE_ACT_BF16;
  const OnStreamDevice on(static_cast<hipStream_t>(stream));
  CHECK(on.ready());
  launch_quantize_rows(r, static_cast<hipStream_t>(stream));
  return launched("the rows' codes");
}

moe_status moe_int8_matmul(const moe_int8_matmul_args* a, moe_stream stream) {
  if (!a) return bad("args is null");
  if (a->T < 0 || a->T > kMaxRows) return bad("T out of range 0..%d", kMaxRows);
  if (a->N < 1 || a->N > kMaxWidth) return bad("N out of range 1..%d", kMaxWidth);
  CHECK(check_k("K", a->K));
  CHECK(check_act("out_dtype", a->out_dtype));
  if (a->T == 0) return MOE_OK;
  const int T = a->T, N = a->N, K = a->K, sz = act_size(a->out_dtype);
  Mat x{"q_x", a->q_x, T, K, a->ld_x, 1}, w{"q_w", a->q_w, N, K, a->ld_w, 1};
  Mat sx{"s_x", a->s_x, 1, T, T, 4}, sw{"s_w", a->s_w, 1, N, N, 4}, bias{"bias", a->bias, 1, N, N, 4};
  Epilogue e{{"y_in", a->y_in, T, N, a->ld_y, 4}, {"res", a->res, T, N, a->ld_res, sz}, {"out", a->out, T, N, a->ld_out, sz}};
  CHECK(check_codes(x));
  CHECK(check_codes(w));
  CHECK(check_mat(sx, true, 4));
  CHECK(check_mat(sw, true, 4));
  CHECK(check_mat(bias, false, 4));
  CHECK(check_epilogue(e));
  for (const Mat* in : {&x, &w, &sx, &sw, &bias}) CHECK(apart(e.out, *in));
  const Int8Args g{a->q_x, a->q_w, x.ld, w.ld, T, N, K,
                   {a->s_x, a->s_w, a->bias, a->y_in, a->res, a->out, e.y.ld, e.res.ld, e.out.ld}};
  const OnStreamDevice on(static_cast<hipStream_t>(stream));
  CHECK(on.ready());
  launch_int8_matmul(g, a->out_dtype == MOE_ACT_BF16, static_cast<hipStream_t>(stream));
  return launched("the 8-bit product");
}

moe_status moe_int8_ffn_workspace(int32_t T, int32_t H, int32_t I, size_t* bytes) {
  if (!bytes) return bad("bytes is null");
  *bytes = 0;
  CHECK(check_ffn_shape(T, H, I));
  *bytes = FfnSpace(T, I).bytes;
  return MOE_OK;
}

moe_status moe_int8_ffn(const moe_int8_ffn_args* a, moe_stream stream) {
  if (!a) return bad("args is null");
  CHECK(check_ffn_shape(a->T, a->H, a->I));
  CHECK(check_act("out_dtype", a->out_dtype));
  if (a->T == 0) return MOE_OK;
  const int T = a->T, H = a->H, I = a->I, sz = act_size(a->out_dtype);
  const FfnSpace f(T, I);
  Mat x{"q_x", a->q_x, T, H, a->ld_x, 1}, gu{"q_gu", a->q_gu, 2 * (int64_t)I, H, a->ld_gu, 1}, dn{"q_dn", a->q_dn, H, I, a->ld_dn, 1};
  Mat sx{"s_x", a->s_x, 1, T, T, 4}, sgu{"s_gu", a->s_gu, 1, 2 * I, 2 * I, 4}, sdn{"s_dn", a->s_dn, 1, H, H, 4};
  Mat ws{"workspace", a->workspace, 1, (int64_t)f.bytes, (int64_t)f.bytes, 1};
  Epilogue e{{"y_in", a->y_in, T, H, a->ld_y, 4}, {"res", a->res, T, H, a->ld_res, sz}, {"out", a->out, T, H, a->ld_out, sz}};
  CHECK(check_codes(x));
  CHECK(check_codes(gu));
  CHECK(check_codes(dn));
  CHECK(check_mat(sx, true, 4));
  CHECK(check_mat(sgu, true, 4));
  CHECK(check_mat(sdn, true, 4));
  CHECK(check_epilogue(e));
  CHECK(check_mat(ws, true, 256));
  if (a->workspace_bytes < f.bytes)
    return bad("the workspace holds %zu bytes, %zu are needed (moe_int8_ffn_workspace)", a->workspace_bytes, f.bytes);
  for (const Mat* in : {&x, &gu, &dn, &sx, &sgu, &sdn}) {
    CHECK(apart(e.out, *in));
    CHECK(apart(ws, *in));
  }
  for (const Mat* m : {&e.y, &e.res, &e.out}) CHECK(apart(ws, *m));
  uint8_t* base = static_cast<uint8_t*>(a->workspace);
  float* h = reinterpret_cast<float*>(base + f.h);
  int8_t* q = reinterpret_cast<int8_t*>(base + f.q);
  float* s = reinterpret_cast<float*>(base + f.s);
  const hipStream_t st = static_cast<hipStream_t>(stream);
  const OnStreamDevice on(st);
  CHECK(on.ready());
  Int8Args g{a->q_x, a->q_gu, x.ld, gu.ld, T, I, H, {a->s_x, a->s_gu, nullptr, nullptr, nullptr, h, 0, 0, I}};
  launch_int8_gated(g, st);
  CHECK(launched("the gated product"));
  Int8Args d{q, a->q_dn, I, dn.ld, T, H, I,
             {s, a->s_dn, nullptr, a->y_in, a->res, a->out, e.y.ld, e.res.ld, e.out.ld}};
  if (int8_down_fits(T, I)) {
    launch_int8_down(d, h, a->out_dtype == MOE_ACT_BF16, st);
    return launched("the block's second product");
  }
  RowArgs r{};
  r.x = h;
  r.q = q;
  r.s = s;
  r.ld_x = r.ld_q = I;
  r.T = T;
  r.H = I;
  launch_quantize_rows(r, st);
  CHECK(launched("the codes of h"));
  launch_int8_matmul(d, a->out_dtype == MOE_ACT_BF16, st);
  return launched("the block's second product");
}

}  // extern "C"
