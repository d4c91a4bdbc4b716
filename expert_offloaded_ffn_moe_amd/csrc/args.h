// Checks of arguments, and the launch's frame, that the entry points without a plan share.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdarg>
#include <cstdint>
#include <cstdio>

#include "dense.h"

namespace moe {
namespace {

constexpr int kMaxRows = 1 << 20;   // T
constexpr int kMaxWidth = 1 << 24;  // N

[[maybe_unused]] moe_status bad(const char* fmt, ...) {
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
[[maybe_unused]] moe_status check_mat(Mat& m, bool required, int align) {
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
[[maybe_unused]] bool overlap(const Mat& a, const Mat& b) {
  if (!a.p || !b.p || a.begin() >= b.end() || b.begin() >= a.end()) return false;
  const int64_t la = a.rows > 1 ? a.ld * a.size : 0, lb = b.rows > 1 ? b.ld * b.size : 0;
  const int64_t ld = la ? la : lb;  // a single row may stand beside the other's
  if (!ld || (la && lb && la != lb)) return true;
  // a's rows are at 0 .. of every ld bytes, b's at d ..
  const int64_t d = ((b.begin() - a.begin()) % ld + ld) % ld;
  return d < a.cols * a.size || d + b.cols * b.size > ld;
}
// the same elements at the same places: a row's reader may write them
[[maybe_unused]] bool same(const Mat& a, const Mat& b) {
  return a.p == b.p && a.size == b.size && a.rows == b.rows && a.cols == b.cols && (a.ld == b.ld || a.rows == 1);
}

[[maybe_unused]] moe_status apart(const Mat& out, const Mat& in) {
  return overlap(out, in) ? bad("%s overlaps %s", out.name, in.name) : MOE_OK;
}
[[maybe_unused]] moe_status apart_or_same(const Mat& out, const Mat& in) { return same(out, in) ? MOE_OK : apart(out, in); }

#define CHECK(expr)                   \
  do {                                \
    const moe_status _s = (expr);     \
    if (_s != MOE_OK) return _s;      \
  } while (0)

[[maybe_unused]] moe_status hip_failed(const char* what, hipError_t e) {
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

[[maybe_unused]] moe_status launched(const char* what) {
  const hipError_t e = hipGetLastError();
  if (e == hipSuccess) return MOE_OK;
  char msg[64];
  std::snprintf(msg, sizeof(msg), "launching %s", what);
  return hip_failed(msg, e);
}

[[maybe_unused]] int act_size(int dtype) { return dtype == MOE_ACT_BF16 ? 2 : 4; }

[[maybe_unused]] moe_status check_act(const char* name, int dtype) {
  return dtype == MOE_ACT_BF16 || dtype == MOE_ACT_F32 ? MOE_OK : bad("%s is neither MOE_ACT_F32 nor MOE_ACT_BF16", name);
}

struct Epilogue {
  Mat y, res, out;
};

[[maybe_unused]] moe_status check_epilogue(Epilogue& e) {
  CHECK(check_mat(e.out, true, e.out.size));
  CHECK(check_mat(e.y, false, 4));
  CHECK(check_mat(e.res, false, e.res.size));
  if (e.y.p) CHECK(apart_or_same(e.out, e.y));
  if (e.res.p) CHECK(apart_or_same(e.out, e.res));
  return MOE_OK;
}

[[maybe_unused]] size_t up256(size_t n) { return (n + 255) & ~size_t(255); }

}  // namespace
}  // namespace moe
