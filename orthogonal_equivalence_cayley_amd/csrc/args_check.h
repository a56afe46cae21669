// Argument checks that the calls around a block's linears share.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "../../include/poetx.h"
#include "poetx_internal.h"

namespace poetx {
namespace args {

inline poetx_status launched(hipError_t e) {
  if (e == hipSuccess) return POETX_OK;
  poetx::set_last_hip(e);
  return POETX_ERR_HIP;
}

inline bool aligned(const void* p, size_t to) { return ((uintptr_t)p & (to - 1)) == 0; }

// A strided matrix of an argument list: its bytes from the first element to the last.
struct Mat {
  const void* p = nullptr;
  int64_t rows = 0, cols = 0, ld = 0;
  int es = 1;
  uintptr_t begin() const { return (uintptr_t)p; }
  uintptr_t end() const { return (uintptr_t)p + (uintptr_t)(((rows - 1) * ld + cols) * es); }
};

// Row strides as documented, and every byte offset within 62 bits.
inline bool strides_ok(Mat& m) {
  if (!m.p) return true;
  if (m.rows <= 1) m.ld = m.cols;
  if (m.ld < m.cols) return false;
  int64_t n;
  return !__builtin_mul_overflow(m.rows, m.ld, &n) && n < (int64_t(1) << 58);
}

// Whether two matrices share a byte. Exact for equal strides (columns of one
// buffer may lie side by side); for others by their first and last bytes.
inline bool overlap(const Mat& a, const Mat& b) {
  if (!a.p || !b.p || a.rows <= 0 || b.rows <= 0) return false;
  if (a.end() <= b.begin() || b.end() <= a.begin()) return false;
  const uintptr_t la = (uintptr_t)a.ld * a.es, lb = (uintptr_t)b.ld * b.es;
  if (la != lb || a.rows <= 1 || b.rows <= 1) return true;
  const uintptr_t wa = (uintptr_t)a.cols * a.es, wb = (uintptr_t)b.cols * b.es;
  const uintptr_t d = b.begin() >= a.begin() ? (b.begin() - a.begin()) % la : (la - (a.begin() - b.begin()) % la) % la;
  return !(d >= wa && d + wb <= la);
}
// the same elements, one by one
inline bool same(const Mat& a, const Mat& b) {
  return a.p == b.p && a.ld == b.ld && a.es == b.es && a.rows == b.rows && a.cols == b.cols;
}
inline Mat vec(const void* p, int64_t n) { return Mat{p, 1, n, n, 4}; }

inline int size_of(int dtype) { return dtype == POETX_FP32 ? 4 : dtype == POETX_BF16 ? 2 : 1; }
inline bool real_type(int dtype) { return dtype == POETX_FP32 || dtype == POETX_BF16; }

constexpr int64_t kMaxRows = 0x7fffffff;

}  // namespace args
}  // namespace poetx
