// Host side of the calls around a block's linears (norm, merged-weight product,
// gradient clipping): argument checks and launches. The arithmetic runs in the
// kernels declared in poetx_internal.h.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <memory>
#include <new>

#include "../../include/poetx.h"
#include "poetx_internal.h"

namespace {

poetx_status launched(hipError_t e) {
  if (e == hipSuccess) return POETX_OK;
  poetx::set_last_hip(e);
  return POETX_ERR_HIP;
}

bool aligned(const void* p, size_t to) { return ((uintptr_t)p & (to - 1)) == 0; }

// A strided matrix of an argument list: its bytes from the first element to the last.
struct Mat {
  const void* p = nullptr;
  int64_t rows = 0, cols = 0, ld = 0;
  int es = 1;
  uintptr_t begin() const { return (uintptr_t)p; }
  uintptr_t end() const { return (uintptr_t)p + (uintptr_t)(((rows - 1) * ld + cols) * es); }
};

// Row strides as documented, and every byte offset within 62 bits.
bool strides_ok(Mat& m) {
  if (!m.p) return true;
  if (m.rows <= 1) m.ld = m.cols;
  if (m.ld < m.cols) return false;
  int64_t n;
  return !__builtin_mul_overflow(m.rows, m.ld, &n) && n < (int64_t(1) << 58);
}

// Whether two matrices share a byte. Exact for equal strides (columns of one
// buffer may lie side by side); for others by their first and last bytes.
bool overlap(const Mat& a, const Mat& b) {
  if (!a.p || !b.p || a.rows <= 0 || b.rows <= 0) return false;
  if (a.end() <= b.begin() || b.end() <= a.begin()) return false;
  const uintptr_t la = (uintptr_t)a.ld * a.es, lb = (uintptr_t)b.ld * b.es;
  if (la != lb || a.rows <= 1 || b.rows <= 1) return true;
  const uintptr_t wa = (uintptr_t)a.cols * a.es, wb = (uintptr_t)b.cols * b.es;
  const uintptr_t d = b.begin() >= a.begin() ? (b.begin() - a.begin()) % la : (la - (a.begin() - b.begin()) % la) % la;
  return !(d >= wa && d + wb <= la);
}
// the same elements, one by one
bool same(const Mat& a, const Mat& b) {
  return a.p == b.p && a.ld == b.ld && a.es == b.es && a.rows == b.rows && a.cols == b.cols;
}
Mat vec(const void* p, int64_t n) { return Mat{p, 1, n, n, 4}; }

int size_of(int dtype) { return dtype == POETX_FP32 ? 4 : dtype == POETX_BF16 ? 2 : 1; }
bool real_type(int dtype) { return dtype == POETX_FP32 || dtype == POETX_BF16; }

constexpr int64_t kMaxRows = 0x7fffffff;

int linear_type(const poetx_linear_desc* d) {
  return d->dtype == POETX_INT8 ? poetx::LINEAR_I8 : d->dtype == POETX_BF16 ? poetx::LINEAR_BF16
                                                                             : poetx::LINEAR_F32;
}
poetx_status linear_desc(const poetx_linear_desc* d) {
  if (!d || d->T < 0) return POETX_ERR_INVALID_ARG;
  if (d->m < 1 || d->m > poetx::kLinearMaxRows || d->n < 1 || d->T > kMaxRows) return POETX_ERR_SHAPE;
  const bool q = d->dtype == POETX_INT8;
  if (!q && !real_type(d->dtype)) return POETX_ERR_DTYPE;
  if (d->y_dtype != POETX_FP32 && !(d->y_dtype == POETX_BF16 && d->dtype != POETX_FP32)) return POETX_ERR_DTYPE;
  if (d->act < POETX_ACT_NONE || d->act > POETX_ACT_GELU_TANH) return POETX_ERR_INVALID_ARG;
  // 128 * 128 * n stays within 32-bit integers
  if (q && d->n > 131071) return POETX_ERR_UNSUPPORTED;
  return POETX_OK;
}
constexpr int32_t kMaxTensors = 1 << 20;
constexpr int64_t kMaxElems = int64_t(1) << 37;   // of one gradient tensor: a launch counts chunks in 31 bits

}  // namespace

extern "C" {

poetx_status poetx_add_rms_norm(const poetx_norm_desc* d, const void* X, const void* R, const float* w,
                                void* H, void* Y, float* scale, float* rstd, void* stream) {
  if (!d || d->T < 0) return POETX_ERR_INVALID_ARG;
  if (d->dim < 1 || d->dim > poetx::kNormMaxDim || d->T > kMaxRows) return POETX_ERR_SHAPE;
  if (!real_type(d->dtype) || (d->y_dtype != d->dtype && d->y_dtype != POETX_INT8)) return POETX_ERR_DTYPE;
  if (!(d->eps >= 0.0) || !std::isfinite(d->eps)) return POETX_ERR_INVALID_ARG;
  if (d->T == 0) return POETX_OK;
  const bool quant = d->y_dtype == POETX_INT8;
  if (!X || !w || !Y || quant != (scale != nullptr)) return POETX_ERR_INVALID_ARG;
  const int es = size_of(d->dtype), ys = size_of(d->y_dtype);
  Mat x{X, d->T, d->dim, d->ld_x, es}, r{R, d->T, d->dim, d->ld_r, es}, h{H, d->T, d->dim, d->ld_h, es},
      y{Y, d->T, d->dim, d->ld_y, ys};
  if (!strides_ok(x) || !strides_ok(r) || !strides_ok(h) || !strides_ok(y)) return POETX_ERR_SHAPE;
  if (!aligned(X, es) || !aligned(R, es) || !aligned(H, es) || !aligned(Y, ys) || !aligned(w, 4) ||
      !aligned(scale, 4) || !aligned(rstd, 4))
    return POETX_ERR_ALIGNMENT;
  const Mat in[] = {x, r, vec(w, d->dim)};
  const Mat out[] = {h, y, vec(scale, d->T), vec(rstd, d->T)};
  for (int i = 0; i < 4; ++i) {
    for (const Mat& m : in)
      if (overlap(out[i], m) && !(i == 0 && &m != &in[2] && same(h, m))) return POETX_ERR_INVALID_ARG;
    for (int j = 0; j < i; ++j)
      if (overlap(out[i], out[j])) return POETX_ERR_INVALID_ARG;
  }
  poetx::NormArgs a{X, R, w, H, Y, scale, rstd, d->T, d->dim, quant ? 1 : 0, x.ld, r.ld, h.ld, y.ld, d->eps};
  return launched(poetx::launch_add_rms_norm(a, d->dtype == POETX_BF16, (hipStream_t)stream));
}

size_t poetx_rms_norm_backward_workspace(int64_t T, int32_t dim) {
  if (T < 0 || T > kMaxRows || dim < 1 || dim > poetx::kNormMaxDim) return 0;
  // partial sums of g_w, then one value per row for rows that no wave holds
  const size_t rows = dim > poetx::kNormRegDim ? (size_t)T * 4 : 0;
  return ((size_t)poetx::norm_backward_parts(T) * dim * 4 + rows + 255) / 256 * 256 + 256;
}

poetx_status poetx_rms_norm_backward(const poetx_norm_backward_desc* d, const void* G, const void* G_H,
                                     const void* H, const float* w, const float* rstd, void* G_X,
                                     float* g_w, void* ws, size_t ws_bytes, void* stream) {
  if (!d || d->T < 0) return POETX_ERR_INVALID_ARG;
  if (d->dim < 1 || d->dim > poetx::kNormMaxDim || d->T > kMaxRows) return POETX_ERR_SHAPE;
  if (!real_type(d->dtype)) return POETX_ERR_DTYPE;
  if (!g_w) return POETX_ERR_INVALID_ARG;
  if (!aligned(g_w, 4)) return POETX_ERR_ALIGNMENT;
  const hipStream_t s = (hipStream_t)stream;
  if (d->T == 0) return launched(poetx::launch_zero(g_w, d->dim, s));
  if (!G || !H || !w || !rstd || !G_X) return POETX_ERR_INVALID_ARG;
  const int es = size_of(d->dtype);
  Mat g{G, d->T, d->dim, d->ld_g, es}, gh{G_H, d->T, d->dim, d->ld_gh, es}, h{H, d->T, d->dim, d->ld_h, es},
      gx{G_X, d->T, d->dim, d->ld_gx, es};
  if (!strides_ok(g) || !strides_ok(gh) || !strides_ok(h) || !strides_ok(gx)) return POETX_ERR_SHAPE;
  if (!aligned(G, es) || !aligned(G_H, es) || !aligned(H, es) || !aligned(G_X, es) || !aligned(w, 4) ||
      !aligned(rstd, 4) || !aligned(ws, 16))
    return POETX_ERR_ALIGNMENT;
  const size_t need = poetx_rms_norm_backward_workspace(d->T, d->dim);
  if (!ws || ws_bytes < need) return POETX_ERR_WORKSPACE;
  const Mat in[] = {g, gh, h, vec(w, d->dim), vec(rstd, d->T)};
  const Mat out[] = {gx, vec(g_w, d->dim), Mat{ws, 1, (int64_t)need, (int64_t)need, 1}};
  for (int i = 0; i < 3; ++i) {
    for (const Mat& m : in)
      if (overlap(out[i], m) && !(i == 0 && (&m == &in[0] || &m == &in[1]) && same(gx, m)))
        return POETX_ERR_INVALID_ARG;
    for (int j = 0; j < i; ++j)
      if (overlap(out[i], out[j])) return POETX_ERR_INVALID_ARG;
  }
  float* part = static_cast<float*>(ws);
  poetx::NormBackArgs a{G, G_H, H, w, rstd, G_X, g_w, part,
                        part + (size_t)poetx::norm_backward_parts(d->T) * d->dim, d->T, d->dim,
                        g.ld, gh.ld, h.ld, gx.ld};
  return launched(poetx::launch_rms_norm_backward(a, d->dtype == POETX_BF16, s));
}

size_t poetx_linear_workspace(const poetx_linear_desc* d) {
  if (linear_desc(d) != POETX_OK || d->T == 0) return 0;
  poetx::LinearArgs a{};   // the split goes by the sizes alone
  a.T = d->T;
  a.m = d->m;
  a.n = d->n;
  const int splits = poetx::linear_splits(a, linear_type(d));
  return splits > 1 ? (size_t)splits * d->T * ((d->m + 3) / 4 * 4) * 4 : 0;
}

poetx_status poetx_linear(const poetx_linear_desc* d, const void* X, const void* W, const float* sx,
                          const float* sw, const float* bias, const void* mul, const void* res, void* Y,
                          void* ws, size_t ws_bytes, void* stream) {
  const poetx_status ok = linear_desc(d);
  if (ok != POETX_OK) return ok;
  const bool q = d->dtype == POETX_INT8;
  if (d->T == 0) return POETX_OK;
  if (!X || !W || !Y || q != (sx != nullptr) || q != (sw != nullptr)) return POETX_ERR_INVALID_ARG;
  const int es = size_of(d->dtype), ys = size_of(d->y_dtype);
  Mat x{X, d->T, d->n, d->ld_x, es}, w{W, d->m, d->n, d->ld_w, es}, y{Y, d->T, d->m, d->ld_y, ys},
      mu{mul, d->T, d->m, d->ld_mul, ys}, re{res, d->T, d->m, d->ld_res, ys};
  if (!strides_ok(x) || !strides_ok(w) || !strides_ok(y) || !strides_ok(mu) || !strides_ok(re))
    return POETX_ERR_SHAPE;
  if (!aligned(X, es) || !aligned(W, es) || !aligned(Y, ys) || !aligned(mul, ys) || !aligned(res, ys) ||
      !aligned(sx, 4) || !aligned(sw, 4) || !aligned(bias, 4))
    return POETX_ERR_ALIGNMENT;
  for (const Mat& m : {x, w, vec(sx, d->T), vec(sw, d->m), vec(bias, d->m)})
    if (overlap(y, m)) return POETX_ERR_INVALID_ARG;
  if ((overlap(y, mu) && !same(y, mu)) || (overlap(y, re) && !same(y, re))) return POETX_ERR_INVALID_ARG;
  poetx::LinearArgs a{X, W, sx, sw, bias, mul, res, Y, d->T, d->m, d->n,
                      x.ld, w.ld, y.ld, mu.ld, re.ld, d->act, d->y_dtype == POETX_BF16 ? 1 : 0};
  const int type = linear_type(d);
  const size_t need = poetx_linear_workspace(d);
  if (need) {
    if (!aligned(ws, 16)) return POETX_ERR_ALIGNMENT;
    if (!ws || ws_bytes < need) return POETX_ERR_WORKSPACE;
    const Mat part{ws, 1, (int64_t)need, (int64_t)need, 1};
    for (const Mat& m : {x, w, y, mu, re, vec(sx, d->T), vec(sw, d->m), vec(bias, d->m)})
      if (overlap(part, m)) return POETX_ERR_INVALID_ARG;
    a.part = ws;
    a.splits = poetx::linear_splits(a, type);
  }
  return launched(poetx::launch_linear(a, type, (hipStream_t)stream));
}

size_t poetx_clip_grads_workspace(int32_t count) {
  if (count < 0 || count > kMaxTensors) return 0;
  return (size_t)poetx::clip_parts(count) * sizeof(double) + 256;
}

poetx_status poetx_clip_grads(int32_t count, const void* const* grads, const int64_t* ns,
                              const int32_t* dtypes, void* const* outs, double max_norm, float* norm_out,
                              void* ws, size_t ws_bytes, void* stream) {
  if (count < 0 || !std::isfinite(max_norm) || max_norm < 0.0) return POETX_ERR_INVALID_ARG;
  if (count > kMaxTensors) return POETX_ERR_SHAPE;
  if (count > 0 && (!grads || !ns || !dtypes)) return POETX_ERR_INVALID_ARG;
  if (!aligned(ws, 16) || !aligned(norm_out, 4)) return POETX_ERR_ALIGNMENT;
  if (!ws || ws_bytes < poetx_clip_grads_workspace(count)) return POETX_ERR_WORKSPACE;
  struct Span {
    uintptr_t b, e;
    bool write;
  };
  std::unique_ptr<poetx::ClipItem[]> items(new (std::nothrow) poetx::ClipItem[(size_t)count + 1]);
  std::unique_ptr<Span[]> spans(new (std::nothrow) Span[2 * (size_t)count + 2]);
  if (!items || !spans) return POETX_ERR_UNSUPPORTED;   // no host memory
  size_t k = 0;
  for (int i = 0; i < count; ++i) {
    if (!real_type(dtypes[i])) return POETX_ERR_DTYPE;
    if (ns[i] < 0) return POETX_ERR_INVALID_ARG;
    if (ns[i] > kMaxElems) return POETX_ERR_SHAPE;
    const int es = size_of(dtypes[i]);
    void* out = outs ? outs[i] : nullptr;
    if (ns[i] > 0) {
      if (!grads[i] || (outs && !out)) return POETX_ERR_INVALID_ARG;
      if (!aligned(grads[i], es) || !aligned(out, es)) return POETX_ERR_ALIGNMENT;
      const uintptr_t len = (uintptr_t)ns[i] * es;
      spans[k++] = Span{(uintptr_t)grads[i], (uintptr_t)grads[i] + len, out == grads[i]};
      if (out && out != grads[i]) spans[k++] = Span{(uintptr_t)out, (uintptr_t)out + len, true};
    }
    items[i] = poetx::ClipItem{grads[i], out, ns[i], dtypes[i] == POETX_BF16 ? 1 : 0};
  }
  if (norm_out) spans[k++] = Span{(uintptr_t)norm_out, (uintptr_t)norm_out + 4, true};
  spans[k++] = Span{(uintptr_t)ws, (uintptr_t)ws + poetx_clip_grads_workspace(count), true};
  const auto before = [](const Span& a, const Span& b) { return a.b < b.b; };
  if (!std::is_sorted(spans.get(), spans.get() + k, before)) std::sort(spans.get(), spans.get() + k, before);
  uintptr_t any = 0, written = 0;   // ends of what lies before
  for (size_t i = 0; i < k; ++i) {
    if (spans[i].b < (spans[i].write ? any : written)) return POETX_ERR_INVALID_ARG;
    any = std::max(any, spans[i].e);
    if (spans[i].write) written = std::max(written, spans[i].e);
  }
  return launched(poetx::launch_clip(items.get(), count, max_norm, static_cast<double*>(ws), norm_out,
                                     outs != nullptr, (hipStream_t)stream));
}

}  // extern "C"
