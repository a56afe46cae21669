// Host side of the calls that train around a block's linears (dropout, layer norm,
// the vocabulary's cross entropy): argument checks and launches. The arithmetic
// runs in the kernels declared in poetx_internal.h.
#include <hip/hip_runtime.h>

#include <cmath>

#include "../../include/poetx.h"
#include "args_check.h"
#include "poetx_internal.h"

namespace {

using namespace poetx::args;

// The kernels' form of a rule; false for a bad one.
bool drop_rule(const poetx_dropout_rule& r, poetx::DropArgs& d) {
  if (!(r.p >= 0.0 && r.p <= 1.0)) return false;
  const long threshold = std::lrint(r.p * 65536.0);
  d.seed = r.seed;
  d.seed_dev = r.seed_dev;
  d.site = r.site;
  d.threshold = (uint32_t)threshold;
  d.scale = threshold < 65536 ? (float)(65536.0 / (double)(65536 - threshold)) : 0.0f;
  return true;
}

poetx_status vocab_desc(const poetx_cross_entropy_desc* d) {
  if (!d || d->T < 0) return POETX_ERR_INVALID_ARG;
  if (d->V < 1 || d->V > poetx::kVocabMax || d->n < 1 || d->n > poetx::kVocabMaxDim || d->T > poetx::kVocabMax)
    return POETX_ERR_SHAPE;
  if (d->T * d->n > poetx::kVocabMaxElems || (int64_t)d->V * d->n > poetx::kVocabMaxElems) return POETX_ERR_SHAPE;
  if (!real_type(d->dtype)) return POETX_ERR_DTYPE;
  return POETX_OK;
}
Mat bytes_at(const void* p, size_t n) { return Mat{p, 1, (int64_t)n, (int64_t)n, 1}; }

Mat seed_of(const poetx_dropout_rule& r) { return Mat{r.seed_dev, 1, 8, 8, 1}; }

}  // namespace

extern "C" {

poetx_status poetx_dropout(const poetx_dropout_desc* d, const void* X, const void* R, void* Y, void* stream) {
  if (!d || d->T < 0) return POETX_ERR_INVALID_ARG;
  if (d->dim < 1 || d->dim > poetx::kNormMaxDim || d->T > kMaxRows) return POETX_ERR_SHAPE;
  if (!real_type(d->dtype)) return POETX_ERR_DTYPE;
  poetx::DropArgs rule{};
  if (!drop_rule(d->drop, rule)) return POETX_ERR_INVALID_ARG;
  if (d->T == 0) return POETX_OK;
  if (!X || !Y) return POETX_ERR_INVALID_ARG;
  const int es = size_of(d->dtype);
  Mat x{X, d->T, d->dim, d->ld_x, es}, r{R, d->T, d->dim, d->ld_r, es}, y{Y, d->T, d->dim, d->ld_y, es};
  if (!strides_ok(x) || !strides_ok(r) || !strides_ok(y)) return POETX_ERR_SHAPE;
  if (!aligned(X, es) || !aligned(R, es) || !aligned(Y, es) || !aligned(d->drop.seed_dev, 8)) return POETX_ERR_ALIGNMENT;
  if ((overlap(y, x) && !same(y, x)) || (overlap(y, r) && !same(y, r)) || overlap(y, seed_of(d->drop)))
    return POETX_ERR_INVALID_ARG;
  poetx::DropoutArgs a{X, R, Y, d->T, d->dim, x.ld, r.ld, y.ld, rule, 0};
  return launched(poetx::launch_dropout(a, d->dtype == POETX_BF16, (hipStream_t)stream));
}

poetx_status poetx_add_layer_norm(const poetx_layer_norm_desc* d, const void* X, const void* R, const float* w,
                                  const float* b, void* H, void* Y, float* scale, float* mean, float* rstd,
                                  void* stream) {
  if (!d || d->T < 0) return POETX_ERR_INVALID_ARG;
  if (d->dim < 1 || d->dim > poetx::kNormMaxDim || d->T > kMaxRows) return POETX_ERR_SHAPE;
  if (!real_type(d->dtype) || (d->y_dtype != d->dtype && d->y_dtype != POETX_INT8)) return POETX_ERR_DTYPE;
  poetx::DropArgs rule{};
  if (!(d->eps >= 0.0) || !std::isfinite(d->eps) || !drop_rule(d->drop, rule)) return POETX_ERR_INVALID_ARG;
  if (d->T == 0) return POETX_OK;
  const bool quant = d->y_dtype == POETX_INT8;
  if (!X || !w || !Y || quant != (scale != nullptr)) return POETX_ERR_INVALID_ARG;
  const int es = size_of(d->dtype), ys = size_of(d->y_dtype);
  Mat x{X, d->T, d->dim, d->ld_x, es}, r{R, d->T, d->dim, d->ld_r, es}, h{H, d->T, d->dim, d->ld_h, es},
      y{Y, d->T, d->dim, d->ld_y, ys};
  if (!strides_ok(x) || !strides_ok(r) || !strides_ok(h) || !strides_ok(y)) return POETX_ERR_SHAPE;
  if (!aligned(X, es) || !aligned(R, es) || !aligned(H, es) || !aligned(Y, ys) || !aligned(w, 4) || !aligned(b, 4) ||
      !aligned(scale, 4) || !aligned(mean, 4) || !aligned(rstd, 4) || !aligned(d->drop.seed_dev, 8))
    return POETX_ERR_ALIGNMENT;
  const Mat in[] = {x, r, vec(w, d->dim), vec(b, d->dim), seed_of(d->drop)};
  const Mat out[] = {h, y, vec(scale, d->T), vec(mean, d->T), vec(rstd, d->T)};
  for (int i = 0; i < 5; ++i) {
    for (const Mat& m : in)
      if (overlap(out[i], m) && !(i == 0 && (&m == &in[0] || &m == &in[1]) && same(h, m))) return POETX_ERR_INVALID_ARG;
    for (int j = 0; j < i; ++j)
      if (overlap(out[i], out[j])) return POETX_ERR_INVALID_ARG;
  }
  poetx::LayerNormArgs a{X, R, w, b, H, Y, scale, mean, rstd, d->T, d->dim, quant ? 1 : 0,
                         x.ld, r.ld, h.ld, y.ld, d->eps, rule, 0};
  return launched(poetx::launch_add_layer_norm(a, d->dtype == POETX_BF16, (hipStream_t)stream));
}

size_t poetx_layer_norm_backward_workspace(int64_t T, int32_t dim) {
  if (T < 0 || T > kMaxRows || dim < 1 || dim > poetx::kNormMaxDim) return 0;
  // partial sums of g_w and g_b, then three values per row for rows that no workgroup holds
  const size_t rows = dim > poetx::layer_norm_back_reg_dim(0) ? (size_t)T * 12 : 0;
  return ((size_t)poetx::layer_norm_backward_parts(T) * dim * 8 + rows + 255) / 256 * 256 + 256;
}

poetx_status poetx_layer_norm_backward(const poetx_layer_norm_backward_desc* d, const void* G, const void* G_H,
                                       const void* H, const float* w, const float* mean, const float* rstd, void* G_X,
                                       void* G_R, float* g_w, float* g_b, void* ws, size_t ws_bytes, void* stream) {
  if (!d || d->T < 0) return POETX_ERR_INVALID_ARG;
  if (d->dim < 1 || d->dim > poetx::kNormMaxDim || d->T > kMaxRows) return POETX_ERR_SHAPE;
  if (!real_type(d->dtype)) return POETX_ERR_DTYPE;
  poetx::DropArgs rule{};
  if (!g_w || !g_b || !drop_rule(d->drop, rule)) return POETX_ERR_INVALID_ARG;
  // without dropout the residual's gradient is that of x
  if (G_R && rule.threshold == 0) return POETX_ERR_INVALID_ARG;
  if (!aligned(g_w, 4) || !aligned(g_b, 4)) return POETX_ERR_ALIGNMENT;
  if (overlap(vec(g_w, d->dim), vec(g_b, d->dim))) return POETX_ERR_INVALID_ARG;
  const hipStream_t s = (hipStream_t)stream;
  if (d->T == 0) {
    const poetx_status st = launched(poetx::launch_zero(g_w, d->dim, s));
    return st == POETX_OK ? launched(poetx::launch_zero(g_b, d->dim, s)) : st;
  }
  if (!G || !H || !w || !mean || !rstd || !G_X) return POETX_ERR_INVALID_ARG;
  const int es = size_of(d->dtype);
  Mat g{G, d->T, d->dim, d->ld_g, es}, gh{G_H, d->T, d->dim, d->ld_gh, es}, h{H, d->T, d->dim, d->ld_h, es},
      gx{G_X, d->T, d->dim, d->ld_gx, es}, gr{G_R, d->T, d->dim, d->ld_gr, es};
  if (!strides_ok(g) || !strides_ok(gh) || !strides_ok(h) || !strides_ok(gx) || !strides_ok(gr)) return POETX_ERR_SHAPE;
  if (!aligned(G, es) || !aligned(G_H, es) || !aligned(H, es) || !aligned(G_X, es) || !aligned(G_R, es) ||
      !aligned(w, 4) || !aligned(mean, 4) || !aligned(rstd, 4) || !aligned(ws, 16) || !aligned(d->drop.seed_dev, 8))
    return POETX_ERR_ALIGNMENT;
  const size_t need = poetx_layer_norm_backward_workspace(d->T, d->dim);
  if (!ws || ws_bytes < need) return POETX_ERR_WORKSPACE;
  const Mat in[] = {g, gh, h, vec(w, d->dim), vec(mean, d->T), vec(rstd, d->T), seed_of(d->drop)};
  const Mat out[] = {gx, gr, vec(g_w, d->dim), vec(g_b, d->dim), Mat{ws, 1, (int64_t)need, (int64_t)need, 1}};
  for (int i = 0; i < 5; ++i) {
    for (const Mat& m : in)
      if (overlap(out[i], m) && !(i <= 1 && (&m == &in[0] || &m == &in[1]) && same(out[i], m)))
        return POETX_ERR_INVALID_ARG;
    for (int j = 0; j < i; ++j)
      if (overlap(out[i], out[j])) return POETX_ERR_INVALID_ARG;
  }
  float* part = static_cast<float*>(ws);
  poetx::LayerNormBackArgs a{G, G_H, H, w, mean, rstd, G_X, G_R, g_w, g_b, part,
                             part + (size_t)poetx::layer_norm_backward_parts(d->T) * d->dim * 2, d->T, d->dim,
                             g.ld, gh.ld, h.ld, gx.ld, gr.ld, rule};
  return launched(poetx::launch_layer_norm_backward(a, d->dtype == POETX_BF16, s));
}

size_t poetx_linear_cross_entropy_workspace(const poetx_cross_entropy_desc* d) {
  if (vocab_desc(d) != POETX_OK || d->T == 0) return 0;
  return poetx::vocab_forward_plan(d->T, d->V, d->n, d->dtype == POETX_BF16).bytes;
}

poetx_status poetx_linear_cross_entropy(const poetx_cross_entropy_desc* d, const void* X, const void* W,
                                        const int64_t* target, float* loss, float* lse, void* ws, size_t ws_bytes,
                                        void* stream) {
  const poetx_status ok = vocab_desc(d);
  if (ok != POETX_OK || d->T == 0) return ok;
  if (!X || !W || !target || !loss || !lse) return POETX_ERR_INVALID_ARG;
  const int es = size_of(d->dtype);
  Mat x{X, d->T, d->n, d->ld_x, es}, w{W, d->V, d->n, d->ld_w, es};
  if (!strides_ok(x) || !strides_ok(w)) return POETX_ERR_SHAPE;
  if (!aligned(X, es) || !aligned(W, es) || !aligned(target, 8) || !aligned(loss, 4) || !aligned(lse, 4) ||
      !aligned(ws, 16))
    return POETX_ERR_ALIGNMENT;
  const size_t need = poetx_linear_cross_entropy_workspace(d);
  if (!ws || ws_bytes < need) return POETX_ERR_WORKSPACE;
  const Mat in[] = {x, w, bytes_at(target, (size_t)d->T * 8)};
  const Mat out[] = {vec(loss, d->T), vec(lse, d->T), bytes_at(ws, need)};
  for (int i = 0; i < 3; ++i) {
    for (const Mat& m : in)
      if (overlap(out[i], m)) return POETX_ERR_INVALID_ARG;
    for (int j = 0; j < i; ++j)
      if (overlap(out[i], out[j])) return POETX_ERR_INVALID_ARG;
  }
  poetx::VocabArgs a{};
  a.X = X;
  a.W = W;
  a.target = target;
  a.T = d->T;
  a.V = d->V;
  a.n = d->n;
  a.ldx = x.ld;
  a.ldw = w.ld;
  a.ignore = d->ignore_index;
  a.loss = loss;
  a.lse_out = lse;
  return launched(poetx::launch_vocab_forward(a, d->dtype == POETX_BF16, ws, (hipStream_t)stream));
}

size_t poetx_linear_cross_entropy_backward_workspace(const poetx_cross_entropy_desc* d, int32_t need_x, int32_t need_w) {
  if (vocab_desc(d) != POETX_OK || d->T == 0) return 0;
  return poetx::vocab_backward_plan(d->T, d->V, d->n, d->dtype == POETX_BF16, need_x != 0, need_w != 0).bytes;
}

poetx_status poetx_linear_cross_entropy_backward(const poetx_cross_entropy_desc* d, const float* g, const void* X,
                                                 const void* W, const int64_t* target, const float* lse, void* G_X,
                                                 void* G_W, void* ws, size_t ws_bytes, void* stream) {
  const poetx_status ok = vocab_desc(d);
  if (ok != POETX_OK) return ok;
  if (!G_X && !G_W) return POETX_ERR_INVALID_ARG;
  if (d->g_count != 1 && d->g_count != d->T) return POETX_ERR_SHAPE;
  const int es = size_of(d->dtype);
  Mat x{X, d->T, d->n, d->ld_x, es}, w{W, d->V, d->n, d->ld_w, es}, gx{G_X, d->T, d->n, d->ld_gx, es},
      gw{G_W, d->V, d->n, d->ld_gw, es};
  if (!strides_ok(x) || !strides_ok(w) || !strides_ok(gx) || !strides_ok(gw)) return POETX_ERR_SHAPE;
  if (!aligned(X, es) || !aligned(W, es) || !aligned(G_X, es) || !aligned(G_W, es) || !aligned(target, 8) ||
      !aligned(g, 4) || !aligned(lse, 4) || !aligned(ws, 16))
    return POETX_ERR_ALIGNMENT;
  const hipStream_t s = (hipStream_t)stream;
  if (d->T == 0) return G_W ? launched(poetx::launch_vocab_zero(G_W, d->V, d->n, gw.ld, es, s)) : POETX_OK;
  if (!g || !X || !W || !target || !lse) return POETX_ERR_INVALID_ARG;
  const size_t need = poetx_linear_cross_entropy_backward_workspace(d, G_X != nullptr, G_W != nullptr);
  if (!ws || ws_bytes < need) return POETX_ERR_WORKSPACE;
  const Mat in[] = {x, w, bytes_at(target, (size_t)d->T * 8), vec(lse, d->T), vec(g, d->g_count)};
  const Mat out[] = {gx, gw, bytes_at(ws, need)};
  for (int i = 0; i < 3; ++i) {
    for (const Mat& m : in)
      if (overlap(out[i], m)) return POETX_ERR_INVALID_ARG;
    for (int j = 0; j < i; ++j)
      if (overlap(out[i], out[j])) return POETX_ERR_INVALID_ARG;
  }
  poetx::VocabArgs a{};
  a.X = X;
  a.W = W;
  a.target = target;
  a.T = d->T;
  a.V = d->V;
  a.n = d->n;
  a.ldx = x.ld;
  a.ldw = w.ld;
  a.ignore = d->ignore_index;
  a.lse = lse;
  a.g = g;
  a.g_each = d->g_count != 1;
  a.GX = G_X;
  a.GW = G_W;
  a.ldgx = gx.ld;
  a.ldgw = gw.ld;
  return launched(poetx::launch_vocab_backward(a, d->dtype == POETX_BF16, ws, s));
}

}  // extern "C"
