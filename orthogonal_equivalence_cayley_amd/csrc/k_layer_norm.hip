// Dropout, the residual's addition and layer norm in one pass, forward and backward,
// with the output in the activations' type or as INT8 rows with one scale each (the
// rule of the INT8 weight rows, k_quant.hip).
//
//   h = rnd(drop(x) + r),  m = mean h,  s = (mean (h - m)^2 + eps)^(-1/2),
//   y = (h - m) s w + b
//   u = (h - m) s,  dh = gh + s (g w - mean(g w) - u mean(g w u)),
//   dr = dh,  dx = drop(dh),  dw = sum_t g u,  db = sum_t g
//
// Bound by memory: 8 bytes a bf16 element forward (x, r, h, y), 8 backward (g, gh, h,
// dx) and 10 with dropout, whose dx is not dr. A row is read once and stays in
// registers; one wave, four or sixteen to a row, every load of a row and of the next one
// out before the first is used. 16384 x 2048 bf16, call after call: forward 45 us, with dropout
// 48 (5.9 and 5.5 TB/s; with the statistics kept and under the profiler 57 to 61), backward 51,
// with dropout 65 (5.2 and 5.1 TB/s; 73).
#include <algorithm>
#include <type_traits>

#include "dropout_common.h"
#include "poetx_internal.h"
#include "row_common.h"

namespace poetx {
namespace {

using namespace row;

constexpr int kThr = 256;
constexpr int threads(int wpr) { return wpr > 4 ? wpr * 64 : kThr; }

template <typename V>
struct Two {
  V a, b;
};
// the sums of both over the WPR waves of a row, as row_reduce
template <int WPR, typename V>
__device__ __forceinline__ Two<V> row_sums(Two<V> v, Two<V>* red) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) {
    v.a += __shfl_xor(v.a, o);
    v.b += __shfl_xor(v.b, o);
  }
  if constexpr (WPR > 1) {
    __syncthreads();   // the last use of `red` is over
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    v = red[0];
#pragma unroll
    for (int i = 1; i < WPR; ++i) {
      v.a += red[i].a;
      v.b += red[i].b;
    }
  }
  return v;
}

// Mean and variance come from one pass, sums of h - c and its square in 64 bits: their
// order then does not show in the fp32 results, so the INT8 decisions are the same for
// every split of a row over lanes. c is the row's own h_0, behind dropout and the residual:
// what the squares cancel by is then (h_0 - mean)^2 over the variance, the row's length at
// most, and a row far from zero keeps its variance. (A value that is not of the row would
// not do: at 1e7 deviations off it costs 1 % of the result, at 1e9 all of it.)
__device__ __forceinline__ double center(float h0) { return fabsf(h0) < __builtin_inff() ? (double)h0 : 0.0; }
// h_0 of row `row` from its parts, where several waves share the row (its only wave takes it
// from its first lane: 16384 x 300 bf16 with dropout 21.7 us, 23.0 from the parts). The row is
// the wave's, so the generator runs on the scalar unit.
template <typename E, bool DROP>
__device__ __forceinline__ float first_h(const DropArgs& d, drop::Key k, uint32_t row, E x0, bool res, E r0) {
  float h[1] = {to_f(x0)};
  if constexpr (DROP) {
    const drop::Bits b = drop::bits(k, 0, __builtin_amdgcn_readfirstlane(row), d.site);
    drop::apply(d, b.of(0) >= d.threshold ? 1u : 0u, h);
  }
  return to_f(from_f<E>(res ? h[0] + to_f(r0) : h[0]));
}
struct Stats {
  float m0, m1;   // the mean as two floats: a row far from zero keeps the digits of h - m
  float s;
};
__device__ __forceinline__ Stats stats_of(Two<double> sums, double c, const LayerNormArgs& a) {
  const double d = sums.a / (double)a.dim, m = c + d, var = sums.b / (double)a.dim - d * d;
  Stats r;
  r.m0 = (float)m;
  r.m1 = (float)(m - (double)r.m0);
  // rounding may leave a constant row's variance a little below zero; a NaN stays
  r.s = (float)(1.0 / sqrt((var < 0.0 ? 0.0 : var) + a.eps));
  return r;
}

// A workgroup takes rows a stride apart, w and b of its columns in registers (read for every
// row from the caches they are as many bytes as x and r: 16384 x 2048 bf16, one wave a row,
// 56 -> 45 us); the next row's loads are in flight while a row is worked on.
template <typename E, int NV, int WPR, bool WHOLE, bool DROP>
__global__ __launch_bounds__(threads(WPR)) void add_layer_norm_kernel(LayerNormArgs a) {
  constexpr int N = 16 / sizeof(E);
  constexpr int RPW = threads(WPR) / 64 / WPR;   // rows per workgroup
  constexpr int STEP = 64 * WPR * N;             // columns between a lane's vectors
  __shared__ Two<double> red[WPR];
  __shared__ uint32_t redu[WPR];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int c0 = ((wave % WPR) * 64 + lane) * N;
  const bool full = a.dim >= N;
  float w[NV][N], b[NV][N];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
#pragma unroll
    for (int e = 0; e < N; ++e) w[i][e] = b[i][e] = 0.0f;
    if (c0 + i * STEP < a.dim) {
      load_raw<WHOLE>(a.w + c0 + i * STEP, a.dim - c0 - i * STEP, full, w[i]);
      if (a.b) load_raw<WHOLE>(a.b + c0 + i * STEP, a.dim - c0 - i * STEP, full, b[i]);
    }
  }
  [[maybe_unused]] drop::Key key{};
  if constexpr (DROP) key = drop::key_of(a.drop);
  E xr[NV][N] = {}, rr[NV][N] = {};
  [[maybe_unused]] E x0 = E(0), r0 = E(0);   // the row's first, for every wave of it
  auto fetch = [&](long long t) {
    const E* x = static_cast<const E*>(a.X) + t * a.ldx;
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (c0 + i * STEP < a.dim) load_raw<WHOLE>(x + c0 + i * STEP, a.dim - c0 - i * STEP, full, xr[i]);
    if constexpr (WPR > 1) x0 = *x;
    if (a.R) {
      const E* r = static_cast<const E*>(a.R) + t * a.ldr;
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (c0 + i * STEP < a.dim) load_raw<WHOLE>(r + c0 + i * STEP, a.dim - c0 - i * STEP, full, rr[i]);
      if constexpr (WPR > 1) r0 = *r;
    }
  };
  const long long stride = (long long)gridDim.x * RPW;
  long long t = (long long)blockIdx.x * RPW + wave / WPR;
  if (t < a.T) fetch(t);
  for (; t < a.T; t += stride) {   // whole rows: with more waves to a row the workgroup has one
    float h[NV][N];
    Two<double> sum{0.0, 0.0};
    double c = 0.0;
    if constexpr (WPR > 1) c = center(first_h<E, DROP>(a.drop, key, a.row0 + (uint32_t)t, x0, a.R != nullptr, r0));
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int left = a.dim - c0 - i * STEP;
#pragma unroll
      for (int e = 0; e < N; ++e) h[i][e] = to_f(xr[i][e]);
      if constexpr (DROP) drop::apply(a.drop, key, a.row0 + (uint32_t)t, c0 + i * STEP, h[i]);
#pragma unroll
      for (int e = 0; e < N; ++e) {
        // rounded to the type before the norm: the kept h is what the norm sees
        if (a.R || DROP) h[i][e] = to_f(from_f<E>(a.R ? h[i][e] + to_f(rr[i][e]) : h[i][e]));
        if constexpr (WPR == 1) {
          if (i == 0 && e == 0) c = center(__uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(h[0][0]))));
        }
        const double d = (WHOLE ? left > 0 : e < left) ? (double)h[i][e] - c : 0.0;
        sum.a += d;
        sum.b += d * d;
      }
    }
    if (t + stride < a.T) fetch(t + stride);
    const Stats st = stats_of(row_sums<WPR>(sum, red), c, a);
    // behind the sums' barrier: H may lie over the first x or r, which every wave reads
    if (a.H) {
      E* ho = static_cast<E*>(a.H) + t * a.ldh + c0;
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (c0 + i * STEP < a.dim) store_n<WHOLE>(ho + i * STEP, a.dim - c0 - i * STEP, h[i]);
    }
    if (lane == 0 && wave % WPR == 0) {
      if (a.mean) a.mean[t] = st.m0;
      if (a.rstd) a.rstd[t] = st.s;
    }
    uint32_t amax = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int left = a.dim - c0 - i * STEP;
#pragma unroll
      for (int e = 0; e < N; ++e) {
        h[i][e] = (((h[i][e] - st.m0) - st.m1) * st.s) * w[i][e] + b[i][e];
        // behind the row's end stands -m s times 0
        if (WHOLE ? left > 0 : e < left) amax = max(amax, __float_as_uint(h[i][e]) & 0x7fffffffu);
      }
      if (!a.quant && left > 0) store_n<WHOLE>(static_cast<E*>(a.Y) + t * a.ldy + c0 + i * STEP, left, h[i]);
    }
    if (!a.quant) continue;
    amax = row_reduce<WPR>(amax, redu, Max{});
    float inv, scale;
    int8_rule(amax, inv, scale);
    if (lane == 0 && wave % WPR == 0) a.scale[t] = scale;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int left = a.dim - c0 - i * STEP;
      if (left <= 0) continue;
      int8_t q[N];
#pragma unroll
      for (int e = 0; e < N; ++e) q[e] = to_q(h[i][e], inv);
      store_raw<WHOLE>(static_cast<int8_t*>(a.Y) + t * a.ldy + c0 + i * STEP, left, q);
    }
  }
}

// Rows too long for registers: sixteen waves to a row, which is read again for each
// pass (from the caches mostly). Where H is written its values are what is read again,
// each by the thread that wrote it, so H may be X or R itself.
constexpr int kLongWaves = 16;
template <typename E, bool DROP>
__global__ __launch_bounds__(kLongWaves * 64) void add_layer_norm_long_kernel(LayerNormArgs a) {
  constexpr int N = 16 / sizeof(E), STEP = kLongWaves * 64 * N;
  __shared__ Two<double> red[kLongWaves];
  __shared__ uint32_t redu[kLongWaves];
  const long long t = blockIdx.x;
  const E* x = static_cast<const E*>(a.X) + t * a.ldx;
  const E* r = a.R ? static_cast<const E*>(a.R) + t * a.ldr : nullptr;
  E* ho = a.H ? static_cast<E*>(a.H) + t * a.ldh : nullptr;
  const int first = (int)threadIdx.x * N;
  [[maybe_unused]] drop::Key key{};
  if constexpr (DROP) key = drop::key_of(a.drop);
  // h from its parts
  auto make = [&](int c, float (&h)[N]) {
    E v[N], q[N];
    load_raw<false>(x + c, a.dim - c, true, v);
#pragma unroll
    for (int e = 0; e < N; ++e) h[e] = to_f(v[e]);
    if constexpr (DROP) drop::apply(a.drop, key, a.row0 + (uint32_t)t, c, h);
    if (r) {
      load_raw<false>(r + c, a.dim - c, true, q);
#pragma unroll
      for (int e = 0; e < N; ++e) h[e] += to_f(q[e]);
    }
#pragma unroll
    for (int e = 0; e < N; ++e) h[e] = to_f(from_f<E>(h[e]));
  };
  Two<double> sum{0.0, 0.0};
  const double mid = center(first_h<E, DROP>(a.drop, key, a.row0 + (uint32_t)t, x[0], r != nullptr, r ? r[0] : E(0)));
  __syncthreads();   // H may lie over the first x or r
  for (int c = first; c < a.dim; c += STEP) {
    float h[N];
    make(c, h);
    if (ho) store_n<false>(ho + c, a.dim - c, h);
#pragma unroll
    for (int e = 0; e < N; ++e) {
      const double d = e < a.dim - c ? (double)h[e] - mid : 0.0;
      sum.a += d;
      sum.b += d * d;
    }
  }
  // A thread reads back only what it wrote itself: a row's cut vector is not read from
  // the vector in front of it, which another thread may not have written yet.
  auto value = [&](int c, float (&h)[N]) {
    if (!ho) {
      make(c, h);
    } else if (a.dim - c >= N) {
      E v[N];
      load_raw<true>(static_cast<const E*>(ho) + c, N, true, v);
#pragma unroll
      for (int e = 0; e < N; ++e) h[e] = to_f(v[e]);
    } else {
#pragma unroll
      for (int e = 0; e < N; ++e) h[e] = e < a.dim - c ? to_f(ho[c + e]) : 0.0f;
    }
  };
  const Stats st = stats_of(row_sums<kLongWaves>(sum, red), mid, a);
  if (threadIdx.x == 0) {
    if (a.mean) a.mean[t] = st.m0;
    if (a.rstd) a.rstd[t] = st.s;
  }
  auto normed = [&](int c, float (&y)[N]) {
    float w[N], b[N] = {};
    value(c, y);
    load_raw<false>(a.w + c, a.dim - c, true, w);
    if (a.b) load_raw<false>(a.b + c, a.dim - c, true, b);
#pragma unroll
    for (int e = 0; e < N; ++e) y[e] = (((y[e] - st.m0) - st.m1) * st.s) * w[e] + b[e];
  };
  uint32_t amax = 0;
  for (int c = first; c < a.dim; c += STEP) {
    float y[N];
    normed(c, y);
#pragma unroll
    for (int e = 0; e < N; ++e)
      if (e < a.dim - c) amax = max(amax, __float_as_uint(y[e]) & 0x7fffffffu);
    if (!a.quant) store_n<false>(static_cast<E*>(a.Y) + t * a.ldy + c, a.dim - c, y);
  }
  if (!a.quant) return;
  amax = row_reduce<kLongWaves>(amax, redu, Max{});
  float inv, scale;
  int8_rule(amax, inv, scale);
  if (threadIdx.x == 0) a.scale[t] = scale;
  for (int c = first; c < a.dim; c += STEP) {
    float y[N];
    normed(c, y);
    int8_t q[N];
#pragma unroll
    for (int e = 0; e < N; ++e) q[e] = to_q(y[e], inv);
    store_raw<false>(static_cast<int8_t*>(a.Y) + t * a.ldy + c, a.dim - c, q);
  }
}

// Where the partial sums of a workgroup go: one row of 2 dim values each, or, for a
// single workgroup, the sums themselves
__device__ __forceinline__ void part_rows(const LayerNormBackArgs& a, int block, float*& pw, float*& pb) {
  pw = a.part ? a.part + (long long)block * 2 * a.dim : a.dw;
  pb = a.part ? pw + a.dim : a.db;
}

// The backward is handed the mean as one float. Its rounding puts u = (h - m) s off by up to
// 2^-24 |m| s in a whole row, which shows in rows far from zero; there, from 16 deviations on
// (2^-20 of u), h - m is exact and its own mean is what the rounding lost: taken once more, by
// the few rows that need it.
__device__ __forceinline__ bool far_mean(float m, float s) { return fabsf(m) * s > 16.0f; }

// Backward: each wave (WPR = 1) or workgroup (WPR = 4, 8) takes rows a stride apart and
// keeps its columns' parts of dw and db in registers, in 64 bits (sums over any number
// of rows: fp32 would lose small terms behind large ones); the parts of a workgroup's
// waves are joined in LDS. The next row's loads are in flight while a row is worked on.
template <typename E, int NV, int WPR, bool WHOLE, bool DROP>
__global__ __launch_bounds__(threads(WPR)) void layer_norm_backward_kernel(LayerNormBackArgs a) {
  constexpr int N = 16 / sizeof(E);
  constexpr int RPW = threads(WPR) / 64 / WPR;
  constexpr int STEP = 64 * WPR * N;
  __shared__ Two<float> red[WPR];
  __shared__ double redm[WPR];
  extern __shared__ double lds[];   // WPR = 1: 2 dim values
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int c0 = ((wave % WPR) * 64 + lane) * N;
  const bool full = a.dim >= N;
  [[maybe_unused]] drop::Key key{};
  if constexpr (DROP) key = drop::key_of(a.drop);
  double dw[NV][N] = {}, db[NV][N] = {};
  float w[NV][N] = {};
#pragma unroll
  for (int i = 0; i < NV; ++i)
    if (c0 + i * STEP < a.dim) load_raw<WHOLE>(a.w + c0 + i * STEP, a.dim - c0 - i * STEP, full, w[i]);
  E gr[NV][N] = {}, hr[NV][N] = {}, qr[NV][N] = {};
  float mn = 0.0f, sn = 0.0f;
  auto fetch = [&](long long t) {
    const E* g = static_cast<const E*>(a.G) + t * a.ldg + c0;
    const E* h = static_cast<const E*>(a.H) + t * a.ldh + c0;
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (c0 + i * STEP < a.dim) {
        load_raw<WHOLE>(g + i * STEP, a.dim - c0 - i * STEP, full, gr[i]);
        load_raw<WHOLE>(h + i * STEP, a.dim - c0 - i * STEP, full, hr[i]);
      }
    if (a.GH) {
      const E* q = static_cast<const E*>(a.GH) + t * a.ldgh + c0;
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (c0 + i * STEP < a.dim) load_raw<WHOLE>(q + i * STEP, a.dim - c0 - i * STEP, full, qr[i]);
    }
    mn = a.mean[t];
    sn = a.rstd[t];
  };
  const long long stride = (long long)gridDim.x * RPW;
  long long t = (long long)blockIdx.x * RPW + wave / WPR;
  if (t < a.T) fetch(t);
  for (; t < a.T; t += stride) {
    const float m = mn, s = sn;
    float gv[NV][N], u[NV][N], q[NV][N];
    Two<float> dot{0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      // behind the row's end g is zero and u a finite number or NaN: not summed
      const int left = a.dim - c0 - i * STEP;
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const bool in = WHOLE ? left > 0 : e < left;
        gv[i][e] = to_f(gr[i][e]) * w[i][e];
        u[i][e] = in ? (to_f(hr[i][e]) - m) * s : 0.0f;
        q[i][e] = to_f(qr[i][e]);
        dot.a += gv[i][e];
        dot.b += gv[i][e] * u[i][e];
      }
    }
    if (far_mean(m, s)) {   // the same for every wave of the row
      double rest = 0.0;
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < N; ++e) rest += c0 + i * STEP + e < a.dim ? (double)(to_f(hr[i][e]) - m) : 0.0;
      const float m1 = (float)(row_reduce<WPR>(rest, redm, Add{}) / (double)a.dim);
      dot.b = 0.0f;
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < N; ++e) {
          u[i][e] = c0 + i * STEP + e < a.dim ? ((to_f(hr[i][e]) - m) - m1) * s : 0.0f;
          dot.b += gv[i][e] * u[i][e];
        }
    }
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < N; ++e) {
        dw[i][e] += (double)(to_f(gr[i][e]) * u[i][e]);
        db[i][e] += (double)to_f(gr[i][e]);
      }
    if (t + stride < a.T) fetch(t + stride);
    // the generator runs while waves wait for each other (a wave of its own waits for none:
    // 8000 x 768 bf16 30 us with it here, 23 behind the sums)
    [[maybe_unused]] uint32_t keep[NV];
    if constexpr (DROP && WPR > 1) {
#pragma unroll
      for (int i = 0; i < NV; ++i) keep[i] = drop::kept<N>(a.drop, key, (uint32_t)t, c0 + i * STEP);
    }
    dot = row_sums<WPR>(dot, red);
    const float ca = dot.a / (float)a.dim, cb = dot.b / (float)a.dim;
    E* o = static_cast<E*>(a.GX) + t * a.ldgx + c0;
    E* ro = DROP && a.GR ? static_cast<E*>(a.GR) + t * a.ldgr + c0 : nullptr;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
#pragma unroll
      for (int e = 0; e < N; ++e) gv[i][e] = s * (gv[i][e] - ca - u[i][e] * cb) + q[i][e];
      if constexpr (DROP) {
        if (ro && c0 + i * STEP < a.dim) store_n<WHOLE>(ro + i * STEP, a.dim - c0 - i * STEP, gv[i]);
        if constexpr (WPR > 1) drop::apply(a.drop, keep[i], gv[i]);
        else drop::apply(a.drop, key, (uint32_t)t, c0 + i * STEP, gv[i]);
      }
      if (c0 + i * STEP < a.dim) store_n<WHOLE>(o + i * STEP, a.dim - c0 - i * STEP, gv[i]);
    }
  }
  float *pw, *pb;
  part_rows(a, blockIdx.x, pw, pb);
  if constexpr (WPR == 1) {
    double* const lw = lds;
    double* const lb = lds + a.dim;
    for (int k = 0; k < kThr / 64; ++k) {
      if (wave == k) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
          for (int e = 0; e < N; ++e) {
            const int c = c0 + i * STEP + e;
            if (c < a.dim) {
              lw[c] = k == 0 ? dw[i][e] : lw[c] + dw[i][e];
              lb[c] = k == 0 ? db[i][e] : lb[c] + db[i][e];
            }
          }
      }
      __syncthreads();
    }
    for (int c = threadIdx.x; c < a.dim; c += kThr) {
      pw[c] = (float)lw[c];
      pb[c] = (float)lb[c];
    }
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float o[N], p[N];
#pragma unroll
      for (int e = 0; e < N; ++e) {
        o[e] = (float)dw[i][e];
        p[e] = (float)db[i][e];
      }
      if (c0 + i * STEP < a.dim) {
        store_raw<WHOLE>(pw + c0 + i * STEP, a.dim - c0 - i * STEP, o);
        store_raw<WHOLE>(pb + c0 + i * STEP, a.dim - c0 - i * STEP, p);
      }
    }
  }
}

// Rows too long for registers: first both means of every row, then tiles of 256 vectors of
// columns by a range of rows. A row has up to 2^24 terms, 2^14 to a thread, and in one fp32
// number what their additions round alike would add up: a thread sums in fp32 within a vector
// and in 64 bits from there. The 1024 threads' sums are joined in fp32 (in 64 bits the kernel
// takes more registers than two workgroups on a CU have: 4096 x 8192 fp32 178 us, so 161).
template <typename E>
__global__ __launch_bounds__(kLongWaves * 64) void layer_norm_means_kernel(LayerNormBackArgs a) {
  constexpr int N = 16 / sizeof(E);
  __shared__ Two<float> red[kLongWaves];
  __shared__ double redm[kLongWaves];
  for (long long t = blockIdx.x; t < a.T; t += gridDim.x) {
    const E* g = static_cast<const E*>(a.G) + t * a.ldg;
    const E* h = static_cast<const E*>(a.H) + t * a.ldh;
    const float m = a.mean[t], s = a.rstd[t];
    Two<double> sum{0.0, 0.0};
    for (int c = (int)threadIdx.x * N; c < a.dim; c += kLongWaves * 64 * N) {
      E gv[N], hv[N];
      float w[N];
      load_raw<false>(g + c, a.dim - c, true, gv);
      load_raw<false>(h + c, a.dim - c, true, hv);
      load_raw<false>(a.w + c, a.dim - c, true, w);
      float da = 0.0f, db = 0.0f;
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const float gw = to_f(gv[e]) * w[e];
        da += gw;
        db += e < a.dim - c ? gw * ((to_f(hv[e]) - m) * s) : 0.0f;
      }
      sum.a += (double)da;
      sum.b += (double)db;
    }
    float m1 = 0.0f;
    if (far_mean(m, s)) {
      double rest = 0.0;
      for (int c = threadIdx.x; c < a.dim; c += kLongWaves * 64) rest += (double)(to_f(h[c]) - m);
      m1 = (float)(row_reduce<kLongWaves>(rest, redm, Add{}) / (double)a.dim);
      sum.b -= (double)m1 * (double)s * sum.a;   // with u of the cols kernel
    }
    const Two<float> dot = row_sums<kLongWaves>(Two<float>{(float)sum.a, (float)sum.b}, red);
    if (threadIdx.x == 0) {
      a.rowc[3 * t] = dot.a / (float)a.dim;
      a.rowc[3 * t + 1] = dot.b / (float)a.dim;
      a.rowc[3 * t + 2] = m1;
    }
  }
}
template <typename E, bool DROP>
__global__ __launch_bounds__(kThr) void layer_norm_cols_kernel(LayerNormBackArgs a, int nparts) {
  constexpr int N = 16 / sizeof(E);
  const int c = ((int)blockIdx.x * kThr + (int)threadIdx.x) * N;
  if (c >= a.dim) return;
  const int left = a.dim - c;
  [[maybe_unused]] drop::Key key{};
  if constexpr (DROP) key = drop::key_of(a.drop);
  float w[N];
  load_raw<false>(a.w + c, left, true, w);
  double dw[N] = {}, db[N] = {};
  for (long long t = blockIdx.y; t < a.T; t += nparts) {
    E g[N], h[N], q[N] = {};
    // A row's cut vector goes by elements: its whole load would take in the vector in
    // front of it, which another thread may have overwritten (dx in place of g or gh)
    auto get = [&](const void* p, long long ld, E (&v)[N]) {
      const E* at = static_cast<const E*>(p) + t * ld + c;
      if (left >= N) {
        load_raw<true>(at, N, true, v);
      } else {
#pragma unroll
        for (int e = 0; e < N; ++e) v[e] = e < left ? at[e] : E(0);
      }
    };
    get(a.G, a.ldg, g);
    get(a.H, a.ldh, h);
    if (a.GH) get(a.GH, a.ldgh, q);
    const float m = a.mean[t], s = a.rstd[t];
    const float ca = a.rowc[3 * t], cb = a.rowc[3 * t + 1], m1 = a.rowc[3 * t + 2];
    float o[N];
#pragma unroll
    for (int e = 0; e < N; ++e) {
      const float gv = to_f(g[e]), u = ((to_f(h[e]) - m) - m1) * s;
      dw[e] += (double)(gv * u);
      db[e] += (double)gv;
      o[e] = s * (gv * w[e] - ca - u * cb) + to_f(q[e]);
    }
    if constexpr (DROP) {
      if (a.GR) store_n<false>(static_cast<E*>(a.GR) + t * a.ldgr + c, left, o);
      drop::apply(a.drop, key, (uint32_t)t, c, o);
    }
    store_n<false>(static_cast<E*>(a.GX) + t * a.ldgx + c, left, o);
  }
  float *pw, *pb, ow[N], ob[N];
  part_rows(a, blockIdx.y, pw, pb);
#pragma unroll
  for (int e = 0; e < N; ++e) {
    ow[e] = (float)dw[e];
    ob[e] = (float)db[e];
  }
  store_raw<false>(pw + c, left, ow);
  store_raw<false>(pb + c, left, ob);
}

// Waves of a CU that share the rows, forward: 16384 x 2048 bf16 45 us with 16, 48 with 24 or 12.
// fp32 rows go one to a group: 94 us, 102 with 16.
template <typename E>
constexpr long long kFwdWaves = sizeof(E) == 2 ? 16 : 1LL << 40;

template <typename E, int NV, int WPR>
void fwd(const LayerNormArgs& a, hipStream_t s) {
  const long long rpw = threads(WPR) / 64 / WPR, groups = (a.T + rpw - 1) / rpw;
  // a few workgroups to a CU, each with as many rows as the others
  const long long most = kFwdWaves<E> * 256 / (threads(WPR) / 64), each = (groups + most - 1) / most;
  const dim3 grid((unsigned)((groups + each - 1) / each)), block(threads(WPR));
  const bool whole = a.dim % (16 / (int)sizeof(E)) == 0, drop = a.drop.threshold != 0;
  if (whole && !drop) hipLaunchKernelGGL((add_layer_norm_kernel<E, NV, WPR, true, false>), grid, block, 0, s, a);
  else if (whole) hipLaunchKernelGGL((add_layer_norm_kernel<E, NV, WPR, true, true>), grid, block, 0, s, a);
  else if (!drop) hipLaunchKernelGGL((add_layer_norm_kernel<E, NV, WPR, false, false>), grid, block, 0, s, a);
  else hipLaunchKernelGGL((add_layer_norm_kernel<E, NV, WPR, false, true>), grid, block, 0, s, a);
}
template <typename E, int NV, int WPR>
void bwd(const LayerNormBackArgs& a, int parts, hipStream_t s) {
  const size_t lds = WPR == 1 ? (size_t)a.dim * 16 : 0;
  const dim3 grid((unsigned)parts), block(threads(WPR));
  const bool whole = a.dim % (16 / (int)sizeof(E)) == 0, drop = a.drop.threshold != 0;
  if (whole && !drop) hipLaunchKernelGGL((layer_norm_backward_kernel<E, NV, WPR, true, false>), grid, block, lds, s, a);
  else if (whole) hipLaunchKernelGGL((layer_norm_backward_kernel<E, NV, WPR, true, true>), grid, block, lds, s, a);
  else if (!drop) hipLaunchKernelGGL((layer_norm_backward_kernel<E, NV, WPR, false, false>), grid, block, lds, s, a);
  else hipLaunchKernelGGL((layer_norm_backward_kernel<E, NV, WPR, false, true>), grid, block, lds, s, a);
}

// f(NV) for the least NV in 1, 2, 3, 4 up to MAX whose NV * per covers dim; false if none
template <int MAX, typename F>
bool with_nv(int dim, int per, F f) {
  if (dim <= per) f(std::integral_constant<int, 1>{});
  else if (dim <= 2 * per) f(std::integral_constant<int, 2>{});
  else if (dim <= 3 * per && MAX >= 3) f(std::integral_constant<int, (MAX >= 3 ? 3 : 1)>{});
  else if (dim <= 4 * per && MAX >= 4) f(std::integral_constant<int, (MAX >= 4 ? 4 : 1)>{});
  else return false;
  return true;
}

// Rows from which one wave takes a row
constexpr long long kManyRows = 1024;

template <typename E>
void fwd_any(const LayerNormArgs& a, hipStream_t s) {
  constexpr int N = 16 / sizeof(E);
  if (a.T >= kManyRows && with_nv<(sizeof(E) == 2 ? 4 : 2)>(a.dim, 64 * N, [&](auto nv) { fwd<E, nv.value, 1>(a, s); })) return;
  if (with_nv<4>(a.dim, 256 * N, [&](auto nv) { fwd<E, nv.value, 4>(a, s); })) return;
  if (with_nv<2>(a.dim, 1024 * N, [&](auto nv) { fwd<E, nv.value, 16>(a, s); })) return;
  const dim3 grid((unsigned)a.T), block(kLongWaves * 64);
  if (a.drop.threshold) hipLaunchKernelGGL((add_layer_norm_long_kernel<E, true>), grid, block, 0, s, a);
  else hipLaunchKernelGGL((add_layer_norm_long_kernel<E, false>), grid, block, 0, s, a);
}
template <typename E>
void bwd_any(const LayerNormBackArgs& a, int parts, hipStream_t s) {
  constexpr int N = 16 / sizeof(E);
  if (a.T >= kManyRows && with_nv<2>(a.dim, 64 * N, [&](auto nv) { bwd<E, nv.value, 1>(a, parts, s); })) return;
  if (with_nv<3>(a.dim, 256 * N, [&](auto nv) { bwd<E, nv.value, 4>(a, parts, s); })) return;
  // four vectors a lane leave a SIMD one wave: eight waves a row instead (4096 x 8192 bf16 65 -> 60 us)
  if (a.dim <= 2 * 512 * N) return bwd<E, 2, 8>(a, parts, s);
  hipLaunchKernelGGL((layer_norm_means_kernel<E>), dim3((unsigned)std::min<long long>(a.T, 4096)), dim3(kLongWaves * 64), 0,
                     s, a);
  const dim3 grid((unsigned)((a.dim + kThr * N - 1) / (kThr * N)), (unsigned)parts);
  if (a.drop.threshold) hipLaunchKernelGGL((layer_norm_cols_kernel<E, true>), grid, dim3(kThr), 0, s, a, parts);
  else hipLaunchKernelGGL((layer_norm_cols_kernel<E, false>), grid, dim3(kThr), 0, s, a, parts);
}

// A launch counts threads in 32 bits: rows of one, for sixteen waves a row
constexpr long long kRowsPerLaunch = 1LL << 21;

template <typename P>
P at(P p, long long bytes) {
  return p ? (P)((uintptr_t)p + bytes) : p;
}

}  // namespace

// Two workgroups to a CU, as in the norm without a mean (k_norm.hip)
int layer_norm_backward_parts(long long T) { return (int)std::min<long long>((T + 1) / 2, 512); }
int layer_norm_back_reg_dim(int bf16) { return 2 * 512 * (bf16 ? 8 : 4); }

hipError_t launch_add_layer_norm(const LayerNormArgs& a, int bf16, hipStream_t s) {
  if (a.dim <= 0 || a.dim > kNormMaxDim) return hipErrorInvalidValue;
  const int es = bf16 ? 2 : 4;
  for (long long t = 0; t < a.T; t += kRowsPerLaunch) {
    LayerNormArgs b = a;
    b.T = std::min(kRowsPerLaunch, a.T - t);
    b.X = at(a.X, t * a.ldx * es);
    b.R = at(a.R, t * a.ldr * es);
    b.H = at(a.H, t * a.ldh * es);
    b.Y = at(a.Y, t * a.ldy * (a.quant ? 1 : es));
    b.scale = at(a.scale, t * 4);
    b.mean = at(a.mean, t * 4);
    b.rstd = at(a.rstd, t * 4);
    b.row0 = (uint32_t)t;
    if (bf16) fwd_any<uint16_t>(b, s);
    else fwd_any<float>(b, s);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

hipError_t launch_layer_norm_backward(const LayerNormBackArgs& a, int bf16, hipStream_t s) {
  if (a.T <= 0 || a.dim <= 0 || a.dim > kNormMaxDim) return hipErrorInvalidValue;
  const int parts = layer_norm_backward_parts(a.T);
  LayerNormBackArgs b = a;
  if (parts == 1) b.part = nullptr;   // the only partial sums are the sums
  if (bf16) bwd_any<uint16_t>(b, parts, s);
  else bwd_any<float>(b, parts, s);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || parts == 1) return e;
  return launch_sum_parts(a.part, parts, 2 * a.dim, a.dw, a.dim, a.db, s);
}

}  // namespace poetx
