// The residual's addition and the root-mean-square norm in front of a block's
// linears, forward and backward, with the output in the activations' type or as
// INT8 rows with one scale each (the rule of the INT8 weight rows, k_quant.hip).
//
//   h = rnd(x + r),  s = (mean h^2 + eps)^(-1/2),  y = (h s) w
//   c = s^2 mean(g w h),  dx = gh + s (g w - h c),  dw = sum_t g h s
//
// Bound by memory: 8 bytes per bf16 element either way (x, r, h, y; g, gh, h,
// dx), 7 with an INT8 output. A row is read once and stays in registers, one
// wave or four to a row, 16-byte loads at any element alignment, every load of a
// row (and, backward, of the next row) out before the first is used. Measured
// with the inputs cold: 16384 x 2048 bf16 forward 43 to 45 us (6.0 to 6.2 TB/s; a kernel that
// only adds two arrays into two others reaches 5.3 to 6.1 TB/s here), backward 46
// + 5 us; 16384 x 4096 to INT8 85 us (5.6 TB/s); one row of 2048 2.4 us.
#include <algorithm>
#include <type_traits>

#include "poetx_internal.h"

namespace poetx {
namespace {

constexpr int kThr = 256;

__device__ __forceinline__ float to_f(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }
__device__ __forceinline__ float to_f(float v) { return v; }
template <typename E>
__device__ __forceinline__ E from_f(float v);
template <>
__device__ __forceinline__ float from_f<float>(float v) { return v; }
template <>
__device__ __forceinline__ uint16_t from_f<uint16_t>(float v) {
  return __builtin_bit_cast(uint16_t, static_cast<__bf16>(v));
}

// N elements of type E as loaded: whole 16-byte vectors at any element alignment.
// `left` elements of the row remain; with WHOLE rows a vector is never cut. A cut
// one of a row of N elements or more (`full`) is the row's last N elements, moved
// into place, so that it costs one load like the others; of a shorter row, it
// goes element by element. (Loops over p[e] under a bound would not do: the
// compiler then splits the whole vectors' loads and stores too, at 74 against 43
// us on 16384 x 2048 bf16.)
template <typename E, int N>
struct __attribute__((packed, aligned(sizeof(E)))) Vec {
  E v[N];
};
// o[e] = x[e + k] (DOWN) or x[e - k], zero where there is none; 0 <= k < N
template <bool DOWN, typename E, int N>
__device__ __forceinline__ void shift(E (&x)[N], int k) {
#pragma unroll
  for (int b = 1; b < N; b *= 2) {
    E y[N];
#pragma unroll
    for (int e = 0; e < N; ++e) {
      const int f = DOWN ? e + b : e - b;
      y[e] = f >= 0 && f < N ? x[f] : E(0);
    }
#pragma unroll
    for (int e = 0; e < N; ++e) x[e] = k & b ? y[e] : x[e];
  }
}
template <bool WHOLE, typename E, int N>
__device__ __forceinline__ void load_raw(const E* p, int left, bool full, E (&o)[N]) {
  const bool cut = !WHOLE && left < N;
  if (cut && !full) {
#pragma unroll
    for (int e = 0; e < N; ++e) o[e] = E(0);
#pragma unroll 1
    for (int k = 0; k < left; ++k) {
      const E x = p[k];
#pragma unroll
      for (int e = 0; e < N; ++e) o[e] = e == k ? x : o[e];
    }
    return;
  }
  const Vec<E, N> v = *reinterpret_cast<const Vec<E, N>*>(cut ? p + left - N : p);
#pragma unroll
  for (int e = 0; e < N; ++e) o[e] = v.v[e];
  if (cut) shift<true>(o, N - left);
}
template <bool WHOLE, typename E, int N>
__device__ __forceinline__ void store_raw(E* p, int left, const E (&x)[N]) {
  if (WHOLE || left >= N) {
    Vec<E, N> v;
#pragma unroll
    for (int e = 0; e < N; ++e) v.v[e] = x[e];
    *reinterpret_cast<Vec<E, N>*>(p) = v;
  } else {
    E y[N];
#pragma unroll
    for (int e = 0; e < N; ++e) y[e] = x[e];
    shift<false>(y, N - left);
    E* q = p + left;   // behind the row's end
#pragma unroll
    for (int e = 0; e < N; ++e)
      if (e >= N - left) q[e - N] = y[e];
  }
}
template <bool WHOLE, typename E, int N>
__device__ __forceinline__ void store_n(E* p, int left, const float (&x)[N]) {
  E v[N];
#pragma unroll
  for (int e = 0; e < N; ++e) v[e] = from_f<E>(x[e]);
  store_raw<WHOLE>(p, left, v);
}

struct Add {
  template <typename V>
  __device__ __forceinline__ V operator()(V a, V b) const { return a + b; }
};
struct Max {
  template <typename V>
  __device__ __forceinline__ V operator()(V a, V b) const { return a > b ? a : b; }
};

// Over the WPR waves of a row, the result in every lane; `red` holds WPR values
// per use. Two barriers where waves have to meet, none for a wave of its own.
template <int WPR, typename V, typename F>
__device__ __forceinline__ V row_reduce(V v, V* red, F f) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v = f(v, __shfl_xor(v, o));
  if constexpr (WPR > 1) {
    const int wave = threadIdx.x >> 6;
    __syncthreads();   // the last use of `red` is over
    if ((threadIdx.x & 63) == 0) red[wave] = v;
    __syncthreads();
    v = red[0];
#pragma unroll
    for (int i = 1; i < WPR; ++i) v = f(v, red[i]);
  }
  return v;
}

// INT8 rule of a row from the bits of its largest magnitude (as unsigned
// numbers NaN > inf > finite): the factor to the 8-bit grid and the scale. A
// magnitude below 2^-119, where 127 / a would overflow, counts as zero; one that
// is not finite gives q = 0 and a NaN scale, so that the row's values are NaN.
__device__ __forceinline__ void int8_rule(uint32_t abits, float& inv, float& scale) {
  const float a = __uint_as_float(abits);
  const bool none = a < 0x1p-119f, bad = abits >= 0x7f800000u;
  inv = none || bad ? 0.0f : 127.0f / a;
  scale = bad ? __uint_as_float(0x7fc00000u) : (none ? 0.0f : a / 127.0f);
}
__device__ __forceinline__ int8_t to_q(float y, float inv) {
  // a factor of 0 marks a row of zeros or one that is not finite: q = 0 there
  return inv == 0.0f ? (int8_t)0 : (int8_t)fminf(fmaxf(rintf(y * inv), -127.0f), 127.0f);
}

template <typename E, int NV, int WPR, bool WHOLE>
__global__ __launch_bounds__(kThr) void add_rms_norm_kernel(NormArgs a) {
  constexpr int N = 16 / sizeof(E);
  constexpr int RPW = kThr / 64 / WPR;   // rows per workgroup
  constexpr int STEP = 64 * WPR * N;     // columns between a lane's vectors
  __shared__ double red[4];
  __shared__ uint32_t redu[4];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const long long t = (long long)blockIdx.x * RPW + wave / WPR;
  if (t >= a.T) return;   // whole rows: with WPR = 4 the workgroup has one row
  const int c0 = ((wave % WPR) * 64 + lane) * N;
  const bool full = a.dim >= N;
  const E* x = static_cast<const E*>(a.X) + t * a.ldx + c0;
  E xr[NV][N], rr[NV][N];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
#pragma unroll
    for (int e = 0; e < N; ++e) xr[i][e] = rr[i][e] = E(0);
    if (c0 + i * STEP < a.dim) load_raw<WHOLE>(x + i * STEP, a.dim - c0 - i * STEP, full, xr[i]);
  }
  if (a.R) {
    const E* r = static_cast<const E*>(a.R) + t * a.ldr + c0;
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (c0 + i * STEP < a.dim) load_raw<WHOLE>(r + i * STEP, a.dim - c0 - i * STEP, full, rr[i]);
  }
  float h[NV][N];
  double ss = 0.0;
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int e = 0; e < N; ++e) {
      h[i][e] = to_f(xr[i][e]);
      // rounded to the type before the norm: the kept h is what the norm sees
      if (a.R) h[i][e] = to_f(from_f<E>(h[i][e] + to_f(rr[i][e])));
      // sums in 64 bits: their order does not show in s, so the INT8 decisions
      // are the same for every split of a row over lanes
      ss += (double)h[i][e] * (double)h[i][e];
    }
  if (a.H) {
    E* ho = static_cast<E*>(a.H) + t * a.ldh + c0;
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (c0 + i * STEP < a.dim) store_n<WHOLE>(ho + i * STEP, a.dim - c0 - i * STEP, h[i]);
  }
  ss = row_reduce<WPR>(ss, red, Add{});
  const float s = (float)(1.0 / sqrt(ss / (double)a.dim + a.eps));
  if (a.rstd && lane == 0 && wave % WPR == 0) a.rstd[t] = s;
  uint32_t amax = 0;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int left = a.dim - c0 - i * STEP;
    if (left <= 0) continue;
    float w[N];
    load_raw<WHOLE>(a.w + c0 + i * STEP, left, full, w);
#pragma unroll
    for (int e = 0; e < N; ++e) {
      h[i][e] = (h[i][e] * s) * w[e];
      // behind the row's end stands 0 s, which an infinite s makes NaN
      if (WHOLE || e < left) amax = max(amax, __float_as_uint(h[i][e]) & 0x7fffffffu);
    }
    if (!a.quant) store_n<WHOLE>(static_cast<E*>(a.Y) + t * a.ldy + c0 + i * STEP, left, h[i]);
  }
  if (!a.quant) return;
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

// Rows too long for registers: one workgroup to a row, which is read again for
// each pass (from the caches mostly). Where H is written its values are what is
// read again, each by the thread that wrote it, so H may be X or R itself.
template <typename E>
__global__ __launch_bounds__(kThr) void add_rms_norm_long_kernel(NormArgs a) {
  __shared__ double red[4];
  __shared__ uint32_t redu[4];
  const long long t = blockIdx.x;
  const E* x = static_cast<const E*>(a.X) + t * a.ldx;
  const E* r = a.R ? static_cast<const E*>(a.R) + t * a.ldr : nullptr;
  E* ho = a.H ? static_cast<E*>(a.H) + t * a.ldh : nullptr;
  double ss = 0.0;
  for (int c = threadIdx.x; c < a.dim; c += kThr) {
    float h = to_f(x[c]);
    if (r) h = to_f(from_f<E>(h + to_f(r[c])));
    if (ho) ho[c] = from_f<E>(h);
    ss += (double)h * (double)h;
  }
  ss = row_reduce<4>(ss, red, Add{});
  const float s = (float)(1.0 / sqrt(ss / (double)a.dim + a.eps));
  if (a.rstd && threadIdx.x == 0) a.rstd[t] = s;
  // a thread reads back only what it wrote itself
  auto value = [&](int c) {
    float h;
    if (ho) {
      h = to_f(ho[c]);
    } else {
      h = to_f(x[c]);
      if (r) h = to_f(from_f<E>(h + to_f(r[c])));
    }
    return (h * s) * a.w[c];
  };
  uint32_t amax = 0;
  for (int c = threadIdx.x; c < a.dim; c += kThr) {
    const float y = value(c);
    amax = max(amax, __float_as_uint(y) & 0x7fffffffu);
    if (!a.quant) static_cast<E*>(a.Y)[t * a.ldy + c] = from_f<E>(y);
  }
  if (!a.quant) return;
  amax = row_reduce<4>(amax, redu, Max{});
  float inv, scale;
  int8_rule(amax, inv, scale);
  if (threadIdx.x == 0) a.scale[t] = scale;
  for (int c = threadIdx.x; c < a.dim; c += kThr)
    static_cast<int8_t*>(a.Y)[t * a.ldy + c] = to_q(value(c), inv);
}

// Backward: each wave (WPR = 1) or workgroup (WPR = 4) takes rows a stride
// apart and keeps its columns' part of dw in registers; the parts of a
// workgroup's waves are joined in LDS, one row of `part` per workgroup. The
// next row's loads are in flight while a row is worked on. dw is a sum over any
// number of rows, so it is held in 64 bits up to the workgroup's part, which is
// rounded once: in fp32 small terms behind large ones were lost, and the error grew
// with the rows (15 times that of a 64-bit sum of fp32 terms at 2^20 rows). It takes
// no time beside the loads: 16384 x 2048 bf16 51 us either way, 4096 x 8192 54.7
// against 53.9, where the registers leave one wave a SIMD instead of two.
template <typename E, int NV, int WPR, bool WHOLE>
__global__ __launch_bounds__(kThr) void rms_norm_backward_kernel(NormBackArgs a) {
  constexpr int N = 16 / sizeof(E);
  constexpr int RPW = kThr / 64 / WPR;
  constexpr int STEP = 64 * WPR * N;
  __shared__ float red[4];
  extern __shared__ double dwl[];   // WPR = 1: dim values
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int c0 = ((wave % WPR) * 64 + lane) * N;
  const bool full = a.dim >= N;
  double dw[NV][N] = {};
  float w[NV][N] = {};
#pragma unroll
  for (int i = 0; i < NV; ++i)
    if (c0 + i * STEP < a.dim) load_raw<WHOLE>(a.w + c0 + i * STEP, a.dim - c0 - i * STEP, full, w[i]);
  E gr[NV][N] = {}, hr[NV][N] = {}, qr[NV][N] = {};
  float sn = 0.0f;
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
    sn = a.rstd[t];
  };
  const long long stride = (long long)gridDim.x * RPW;
  long long t = (long long)blockIdx.x * RPW + wave / WPR;
  if (t < a.T) fetch(t);
  for (; t < a.T; t += stride) {
    const float s = sn;
    float gv[NV][N], hv[NV][N], q[NV][N];
    float dot = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < N; ++e) {
        gv[i][e] = to_f(gr[i][e]);
        hv[i][e] = to_f(hr[i][e]);
        q[i][e] = to_f(qr[i][e]);
        dw[i][e] += (double)(gv[i][e] * (hv[i][e] * s));
        gv[i][e] *= w[i][e];
        dot += gv[i][e] * hv[i][e];
      }
    if (t + stride < a.T) fetch(t + stride);
    dot = row_reduce<WPR>(dot, red, Add{});
    const float c = dot / (float)a.dim * s * s;
    E* o = static_cast<E*>(a.GX) + t * a.ldgx + c0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
#pragma unroll
      for (int e = 0; e < N; ++e) gv[i][e] = s * (gv[i][e] - hv[i][e] * c) + q[i][e];
      if (c0 + i * STEP < a.dim) store_n<WHOLE>(o + i * STEP, a.dim - c0 - i * STEP, gv[i]);
    }
  }
  float* out = a.part + (long long)blockIdx.x * a.dim;
  if constexpr (WPR == 1) {
    for (int k = 0; k < kThr / 64; ++k) {
      if (wave == k) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
          for (int e = 0; e < N; ++e) {
            const int c = c0 + i * STEP + e;
            if (c < a.dim) dwl[c] = k == 0 ? dw[i][e] : dwl[c] + dw[i][e];
          }
      }
      __syncthreads();
    }
    for (int c = threadIdx.x; c < a.dim; c += kThr) out[c] = (float)dwl[c];
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float o[N];
#pragma unroll
      for (int e = 0; e < N; ++e) o[e] = (float)dw[i][e];
      if (c0 + i * STEP < a.dim) store_raw<WHOLE>(out + c0 + i * STEP, a.dim - c0 - i * STEP, o);
    }
  }
}

// Rows too long for registers: first the factor c of every row, then tiles of
// 256 columns by a range of rows.
template <typename E>
__global__ __launch_bounds__(kThr) void rms_norm_dot_kernel(NormBackArgs a) {
  __shared__ float red[4];
  for (long long t = blockIdx.x; t < a.T; t += gridDim.x) {
    const E* g = static_cast<const E*>(a.G) + t * a.ldg;
    const E* h = static_cast<const E*>(a.H) + t * a.ldh;
    float dot = 0.0f;
    for (int c = threadIdx.x; c < a.dim; c += kThr) dot += (to_f(g[c]) * a.w[c]) * to_f(h[c]);
    dot = row_reduce<4>(dot, red, Add{});
    const float s = a.rstd[t];
    if (threadIdx.x == 0) a.rowc[t] = dot / (float)a.dim * s * s;
  }
}
template <typename E>
__global__ __launch_bounds__(kThr) void rms_norm_cols_kernel(NormBackArgs a, int nparts) {
  const int c = blockIdx.x * kThr + threadIdx.x;
  if (c >= a.dim) return;
  const float w = a.w[c];
  double dw = 0.0;
  for (long long t = blockIdx.y; t < a.T; t += nparts) {
    const float g = to_f(static_cast<const E*>(a.G)[t * a.ldg + c]);
    const float h = to_f(static_cast<const E*>(a.H)[t * a.ldh + c]);
    const float s = a.rstd[t];
    dw += (double)(g * (h * s));
    float dx = s * (g * w - h * a.rowc[t]);
    if (a.GH) dx += to_f(static_cast<const E*>(a.GH)[t * a.ldgh + c]);
    static_cast<E*>(a.GX)[t * a.ldgx + c] = from_f<E>(dx);
  }
  a.part[(long long)blockIdx.y * a.dim + c] = (float)dw;
}

// dw[c] = sum over the parts, in 64 bits and in a fixed order: 32 columns per
// workgroup, its 32 half-waves take parts a stride apart, 16 loads out at once
// (512 parts of 2048 columns 5.0 us, 502 of 1365 3.9 us; 5.4 with the loads behind
// the last whole batch one by one)
constexpr int kRedThr = 1024, kRedCols = 32;
__global__ __launch_bounds__(kRedThr) void sum_parts_kernel(const float* part, int nparts, int dim,
                                                            float* out) {
  constexpr int G = kRedThr / kRedCols;
  __shared__ double red[G][kRedCols];
  const int col = threadIdx.x % kRedCols, grp = threadIdx.x / kRedCols;
  const int c = blockIdx.x * kRedCols + col;
  double v = 0.0;
  const float* const at = part + min(c, dim - 1);
  for (int p0 = grp; p0 < nparts; p0 += 16 * G) {
    float x[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = at[(long long)min(p0 + i * G, nparts - 1) * dim];
#pragma unroll
    for (int i = 0; i < 16; ++i) v += p0 + i * G < nparts ? (double)x[i] : 0.0;
  }
  red[grp][col] = v;
  __syncthreads();
  if (grp == 0 && c < dim) {
#pragma unroll
    for (int i = 1; i < G; ++i) v += red[i][col];
    out[c] = (float)v;
  }
}

template <typename E, int NV, int WPR>
void fwd(const NormArgs& a, hipStream_t s) {
  const long long rpw = kThr / 64 / WPR;
  const dim3 grid((unsigned)((a.T + rpw - 1) / rpw));
  if (a.dim % (16 / (int)sizeof(E)) == 0)
    hipLaunchKernelGGL((add_rms_norm_kernel<E, NV, WPR, true>), grid, dim3(kThr), 0, s, a);
  else
    hipLaunchKernelGGL((add_rms_norm_kernel<E, NV, WPR, false>), grid, dim3(kThr), 0, s, a);
}
template <typename E, int NV, int WPR>
void bwd(const NormBackArgs& a, int parts, hipStream_t s) {
  const size_t lds = WPR == 1 ? (size_t)a.dim * 8 : 0;
  if (a.dim % (16 / (int)sizeof(E)) == 0)
    hipLaunchKernelGGL((rms_norm_backward_kernel<E, NV, WPR, true>), dim3((unsigned)parts), dim3(kThr), lds, s, a);
  else
    hipLaunchKernelGGL((rms_norm_backward_kernel<E, NV, WPR, false>), dim3((unsigned)parts), dim3(kThr), lds, s,
                       a);
}

// f(NV) for the least NV in 1, 2, 4, 8 up to MAX whose NV * per covers dim; false if none
template <int MAX, typename F>
bool with_nv(int dim, int per, F f) {
  if (dim <= per) f(std::integral_constant<int, 1>{});
  else if (dim <= 2 * per) f(std::integral_constant<int, 2>{});
  else if (dim <= 4 * per && MAX >= 4) f(std::integral_constant<int, (MAX >= 4 ? 4 : 1)>{});
  else if (dim <= 8 * per && MAX >= 8) f(std::integral_constant<int, (MAX >= 8 ? 8 : 1)>{});
  else return false;
  return true;
}

// Rows from which one wave takes a row: forward the border is here (1024 x 512 bf16
// 3.6 against 4.3 us, 512 x 1024 4.6 against 3.9); backward four waves stay ahead up
// to some 2000 rows (1024 x 1024 bf16 11.4 against 8.8 us, 2048 x 512 9.7 against 9.8,
// 4096 x 512 11.5 against 13.8).
constexpr long long kManyRows = 1024;

template <typename E>
void fwd_any(const NormArgs& a, hipStream_t s) {
  constexpr int N = 16 / sizeof(E);
  // One wave to a row where it is short and rows are many, else four: 16384 x
  // 1024 bf16 22.5 against 26.9 us, but one row of 1024 3.0 against 2.5 us, and
  // 16384 x 2048 50 against 43 us.
  if (a.T >= kManyRows && with_nv<2>(a.dim, 64 * N, [&](auto nv) { fwd<E, nv.value, 1>(a, s); })) return;
  if (!with_nv<8>(a.dim, 256 * N, [&](auto nv) { fwd<E, nv.value, 4>(a, s); }))
    hipLaunchKernelGGL((add_rms_norm_long_kernel<E>), dim3((unsigned)a.T), dim3(kThr), 0, s, a);
}
template <typename E>
void bwd_any(const NormBackArgs& a, int parts, hipStream_t s) {
  constexpr int N = 16 / sizeof(E);
  // as forward: 16384 x 1024 bf16 28.3 against 35.3 us, one row 7.8 against 4.6
  // us, 16384 x 2048 64 against 50 us
  if (a.T >= kManyRows && with_nv<2>(a.dim, 64 * N, [&](auto nv) { bwd<E, nv.value, 1>(a, parts, s); })) return;
  if (with_nv<4>(a.dim, 256 * N, [&](auto nv) { bwd<E, nv.value, 4>(a, parts, s); })) return;
  hipLaunchKernelGGL((rms_norm_dot_kernel<E>), dim3((unsigned)std::min<long long>(a.T, 8192)), dim3(kThr), 0, s, a);
  hipLaunchKernelGGL((rms_norm_cols_kernel<E>), dim3((unsigned)((a.dim + kThr - 1) / kThr), (unsigned)parts),
                     dim3(kThr), 0, s, a, parts);
}

}  // namespace

// Two workgroups to a CU: 16384 x 2048 bf16 takes 45 us with 512, 58 with 256
// (too few loads in flight) and 50 with 1024 (twice the partial sums).
int norm_backward_parts(long long T) { return (int)std::min<long long>((T + 1) / 2, 512); }

namespace {

// A launch counts threads in 32 bits: rows of one, for a workgroup of 256 a row
constexpr long long kRowsPerLaunch = 1LL << 23;

template <typename E>
const E* at(const E* p, long long n) { return p ? p + n : nullptr; }
template <typename E>
E* at(E* p, long long n) { return p ? p + n : nullptr; }
const void* at(const void* p, long long bytes) { return at(static_cast<const char*>(p), bytes); }
void* at(void* p, long long bytes) { return at(static_cast<char*>(p), bytes); }

}  // namespace

hipError_t launch_add_rms_norm(const NormArgs& a, int bf16, hipStream_t s) {
  if (a.dim <= 0 || a.dim > kNormMaxDim) return hipErrorInvalidValue;
  const int es = bf16 ? 2 : 4;
  for (long long t = 0; t < a.T; t += kRowsPerLaunch) {
    NormArgs b = a;
    b.T = std::min(kRowsPerLaunch, a.T - t);
    b.X = at(a.X, t * a.ldx * es);
    b.R = at(a.R, t * a.ldr * es);
    b.H = at(a.H, t * a.ldh * es);
    b.Y = at(a.Y, t * a.ldy * (a.quant ? 1 : es));
    b.scale = at(a.scale, t);
    b.rstd = at(a.rstd, t);
    if (bf16) fwd_any<uint16_t>(b, s);
    else fwd_any<float>(b, s);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

hipError_t launch_rms_norm_backward(const NormBackArgs& a, int bf16, hipStream_t s) {
  if (a.T <= 0 || a.dim <= 0 || a.dim > kNormMaxDim) return hipErrorInvalidValue;
  const int parts = norm_backward_parts(a.T);
  NormBackArgs b = a;
  if (parts == 1) b.part = a.dw;   // the only partial sum is the sum
  if (bf16) bwd_any<uint16_t>(b, parts, s);
  else bwd_any<float>(b, parts, s);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || parts == 1) return e;
  hipLaunchKernelGGL(sum_parts_kernel, dim3((unsigned)((a.dim + kRedCols - 1) / kRedCols)), dim3(kRedThr), 0, s, a.part, parts,
                     a.dim, a.dw);
  return hipGetLastError();
}

}  // namespace poetx
