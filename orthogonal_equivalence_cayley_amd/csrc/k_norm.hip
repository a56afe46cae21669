// The residual's addition and the root-mean-square norm in front of a block's
// linears, forward and backward, with the output in the activations' type or as
// INT8 rows with one scale each (the rule of the INT8 weight rows, k_quant.hip).
//
//   h = rnd(x + r),  s = (mean h^2 + eps)^(-1/2),  y = (h s) w
//   c = s^2 mean(g w h),  dx = gh + s (g w - h c),  dw = sum_t g h s
//
// Bound by memory: 8 bytes per bf16 element either way (x, r, h, y; g, gh, h,
// dx), 7 with an INT8 output. A row is read once and stays in registers, one
// wave or four to a row, 16-byte loads at any element alignment (the end of a
// row that is no multiple of 16 bytes goes element by element).
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

// `valid` of N elements at p, the rest zero
template <typename E, int N>
__device__ __forceinline__ void load_n(const E* p, int valid, float (&o)[N]) {
  E v[N];
  if (valid >= N) {
    __builtin_memcpy(v, p, sizeof(v));
  } else {
#pragma unroll
    for (int e = 0; e < N; ++e) v[e] = e < valid ? p[e] : E(0);
  }
#pragma unroll
  for (int e = 0; e < N; ++e) o[e] = to_f(v[e]);
}
template <typename E, int N>
__device__ __forceinline__ void store_n(E* p, int valid, const float (&x)[N]) {
  E v[N];
#pragma unroll
  for (int e = 0; e < N; ++e) v[e] = from_f<E>(x[e]);
  if (valid >= N) {
    __builtin_memcpy(p, v, sizeof(v));
  } else {
#pragma unroll
    for (int e = 0; e < N; ++e)
      if (e < valid) p[e] = v[e];
  }
}
template <int N>
__device__ __forceinline__ void store_q(int8_t* p, int valid, const int8_t (&v)[N]) {
  if (valid >= N) {
    __builtin_memcpy(p, v, N);
  } else {
#pragma unroll
    for (int e = 0; e < N; ++e)
      if (e < valid) p[e] = v[e];
  }
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

template <typename E, int NV, int WPR>
__global__ __launch_bounds__(kThr) void add_rms_norm_kernel(NormArgs a) {
  constexpr int N = 16 / sizeof(E);
  constexpr int RPW = kThr / 64 / WPR;   // rows per workgroup
  __shared__ double red[4];
  __shared__ uint32_t redu[4];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const long long t = (long long)blockIdx.x * RPW + wave / WPR;
  if (t >= a.T) return;   // whole rows: with WPR = 4 the workgroup has one row
  const int c0 = ((wave % WPR) * 64 + lane) * N;
  const E* x = static_cast<const E*>(a.X) + t * a.ldx;
  const E* r = a.R ? static_cast<const E*>(a.R) + t * a.ldr : nullptr;
  float h[NV][N];
  double ss = 0.0;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = c0 + i * 64 * WPR * N, left = a.dim - c;
    if (left <= 0) {
#pragma unroll
      for (int e = 0; e < N; ++e) h[i][e] = 0.0f;
      continue;
    }
    load_n<E, N>(x + c, left, h[i]);
    if (r) {
      float q[N];
      load_n<E, N>(r + c, left, q);
      // rounded to the type before the norm: the kept h is what the norm sees
#pragma unroll
      for (int e = 0; e < N; ++e) h[i][e] = to_f(from_f<E>(h[i][e] + q[e]));
    }
    // sums in 64 bits: their order does not show in s, so the INT8 decisions
    // are the same for every split of a row over lanes
#pragma unroll
    for (int e = 0; e < N; ++e) ss += (double)h[i][e] * (double)h[i][e];
  }
  if (a.H) {
    E* ho = static_cast<E*>(a.H) + t * a.ldh;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = c0 + i * 64 * WPR * N;
      if (c < a.dim) store_n<E, N>(ho + c, a.dim - c, h[i]);
    }
  }
  ss = row_reduce<WPR>(ss, red, Add{});
  const float s = (float)(1.0 / sqrt(ss / (double)a.dim + a.eps));
  if (a.rstd && lane == 0 && wave % WPR == 0) a.rstd[t] = s;
  uint32_t amax = 0;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = c0 + i * 64 * WPR * N, left = a.dim - c;
    if (left <= 0) continue;
    float w[N];
    load_n<float, N>(a.w + c, left, w);
#pragma unroll
    for (int e = 0; e < N; ++e) {
      h[i][e] = (h[i][e] * s) * w[e];
      // the elements behind the row's end hold h = 0 and w = 0
      if (e < left) amax = max(amax, __float_as_uint(h[i][e]) & 0x7fffffffu);
    }
    if (!a.quant) store_n<E, N>(static_cast<E*>(a.Y) + t * a.ldy + c, left, h[i]);
  }
  if (!a.quant) return;
  amax = row_reduce<WPR>(amax, redu, Max{});
  float inv, scale;
  int8_rule(amax, inv, scale);
  if (lane == 0 && wave % WPR == 0) a.scale[t] = scale;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = c0 + i * 64 * WPR * N;
    if (c >= a.dim) continue;
    int8_t q[N];
#pragma unroll
    for (int e = 0; e < N; ++e) q[e] = to_q(h[i][e], inv);
    store_q<N>(static_cast<int8_t*>(a.Y) + t * a.ldy + c, a.dim - c, q);
  }
}

// Rows too long for registers: one workgroup to a row, which is read again for
// each pass (from the caches mostly). x and r are read again, never H, so H may
// be x or r only where the registers hold the row; here the sum is taken from H
// once it is written.
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
// workgroup's waves are joined in LDS, one row of `part` per workgroup.
template <typename E, int NV, int WPR>
__global__ __launch_bounds__(kThr) void rms_norm_backward_kernel(NormBackArgs a) {
  constexpr int N = 16 / sizeof(E);
  constexpr int RPW = kThr / 64 / WPR;
  __shared__ float red[4];
  extern __shared__ float dwl[];   // WPR = 1: dim values
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int c0 = ((wave % WPR) * 64 + lane) * N;
  float dw[NV][N] = {};
  for (long long t = (long long)blockIdx.x * RPW + wave / WPR; t < a.T; t += (long long)gridDim.x * RPW) {
    const E* g = static_cast<const E*>(a.G) + t * a.ldg;
    const E* h = static_cast<const E*>(a.H) + t * a.ldh;
    const float s = a.rstd[t];
    float gv[NV][N], hv[NV][N];
    float dot = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = c0 + i * 64 * WPR * N, left = a.dim - c;
      if (left <= 0) {
#pragma unroll
        for (int e = 0; e < N; ++e) gv[i][e] = hv[i][e] = 0.0f;
        continue;
      }
      load_n<E, N>(g + c, left, gv[i]);
      load_n<E, N>(h + c, left, hv[i]);
      float w[N];
      load_n<float, N>(a.w + c, left, w);
#pragma unroll
      for (int e = 0; e < N; ++e) {
        if (e < left) dw[i][e] += gv[i][e] * (hv[i][e] * s);
        gv[i][e] *= w[e];
        dot += gv[i][e] * hv[i][e];
      }
    }
    dot = row_reduce<WPR>(dot, red, Add{});
    const float c_ = dot / (float)a.dim * s * s;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = c0 + i * 64 * WPR * N, left = a.dim - c;
      if (left <= 0) continue;
#pragma unroll
      for (int e = 0; e < N; ++e) gv[i][e] = s * (gv[i][e] - hv[i][e] * c_);
      if (a.GH) {
        float q[N];
        load_n<E, N>(static_cast<const E*>(a.GH) + t * a.ldgh + c, left, q);
#pragma unroll
        for (int e = 0; e < N; ++e) gv[i][e] += q[e];
      }
      store_n<E, N>(static_cast<E*>(a.GX) + t * a.ldgx + c, left, gv[i]);
    }
  }
  float* out = a.part + (long long)blockIdx.x * a.dim;
  if constexpr (WPR == 1) {
    for (int w = 0; w < 4; ++w) {
      if (wave == w) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
          for (int e = 0; e < N; ++e) {
            const int c = c0 + i * 64 * N + e;
            if (c < a.dim) dwl[c] = w == 0 ? dw[i][e] : dwl[c] + dw[i][e];
          }
      }
      __syncthreads();
    }
    for (int c = threadIdx.x; c < a.dim; c += kThr) out[c] = dwl[c];
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = c0 + i * 64 * WPR * N;
      if (c < a.dim) store_n<float, N>(out + c, a.dim - c, dw[i]);
    }
  }
}

// Rows too long for registers: first the factor c of every row, then tiles of
// 256 columns by a range of rows.
template <typename E>
__global__ __launch_bounds__(kThr) void rms_norm_dot_kernel(NormBackArgs a) {
  __shared__ float red[4];
  const long long t = blockIdx.x;
  const E* g = static_cast<const E*>(a.G) + t * a.ldg;
  const E* h = static_cast<const E*>(a.H) + t * a.ldh;
  float dot = 0.0f;
  for (int c = threadIdx.x; c < a.dim; c += kThr) dot += (to_f(g[c]) * a.w[c]) * to_f(h[c]);
  dot = row_reduce<4>(dot, red, Add{});
  const float s = a.rstd[t];
  if (threadIdx.x == 0) a.rowc[t] = dot / (float)a.dim * s * s;
}
template <typename E>
__global__ __launch_bounds__(kThr) void rms_norm_cols_kernel(NormBackArgs a, int nparts) {
  const int c = blockIdx.x * kThr + threadIdx.x;
  if (c >= a.dim) return;
  const float w = a.w[c];
  float dw = 0.0f;
  for (long long t = blockIdx.y; t < a.T; t += nparts) {
    const float g = to_f(static_cast<const E*>(a.G)[t * a.ldg + c]);
    const float h = to_f(static_cast<const E*>(a.H)[t * a.ldh + c]);
    const float s = a.rstd[t];
    dw += g * (h * s);
    float dx = s * (g * w - h * a.rowc[t]);
    if (a.GH) dx += to_f(static_cast<const E*>(a.GH)[t * a.ldgh + c]);
    static_cast<E*>(a.GX)[t * a.ldgx + c] = from_f<E>(dx);
  }
  a.part[(long long)blockIdx.y * a.dim + c] = dw;
}

// dw[c] = sum over the parts, in 64 bits and in a fixed order: 64 columns per
// workgroup, its 16 waves take parts a stride apart
constexpr int kRedThr = 1024;
__global__ __launch_bounds__(kRedThr) void sum_parts_kernel(const float* part, int nparts, int dim,
                                                            float* out) {
  __shared__ double red[kRedThr / 64][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int c = blockIdx.x * 64 + lane;
  double v = 0.0;
  if (c < dim)
#pragma unroll 8
    for (int p = wave; p < nparts; p += kRedThr / 64) v += (double)part[(long long)p * dim + c];
  red[wave][lane] = v;
  __syncthreads();
  if (wave == 0 && c < dim) {
#pragma unroll
    for (int i = 1; i < kRedThr / 64; ++i) v += red[i][lane];
    out[c] = (float)v;
  }
}

template <typename E, int NV, int WPR>
void fwd(const NormArgs& a, hipStream_t s) {
  const long long rpw = kThr / 64 / WPR;
  hipLaunchKernelGGL((add_rms_norm_kernel<E, NV, WPR>), dim3((unsigned)((a.T + rpw - 1) / rpw)), dim3(kThr),
                     0, s, a);
}
template <typename E, int NV, int WPR>
void bwd(const NormBackArgs& a, int parts, hipStream_t s) {
  const size_t lds = WPR == 1 ? (size_t)a.dim * 4 : 0;
  hipLaunchKernelGGL((rms_norm_backward_kernel<E, NV, WPR>), dim3((unsigned)parts), dim3(kThr), lds, s, a);
}

// f(NV) for the least NV in 1, 2, 4, 8 whose NV * per covers dim; false if none
template <typename F>
bool with_nv(int dim, int per, F f) {
  if (dim <= per) f(std::integral_constant<int, 1>{});
  else if (dim <= 2 * per) f(std::integral_constant<int, 2>{});
  else if (dim <= 4 * per) f(std::integral_constant<int, 4>{});
  else if (dim <= 8 * per) f(std::integral_constant<int, 8>{});
  else return false;
  return true;
}

template <typename E>
void fwd_any(const NormArgs& a, hipStream_t s) {
  constexpr int N = 16 / sizeof(E);
  if (a.dim <= 64 * N * 2) {
    with_nv(a.dim, 64 * N, [&](auto nv) { fwd<E, (nv.value > 2 ? 2 : nv.value), 1>(a, s); });
    return;
  }
  if (!with_nv(a.dim, 256 * N, [&](auto nv) { fwd<E, nv.value, 4>(a, s); }))
    hipLaunchKernelGGL((add_rms_norm_long_kernel<E>), dim3((unsigned)a.T), dim3(kThr), 0, s, a);
}
template <typename E>
void bwd_any(const NormBackArgs& a, int parts, hipStream_t s) {
  constexpr int N = 16 / sizeof(E);
  if (a.dim <= 64 * N * 4) {
    with_nv(a.dim, 64 * N, [&](auto nv) { bwd<E, (nv.value > 4 ? 4 : nv.value), 1>(a, parts, s); });
  } else if (a.dim <= 256 * N * 4) {
    with_nv(a.dim, 256 * N, [&](auto nv) { bwd<E, (nv.value > 4 ? 4 : nv.value), 4>(a, parts, s); });
  } else {
    hipLaunchKernelGGL((rms_norm_dot_kernel<E>), dim3((unsigned)a.T), dim3(kThr), 0, s, a);
    hipLaunchKernelGGL((rms_norm_cols_kernel<E>), dim3((unsigned)((a.dim + kThr - 1) / kThr), (unsigned)parts),
                       dim3(kThr), 0, s, a, parts);
  }
}

}  // namespace

int norm_backward_parts(long long T) { return (int)std::min<long long>((T + 3) / 4, 512); }

hipError_t launch_add_rms_norm(const NormArgs& a, int bf16, hipStream_t s) {
  if (a.T <= 0) return hipSuccess;
  if (a.T > 0x7fffffffLL || a.dim <= 0) return hipErrorInvalidValue;
  if (bf16) fwd_any<uint16_t>(a, s);
  else fwd_any<float>(a, s);
  return hipGetLastError();
}

hipError_t launch_rms_norm_backward(const NormBackArgs& a, int bf16, hipStream_t s) {
  if (a.T <= 0 || a.T > 0x7fffffffLL || a.dim <= 0) return hipErrorInvalidValue;
  const int parts = norm_backward_parts(a.T);
  if (bf16) bwd_any<uint16_t>(a, parts, s);
  else bwd_any<float>(a, parts, s);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(sum_parts_kernel, dim3((unsigned)((a.dim + 63) / 64)), dim3(kRedThr), 0, s, a.part, parts,
                     a.dim, a.dw);
  return hipGetLastError();
}

}  // namespace poetx
