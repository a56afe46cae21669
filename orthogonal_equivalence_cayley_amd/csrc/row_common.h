// What the kernels of the norms (k_norm.hip, k_layer_norm.hip) and of dropout
// (k_dropout.hip) share: a row's loads and stores in 16-byte vectors, sums over the
// waves of a row, the rule of INT8 rows.
#pragma once

#include "poetx_internal.h"

namespace poetx {
namespace row {

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

}  // namespace row
}  // namespace poetx
