// What the kernels of the merged-weight product (k_linear.hip) share: the
// element types with their matrix instructions, and the epilogue.
#pragma once

#include <type_traits>

#include "../../include/poetx.h"
#include "poetx_internal.h"

namespace poetx {
namespace lin {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

// 16 bytes of one operand row per lane: lane l of a 16 x 16 tile holds bytes
// 16 (l >> 4) .. + 15 of a 64-byte slab of row l & 15. Both operands are laid
// out alike, so every product of a slab meets its partner whatever order the
// instruction takes them in. D: lane l holds D[4 (l >> 4) + v][l & 15].
struct TypeBf16 {
  static constexpr int kSize = 2;
  typedef f32x4 Acc;
  typedef float Sum;
  static __device__ __forceinline__ void mma(const i32x4& a, const i32x4& b, Acc& c) {
    c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b),
                                                c, 0, 0, 0);
  }
  // plain products of the 16 bytes, for rows too few for a tile
  static __device__ __forceinline__ void dot(const i32x4& a, const i32x4& b, float& c) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      c = fmaf(__uint_as_float((uint32_t)a[i] << 16), __uint_as_float((uint32_t)b[i] << 16), c);
      c = fmaf(__uint_as_float((uint32_t)a[i] & 0xffff0000u), __uint_as_float((uint32_t)b[i] & 0xffff0000u), c);
    }
  }
};
struct TypeI8 {
  static constexpr int kSize = 1;
  typedef i32x4 Acc;
  typedef int Sum;
  static __device__ __forceinline__ void mma(const i32x4& a, const i32x4& b, Acc& c) {
    c = __builtin_amdgcn_mfma_i32_16x16x64_i8(a, b, c, 0, 0, 0);
  }
  static __device__ __forceinline__ void dot(const i32x4& a, const i32x4& b, int& c) {
#pragma unroll
    for (int i = 0; i < 4; ++i) c = __builtin_amdgcn_sdot4(a[i], b[i], c, false);
  }
};
struct TypeF32 {
  static constexpr int kSize = 4;
  typedef f32x4 Acc;
  typedef float Sum;
  static __device__ __forceinline__ void mma(const i32x4& a, const i32x4& b, Acc& c) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      c = __builtin_amdgcn_mfma_f32_16x16x4f32(__int_as_float(a[i]), __int_as_float(b[i]), c, 0, 0, 0);
  }
  static __device__ __forceinline__ void dot(const i32x4& a, const i32x4& b, float& c) {
#pragma unroll
    for (int i = 0; i < 4; ++i) c = fmaf(__int_as_float(a[i]), __int_as_float(b[i]), c);
  }
};

// This wave's loads and stores but for the last N are done.
template <int N>
__device__ __forceinline__ void vm_wait() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}
// Barrier that waits for this wave's LDS traffic only: global loads stay in flight.
__device__ __forceinline__ void lds_sync() {
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

// 16 bytes of a row of kb bytes from byte k on; what is behind its end counts as
// zero and is not read. Global loads take any alignment on this target. A chunk
// the end cuts is the row's last 16 bytes, moved into place, so that it costs one
// load like the others; a row of less than 16 bytes goes element by element.
template <int ES>
__device__ __forceinline__ i32x4 load16(const char* row, long long k, long long kb) {
  i32x4 v = {0, 0, 0, 0};
  if (kb < 16) {
    uint32_t w[4] = {0, 0, 0, 0};
    for (int b = 0; b < 16 / ES; ++b) {
      if (k + b * ES < kb) {
        uint32_t e = 0;
        __builtin_memcpy(&e, row + k + b * ES, ES);
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] |= b * ES / 4 == i ? e << (8 * (b * ES % 4)) : 0u;
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = (int)w[i];
    return v;
  }
  uint64_t q[2];
  __builtin_memcpy(q, row + (k + 16 <= kb ? k : kb - 16), 16);
  // the chunk starts `cut` bytes into what was loaded
  const int cut = (int)(k + 16 <= kb ? 0 : k - (kb - 16) < 16 ? k - (kb - 16) : 16);
  const int sh = (cut & 7) * 8;
  const uint64_t next = cut < 8 ? q[1] : 0, low = cut < 8 ? q[0] : q[1];
  q[0] = sh ? low >> sh | next << (64 - sh) : low;
  q[1] = next >> sh;
  if (cut >= 16) q[0] = q[1] = 0;
  __builtin_memcpy(&v, q, 16);
  return v;
}

// The tile of this workgroup: XCD x = blockIdx.x % 8 takes the tiles [ntile x / 8,
// ntile (x + 1) / 8) in groups of 4 tile-rows, so that those resident together share
// operand rows in its L2. False for workgroups behind the range. Grid: tile_grid.
__device__ __forceinline__ bool tile_origin(long long T, int m, int bm, int bn, int& m0, int& n0) {
  const int tn = (m + bn - 1) / bn, tm = (int)((T + bm - 1) / bm), ntile = tn * tm;
  const int x = blockIdx.x % 8;
  const int lin = (int)((long long)ntile * x / 8) + (int)blockIdx.x / 8;
  if (lin >= (int)((long long)ntile * (x + 1) / 8)) return false;
  const int grp = lin / (4 * tn), first = grp * 4;
  const int gsz = min(4, tm - first), in = lin - grp * (4 * tn);
  m0 = __builtin_amdgcn_readfirstlane((first + in % gsz) * bm);
  n0 = __builtin_amdgcn_readfirstlane((in / gsz) * bn);
  return true;
}
inline long long tile_grid(long long T, int m, int bm, int bn) {
  return (((T + bm - 1) / bm) * ((m + bn - 1) / bn) + 7) / 8 * 8;
}

// The activations in 32 bits. A result that is rounded to bf16 takes the
// hardware's exponential and reciprocal (a few units of 2^-24 off), an fp32 one
// the library's functions.
template <bool BF16>
__device__ __forceinline__ float logistic(float z) {
  if constexpr (BF16) return __builtin_amdgcn_rcpf(1.0f + __expf(-z));
  else return 1.0f / (1.0f + expf(-z));
}
// z (1 + erf(z / sqrt 2)) / 2 = max(z, 0) - a Q(a) with a = |z| and the normal
// distribution's tail Q(a) = t P(q) exp(-a^2 / 2), t = 1 / (1 + c a), q = 1 - 2 t, P
// fitted for the least relative error over 0 <= a <= 13.3 (a Chebyshev basis, least
// squares with weights raised where the error is largest): 7.5e-9 with degree 9, and
// 6.2e-7 with 6, for results that are rounded to bf16. Nothing cancels, so the result
// is within 14 units of 2^-24 of its own size (bf16: 11 and (3 / 2) z^2 more) down to
// where exp(-a^2 / 2) leaves the normal range; 1 + erf is 4 % off at -5 and zero at
// -5.5. Near a = 0 the tail moves three times as fast as t, so fp32 results put back
// what the reciprocal lost (c a is exact there), and what a^2 and its product with
// log2(e) lost goes back in behind the exponential: 0.7 units rms in 0 .. 1 and 1.2 in
// -1 .. 0, about as 1 + erf, against 1.5 and 2.6. 16384 x 256 x 4096 bf16 to fp32 110 us
// (111 with 1 + erff, 137 with the library's erfcf), to bf16 88 us.
template <bool BF16>
__device__ __forceinline__ float gelu(float z) {
  const float m = fabsf(z), a = m > 16.0f ? 16.0f : m;   // infinities end at Q = 0; NaN stays
  constexpr float kC = -0.72134752044f, kCLow = -0.72134752044448170368 - (double)kC;   // -log2(e) / 2
  const float s = a * a, k = s * kC;
  float e = __builtin_amdgcn_exp2f(k), t, p;
  if constexpr (BF16) {
    t = __builtin_amdgcn_rcpf(fmaf(0.265f, a, 1.0f));
    const float q = fmaf(-2.0f, t, 1.0f);
    p = fmaf(-1.059172291e-3f, q, 2.527494554e-4f);
    p = fmaf(p, q, 1.047615789e-2f);
    p = fmaf(p, q, -4.106033863e-2f);
    p = fmaf(p, q, 9.44208143e-2f);
    p = fmaf(p, q, -1.563923402e-1f);
    p = fmaf(p, q, 1.989619594e-1f);
  } else {
    const float ca = 0.25f * a;
    t = __builtin_amdgcn_rcpf(1.0f + ca);
    const float d = t * fmaf(-ca, t, 1.0f - t);
    const float q = fmaf(-2.0f, d, fmaf(-2.0f, t, 1.0f));
    t += d;
    p = fmaf(-3.142248372e-5f, q, 4.828958238e-5f);
    p = fmaf(p, q, 3.938651346e-4f);
    p = fmaf(p, q, -8.796188821e-4f);
    p = fmaf(p, q, -1.882281462e-3f);
    p = fmaf(p, q, 1.510112642e-2f);
    p = fmaf(p, q, -4.663071063e-2f);
    p = fmaf(p, q, 9.678422074e-2f);
    p = fmaf(p, q, -1.519741526e-1f);
    p = fmaf(p, q, 1.888212839e-1f);
    const float low = fmaf(fmaf(a, a, -s), kC, fmaf(s, kCLow, fmaf(s, kC, -k)));
    e = fmaf(e, low * 0.69314718056f, e);
  }
  return fmaf(-a, t * p * e, fmaxf(z, 0.0f));
}
template <bool BF16>
__device__ __forceinline__ float activate(float z, int act) {
  switch (act) {
    case POETX_ACT_RELU: return z > 0.0f || z != z ? z : 0.0f;
    case POETX_ACT_SILU: return z * logistic<BF16>(z);
    case POETX_ACT_GELU: return gelu<BF16>(z);
    case POETX_ACT_GELU_TANH: {
      const float u = 0.79788456080286536f * (z + 0.044715f * z * z * z);
      // (1 + tanh u) / 2 is the logistic function of 2 u
      return z * logistic<BF16>(2.0f * u);
    }
    default: return z;
  }
}

template <typename E, int N>
struct __attribute__((packed, aligned(sizeof(E)))) Pack {
  E v[N];
};
// N values at p as fp32; the first `cols` with EDGE
template <bool EDGE, int N>
__device__ __forceinline__ void load_cols(const float* p, int cols, float (&o)[N]) {
  if constexpr (EDGE) {
#pragma unroll
    for (int i = 0; i < N; ++i) o[i] = i < cols ? p[i] : 0.0f;
  } else {
    const Pack<float, N> v = *reinterpret_cast<const Pack<float, N>*>(p);
#pragma unroll
    for (int i = 0; i < N; ++i) o[i] = v.v[i];
  }
}
template <bool EDGE, int N>
__device__ __forceinline__ void load_cols(const uint16_t* p, int cols, float (&o)[N]) {
  if constexpr (EDGE) {
#pragma unroll
    for (int i = 0; i < N; ++i) o[i] = i < cols ? __uint_as_float((uint32_t)p[i] << 16) : 0.0f;
  } else {
    const Pack<uint16_t, N> v = *reinterpret_cast<const Pack<uint16_t, N>*>(p);
#pragma unroll
    for (int i = 0; i < N; ++i) o[i] = __uint_as_float((uint32_t)v.v[i] << 16);
  }
}

// N consecutive columns c .. of row t, all of them inside the result (or the first
// `cols` with EDGE). ACT: the activation where the kernel is made for one.
constexpr int kAnyAct = -1;
template <bool BF16, int ACT, bool EDGE, typename S, int N>
__device__ __forceinline__ void finish_cols(const LinearArgs& a, const S (&acc)[N], long long t, int c,
                                            int cols) {
  typedef typename std::conditional<BF16, uint16_t, float>::type E;
  constexpr bool SCALED = std::is_same<S, int>::value;
  // every load out before the first is used: one wait for memory, not four
  float v[N], w[N], b[N], m[N], r0[N];
  float sx = 1.0f;
  if constexpr (SCALED) {
    sx = a.sx[t];
    load_cols<EDGE>(a.sw + c, cols, w);
  }
  if (a.bias) load_cols<EDGE>(a.bias + c, cols, b);
  if (a.mul) load_cols<EDGE>(static_cast<const E*>(a.mul) + t * a.ldm + c, cols, m);
  if (a.res) load_cols<EDGE>(static_cast<const E*>(a.res) + t * a.ldr + c, cols, r0);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    v[i] = (float)acc[i];
    if constexpr (SCALED) v[i] = v[i] * sx * w[i];
    if (a.bias) v[i] += b[i];
    v[i] = activate<BF16>(v[i], ACT == kAnyAct ? a.act : ACT);
    if (a.mul) v[i] *= m[i];
    if (a.res) v[i] += r0[i];
  }
  Pack<E, N> r;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if constexpr (BF16) r.v[i] = __builtin_bit_cast(uint16_t, static_cast<__bf16>(v[i]));
    else r.v[i] = v[i];
  }
  E* y = static_cast<E*>(a.Y) + t * a.ldy + c;
  if constexpr (EDGE) {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (i < cols) y[i] = r.v[i];
  } else {
    *reinterpret_cast<Pack<E, N>*>(y) = r;
  }
}
// the same where the columns may end inside the N
template <bool BF16, int ACT = kAnyAct, typename S, int N>
__device__ __forceinline__ void finish(const LinearArgs& a, const S (&acc)[N], long long t, int c) {
  if (c + N <= a.m) finish_cols<BF16, ACT, false>(a, acc, t, c, N);
  else finish_cols<BF16, ACT, true>(a, acc, t, c, a.m - c);
}

// The sums of split `z` of a shared n: 4 columns of one row (c a multiple of 4; the
// rows of `part` are as long as m up to a multiple of 4)
__device__ __forceinline__ long long part_row(const LinearArgs& a, int z, long long t) {
  return ((long long)z * a.T + t) * ((a.m + 3) / 4 * 4);
}
template <typename Ty>
__device__ __forceinline__ void store_part(const LinearArgs& a, int z, long long t, int c,
                                           const typename Ty::Acc& v) {
  *reinterpret_cast<typename Ty::Acc*>(static_cast<typename Ty::Sum*>(a.part) + part_row(a, z, t) + c) = v;
}

}  // namespace lin
}  // namespace poetx
