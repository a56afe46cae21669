// What the kernels of the merged-weight product (k_linear.hip) share: the
// element types with their matrix instructions, and the epilogue.
#pragma once

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

// 16 bytes at p, of which `left` (a multiple of the element size) belong to the
// row; what is behind them counts as zero and is not read. Global loads take
// any alignment on this target.
template <int ES>
__device__ __forceinline__ i32x4 load16(const char* p, long long left) {
  i32x4 v = {0, 0, 0, 0};
  if (left >= 16) {
    __builtin_memcpy(&v, p, 16);
  } else if (left > 0) {
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 16 / ES; ++i) {
      if (i * ES < left) {
        uint32_t b = 0;
        __builtin_memcpy(&b, p + i * ES, ES);
        w[i * ES / 4] |= b << (8 * (i * ES % 4));
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = (int)w[i];
  }
  return v;
}

__device__ __forceinline__ float load_y(const void* p, long long i, int bf16) {
  return bf16 ? __uint_as_float((uint32_t)static_cast<const uint16_t*>(p)[i] << 16)
              : static_cast<const float*>(p)[i];
}

// The activations in 32 bits. A result that is rounded to bf16 takes the
// hardware's exponential and reciprocal (a few units of 2^-24 off), an fp32 one
// the library's functions.
template <bool BF16>
__device__ __forceinline__ float logistic(float z) {
  if constexpr (BF16) return __builtin_amdgcn_rcpf(1.0f + __expf(-z));
  else return 1.0f / (1.0f + expf(-z));
}
template <bool BF16>
__device__ __forceinline__ float activate(float z, int act) {
  switch (act) {
    case POETX_ACT_RELU: return z > 0.0f || z != z ? z : 0.0f;
    case POETX_ACT_SILU: return z * logistic<BF16>(z);
    case POETX_ACT_GELU: return 0.5f * z * (1.0f + erff(z * 0.70710678118654752f));
    case POETX_ACT_GELU_TANH: {
      const float u = 0.79788456080286536f * (z + 0.044715f * z * z * z);
      // (1 + tanh u) / 2 is the logistic function of 2 u
      return z * logistic<BF16>(2.0f * u);
    }
    default: return z;
  }
}

template <typename S>
__device__ __forceinline__ float scaled(const LinearArgs& a, S acc, long long t, int c) {
  return (float)acc;
}
template <>
__device__ __forceinline__ float scaled<int>(const LinearArgs& a, int acc, long long t, int c) {
  return (float)acc * a.sx[t] * a.sw[c];
}

// N consecutive columns c .. of row t; `cols` of them exist
template <bool BF16, typename S, int N>
__device__ __forceinline__ void finish(const LinearArgs& a, const S (&acc)[N], long long t, int c) {
  const int cols = min(N, a.m - c);
  float v[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if (i >= cols) continue;
    float z = scaled(a, acc[i], t, c + i);
    if (a.bias) z += a.bias[c + i];
    v[i] = activate<BF16>(z, a.act);
  }
  auto operand = [&](const void* p, long long ld, float (&o)[N]) {
    if constexpr (BF16) {
      uint16_t h[N];
      const uint16_t* q = static_cast<const uint16_t*>(p) + t * ld + c;
      if (cols == N) {
        __builtin_memcpy(h, q, sizeof(h));
      } else {
#pragma unroll
        for (int i = 0; i < N; ++i) h[i] = i < cols ? q[i] : 0;
      }
#pragma unroll
      for (int i = 0; i < N; ++i) o[i] = __uint_as_float((uint32_t)h[i] << 16);
    } else {
      const float* q = static_cast<const float*>(p) + t * ld + c;
      if (cols == N) {
        __builtin_memcpy(o, q, sizeof(o));
      } else {
#pragma unroll
        for (int i = 0; i < N; ++i) o[i] = i < cols ? q[i] : 0.0f;
      }
    }
  };
  float o[N];
  if (a.mul) {
    operand(a.mul, a.ldm, o);
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] *= o[i];
  }
  if (a.res) {
    operand(a.res, a.ldr, o);
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += o[i];
  }
  if constexpr (BF16) {
    uint16_t h[N];
#pragma unroll
    for (int i = 0; i < N; ++i) h[i] = __builtin_bit_cast(uint16_t, static_cast<__bf16>(v[i]));
    uint16_t* y = static_cast<uint16_t*>(a.Y) + t * a.ldy + c;
    if (cols == N) {
      __builtin_memcpy(y, h, sizeof(h));
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (i < cols) y[i] = h[i];
    }
  } else {
    float* y = static_cast<float*>(a.Y) + t * a.ldy + c;
    if (cols == N) {
      __builtin_memcpy(y, v, sizeof(v));
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (i < cols) y[i] = v[i];
    }
  }
}

}  // namespace lin
}  // namespace poetx
