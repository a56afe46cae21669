// What the kernels of the vocabulary's cross entropy share (k_vocab_loss.hip,
// k_vocab_loss_pipe.hip, k_vocab_loss_ring.hip): loads to LDS, the parts of their epilogues.
#pragma once

#include "linear_common.h"

namespace poetx {
namespace vocab {

using lin::Pack;

// 16 bytes per lane from the buffer's byte `off` + `soff` to lane * 16 behind the LDS address
// `to`. WRITTEN out for kernels that read by the transposing LDS read: beside the builtin the
// compiler lets every such read of the wave wait for all its loads (16384 tokens, 8192 rows
// of 2048: d W 553 -> 421, d^T X 591 -> 422 us). It has no result in registers; vm_wait waits
// for it. M0, which the compiler keeps to itself, is left as it was; the s_nop is for scalar
// operands that a vector instruction wrote.
typedef uint32_t Buffer __attribute__((ext_vector_type(4)));
__device__ __forceinline__ Buffer buffer_at(const char* p, uint32_t bytes) {
  const uint64_t a = (uint64_t)(uintptr_t)p;
  return Buffer{(uint32_t)a, (uint32_t)(a >> 32) & 0xffffu, bytes, 0x00020000u};
}
template <bool WRITTEN>
__device__ __forceinline__ void load_lds(const char* p, uint32_t bytes, uint32_t to, uint32_t off, uint32_t soff) {
  if constexpr (WRITTEN) {
    uint32_t m0;
    asm volatile(
        "s_mov_b32 %0, m0\n\ts_mov_b32 m0, %1\n\ts_nop 4\n\tbuffer_load_dwordx4 %2, %3, %4 offen lds\n\ts_mov_b32 m0, %0"
        : "=&s"(m0)
        : "s"(to), "v"(off), "s"(buffer_at(p, bytes)), "s"(soff));
  } else {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(
        __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(p), (short)0, (int)bytes, 0x00020000),
        (__attribute__((address_space(3))) void*)(uintptr_t)to, 16, off, soff, 0, 0);
  }
}

// exp of fp32 logits by the library's function, of bf16 products by the hardware's (its
// result is summed beside thousands of others, or rounded to bf16)
template <bool F32>
__device__ __forceinline__ float exp_of(float x) {
  if constexpr (F32) return expf(x);
  else return __expf(x);
}

enum Mode { STATS, GRAD, DX, DW };   // logits with their statistics or as dL/dz, d W, d^T X

// One factor for all tokens is left out of d and multiplied into the results. Not so if it is no
// finite number (the mean's 1 / count where no token counts): 0 times it would not be the 0 of
// ignored tokens, so it goes into the d of the others.
__device__ __forceinline__ bool behind_sums(const VocabArgs& a) { return !a.g_each && fabsf(*a.g) < __builtin_inff(); }
__device__ __forceinline__ float scale_of(const VocabArgs& a) { return behind_sums(a) ? *a.g : 1.0f; }

// What the backward needs of a row
struct Row {
  float lse, factor;
  long long target;   // -1: none (ignored, factor 0)
};
__device__ __forceinline__ Row token_of(const VocabArgs& a, long long t) {
  const long long target = a.target[t];
  if (target == a.ignore) return Row{0.0f, 0.0f, -1};
  // a target outside the vocabulary has no loss: its gradients are NaN
  const bool bad = target < 0 || target >= a.V;
  return Row{a.lse[t], bad ? __builtin_nanf("") : a.g_each ? a.g[t] : behind_sums(a) ? 1.0f : *a.g, target};
}
// dL/dz of column v, but for a factor behind the sums
template <bool F32>
__device__ __forceinline__ float grad_of(const Row& r, float z, long long v) {
  // an ignored row is zero whatever its logits are
  if (r.target < 0 && r.factor == 0.0f) return 0.0f;
  const float p = exp_of<F32>(z - r.lse);
  return (v == r.target ? p - 1.0f : p) * r.factor;
}

template <bool F32>
__device__ __forceinline__ void put(const void* base, long long at, const float (&v)[4], int cols) {
  if constexpr (F32) {
    float* const p = static_cast<float*>(const_cast<void*>(base)) + at;
    if (cols >= 4) {
      *reinterpret_cast<Pack<float, 4>*>(p) = Pack<float, 4>{{v[0], v[1], v[2], v[3]}};
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < cols) p[i] = v[i];
    }
  } else {
    uint16_t* const p = static_cast<uint16_t*>(const_cast<void*>(base)) + at;
    Pack<uint16_t, 4> o;
#pragma unroll
    for (int i = 0; i < 4; ++i) o.v[i] = __builtin_bit_cast(uint16_t, static_cast<__bf16>(v[i]));
    if (cols >= 4) {
      *reinterpret_cast<Pack<uint16_t, 4>*>(p) = o;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < cols) p[i] = o.v[i];
    }
  }
}

// What becomes of a wave's TM x TN tiles of 16 x 16 at row m0 + wm and column n0 + wn of a
// product of rows x cols; `share`: the workgroup's among those that share a sum (DX).
template <typename Ty, int BN, int TM, int TN, Mode MODE>
__device__ __forceinline__ void epilogue(const VocabArgs& a, typename Ty::Acc (&acc)[TM][TN], int rows, int cols, int m0,
                                         int n0, int wm, int wn, int share) {
  constexpr bool F32 = Ty::kSize == 4;
  const int lane = threadIdx.x & 63;
  // lane l holds row l & 15 of each tile and 4 of its columns, from 4 (l >> 4) on
  const int r0 = m0 + wm + (lane & 15), c0 = n0 + wn + 4 * (lane >> 4);
  if constexpr (MODE == STATS) {
    const int groups = (cols + BN / 2 - 1) / (BN / 2), group = (n0 + wn) / (BN / 2);
#pragma unroll
    for (int i = 0; i < TM; ++i) {
      const int t = r0 + i * 16;
      float m = -__builtin_inff(), s = 0.0f;
#pragma unroll
      for (int j = 0; j < TN; ++j)
#pragma unroll
        for (int v = 0; v < 4; ++v)
          if (c0 + j * 16 + v < cols) m = fmaxf(m, acc[i][j][v]);
      m = fmaxf(m, __shfl_xor(m, 16));
      m = fmaxf(m, __shfl_xor(m, 32));
      // all -inf: each term is exp(-inf), not exp(-inf + inf); a NaN stays one
      const float base = m == -__builtin_inff() ? 0.0f : m;
#pragma unroll
      for (int j = 0; j < TN; ++j)
#pragma unroll
        for (int v = 0; v < 4; ++v)
          if (c0 + j * 16 + v < cols) s += exp_of<F32>(acc[i][j][v] - base);
      s += __shfl_xor(s, 16);
      s += __shfl_xor(s, 32);
      if (t >= rows || group >= groups) continue;
      if (lane < 16) a.part[(long long)t * a.groups + a.group0 + group] = float2{m, s};
      const long long target = a.target[t];
#pragma unroll
      for (int j = 0; j < TN; ++j)
#pragma unroll
        for (int v = 0; v < 4; ++v)
          if ((long long)a.v0 + c0 + j * 16 + v == target && c0 + j * 16 + v < cols) a.zt[t] = acc[i][j][v];
    }
  } else if constexpr (MODE == GRAD) {
#pragma unroll
    for (int i = 0; i < TM; ++i) {
      const int t = r0 + i * 16;
      if (t >= rows) continue;
      const Row r = token_of(a, t);
#pragma unroll
      for (int j = 0; j < TN; ++j) {
        const int c = c0 + j * 16;
        if (c >= cols) continue;
        float d[4];
#pragma unroll
        for (int v = 0; v < 4; ++v) d[v] = grad_of<F32>(r, acc[i][j][v], (long long)a.v0 + c + v);
        put<F32>(a.dS, t * a.ldp + c, d, cols - c);
        if (!F32 && a.Td > a.T) {
#pragma unroll
          for (int v = 0; v < 4; ++v) d[v] -= (float)static_cast<__bf16>(d[v]);
          put<F32>(a.dS, (t + a.T) * a.ldp + c, d, cols - c);
        }
      }
    }
  } else {
    const float scale = scale_of(a);
#pragma unroll
    for (int i = 0; i < TM; ++i) {
      const int t = r0 + i * 16;
      if (t >= rows) continue;
#pragma unroll
      for (int j = 0; j < TN; ++j) {
        const int c = c0 + j * 16;
        if (c >= cols) continue;
        float o[4];
        if (MODE == DX && a.acc) {
          float4* const to = reinterpret_cast<float4*>(a.acc + ((long long)share * a.Td + t) * a.lda + c);
          float4 v = {acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3]};
          if (a.v0 > 0) {
            const float4 b = *to;
            v = float4{v.x + b.x, v.y + b.y, v.z + b.z, v.w + b.w};
          }
          *to = v;
          continue;
        }
#pragma unroll
        for (int v = 0; v < 4; ++v) o[v] = acc[i][j][v] * scale;
        if constexpr (MODE == DX) put<F32>(a.GX, t * a.ldgx + c, o, cols - c);
        else put<F32>(a.GW, (long long)(a.v0 + t) * a.ldgw + c, o, cols - c);
      }
    }
  }
}

}  // namespace vocab
}  // namespace poetx
