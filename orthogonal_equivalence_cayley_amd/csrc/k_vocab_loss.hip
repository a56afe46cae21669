// The cross entropy of a vocabulary's product without its logits, forward and backward:
// which kernels a call takes, those for rows of any alignment, for few tokens, and the
// small ones around the products (k_vocab_loss_pipe.hip, k_vocab_loss_ring.hip: the
// products over rows of whole 16 bytes)
//
//   z_tv = sum_k x_tk w_vk,  lse_t = log sum_v exp(z_tv),  loss_t = lse_t - z_t,target
//   d_tv = g_t (exp(z_tv - lse_t) - [v = target]),  dX = d W,  dW = d^T X
//
// Forward (STATS): a tile of logits stays in registers, where each row's maximum and sum of
// exponentials over the tile's columns are taken; vocab_join_kernel joins them. Backward,
// in pieces of the vocabulary: the tile is multiplied again and left as d (GRAD; in the
// operands' type, which the products that follow take; d of a row sums to 0, so what its
// rounding to bf16 costs is of the size of the result's own), then d W is added into dX
// (DX; fp32 across pieces, one rounding at the end) and d^T X is the piece's dW (DW; d and
// the masked X are the call's own, so its rows are always whole 16 bytes).
//
// Tiles here as in linear_tile_kernel (k_linear.hip): four waves of BM/2 x BN/2, 128 bytes
// of the summed axis a stage, two LDS buffers, the next two stages under way in registers.
// W in d W, whose rows run along the other axis, is kept the way it comes, 128 bytes' worth
// of summed rows of BN columns, and read across: bf16 by the transposing LDS read, fp32 by
// words. Its rows are padded by 32 bytes (fp32 16) and every eight of them (bf16) by 128
// more, so that the rows a read takes together fall in distinct banks.
//
// 16384 x 2048 x 32000 bf16 with both gradients 6.76 ms: 1270 TFLOP/s over the four
// products, bound by the matrix units at the clock they hold.
#include <algorithm>
#include <cmath>

#include "linear_common.h"
#include "row_common.h"
#include "vocab_loss.h"

namespace poetx {
namespace {

using namespace lin;
using namespace vocab;

typedef short i16x4 __attribute__((ext_vector_type(4)));

constexpr int kThr = 256;

// An operand: R rows (of the result's axis) by KB bytes of the summed axis a stage
template <typename Ty, int R, int KB, bool ACROSS>
struct Operand;

// rows along the summed axis
template <typename Ty, int R, int KB>
struct Operand<Ty, R, KB, false> {
  static constexpr int CPR = KB / 16, RPL = kThr / CPR;   // chunks of a row, rows a load
  static constexpr int ES = Ty::kSize, L = R / RPL, BYTES = R * KB;
  static_assert(L * RPL == R, "whole loads");
  const char* p[L];
  __device__ __forceinline__ void init(const void* base, long long ld, int r0, int rows) {
#pragma unroll
    for (int i = 0; i < L; ++i)
      p[i] = static_cast<const char*>(base) + (long long)min(r0 + i * RPL + (int)threadIdx.x / CPR, rows - 1) * ld * ES;
  }
  // of the stage from element k0 on; zero from kend on
  __device__ __forceinline__ void fetch(i32x4 (&r)[L], int k0, int kend) const {
    const long long k = (long long)k0 * ES + (threadIdx.x % CPR) * 16, kb = (long long)kend * ES;
    if (k0 + KB / ES <= kend) {
#pragma unroll
      for (int i = 0; i < L; ++i) __builtin_memcpy(&r[i], p[i] + k, 16);
    } else {
#pragma unroll
      for (int i = 0; i < L; ++i) r[i] = load16<ES>(p[i], k, kb);
    }
  }
  static __device__ __forceinline__ int slot(int r, int c) { return r * CPR + (c ^ (CPR == 8 ? (r / 2) & 7 : r & (CPR - 1))); }
  static __device__ __forceinline__ void keep(char* st, const i32x4 (&r)[L]) {
#pragma unroll
    for (int i = 0; i < L; ++i)
      reinterpret_cast<i32x4*>(st)[slot(i * RPL + (int)threadIdx.x / CPR, (int)threadIdx.x % CPR)] = r[i];
  }
  // 16 bytes along the summed axis of row r + (lane & 15), chunk 4 q + (lane >> 4)
  static __device__ __forceinline__ i32x4 frag(const char* st, int r, int q, int lane) {
    return reinterpret_cast<const i32x4*>(st)[slot(r + (lane & 15), q * 4 + (lane >> 4))];
  }
};

// rows across it
template <typename Ty, int R, int KB>
struct Operand<Ty, R, KB, true> {
  static constexpr int ES = Ty::kSize, K = KB / ES;
  static constexpr int CPR = R * ES / 16, RPL = kThr / CPR, L = K / RPL;   // chunks of a summed row, summed rows a load
  static constexpr int PITCH = R * ES + (ES == 2 ? 32 : 16), BYTES = K * PITCH + (ES == 2 ? K / 8 * 128 : 0);
  static_assert(RPL * L == K, "whole loads");
  const char* p;   // the first summed row's first chunk of this thread
  long long ld, c, cb;
  bool whole;
  __device__ __forceinline__ void init(const void* base, long long ld_, int r0, int rows) {
    p = static_cast<const char*>(base);
    ld = ld_ * ES;
    c = (long long)r0 * ES + (threadIdx.x % CPR) * 16;
    cb = (long long)rows * ES;
    whole = r0 + R <= rows;
  }
  __device__ __forceinline__ void fetch(i32x4 (&r)[L], int k0, int kend) const {
    const int k = k0 + (int)threadIdx.x / CPR;
    if (whole && k0 + K <= kend) {
#pragma unroll
      for (int i = 0; i < L; ++i) __builtin_memcpy(&r[i], p + (long long)(k + i * RPL) * ld + c, 16);
    } else {
#pragma unroll
      for (int i = 0; i < L; ++i) {
        r[i] = i32x4{0, 0, 0, 0};
        if (k + i * RPL < kend && c < cb) r[i] = load16<ES>(p + (long long)(k + i * RPL) * ld, c, cb);
      }
    }
  }
  static __device__ __forceinline__ int at(int k) { return k * PITCH + (ES == 2 ? (k >> 3) * 128 : 0); }
  static __device__ __forceinline__ void keep(char* st, const i32x4 (&r)[L]) {
#pragma unroll
    for (int i = 0; i < L; ++i)
      *reinterpret_cast<i32x4*>(st + at((int)threadIdx.x / CPR + i * RPL) + ((int)threadIdx.x % CPR) * 16) = r[i];
  }
  static __device__ __forceinline__ i32x4 frag(const char* st, int r, int q, int lane) {
    if constexpr (ES == 2) {
      // 16 lanes read a 4 x 16 block, lane i its 8 bytes of summed row i / 4, and get column i
      const int k = 32 * q + 8 * (lane >> 4) + (lane >> 2 & 3), col = r + 4 * (lane & 3);
      typedef short i16x8 __attribute__((ext_vector_type(8)));
      const i16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
          (__attribute__((address_space(3))) i16x4*)(st + at(k) + col * 2));
      const i16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
          (__attribute__((address_space(3))) i16x4*)(st + at(k + 4) + col * 2));
      const i16x8 v = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
      return __builtin_bit_cast(i32x4, v);
    } else {
      const int k = 16 * q + 4 * (lane >> 4), col = r + (lane & 15);
      i32x4 v;
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = *reinterpret_cast<const int*>(st + at(k + i) + col * 4);
      return v;
    }
  }
};

// Bytes of the summed axis a stage: twice as many for the smallest tiles, which leave the
// memory too few loads otherwise (16 tokens, 32000 x 2048 36.4 -> 35.6 us, 3000 x 512 15.6 ->
// 13.1)
constexpr int stage_bytes(int bm) { return bm == 32 ? 256 : 128; }
template <typename Ty, int BM, int BN, Mode M>
struct Tile {
  static constexpr int KB = stage_bytes(BM);
  using A = Operand<Ty, BM, KB, false>;
  using B = Operand<Ty, BN, KB, M == DX>;
  static constexpr int STAGE = A::BYTES + B::BYTES;
  static_assert(STAGE % 16 == 0 && A::BYTES % 16 == 0, "16-byte pieces");
};

template <typename Ty, int BM, int BN, Mode MODE>
__global__ __launch_bounds__(kThr) __attribute__((amdgpu_waves_per_eu(2, 2)))
void vocab_tile_kernel(VocabArgs a) {
  using Cfg = Tile<Ty, BM, BN, MODE>;
  using OA = typename Cfg::A;
  using OB = typename Cfg::B;
  constexpr int KE = Cfg::KB / Ty::kSize;      // elements of the summed axis a stage
  constexpr int Q = Cfg::KB / 64;              // 64-byte slabs of it
  constexpr int TM = BM / 32, TN = BN / 32;    // 16 x 16 tiles of a wave
  extern __shared__ __align__(16) char lds[];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int wm = (wave >> 1) * (BM / 2), wn = (wave & 1) * (BN / 2);
  const int rows = (int)(MODE == DX ? a.Td : a.T), cols = MODE == DX ? a.n : a.vp;
  int m0, n0;
  if (!tile_origin(rows, cols, BM, BN, m0, n0)) return;
  int k0 = 0, kend = MODE == DX ? a.vp : a.n;
  if (MODE == DX && a.splits > 1) {
    const int per = ((kend + a.splits - 1) / a.splits + KE - 1) / KE * KE;
    k0 = min(kend, (int)blockIdx.y * per);
    kend = min(kend, k0 + per);
  }
  const char* const w = static_cast<const char*>(a.W) + (long long)a.v0 * a.ldw * Ty::kSize;
  OA oa;
  OB ob;
  if constexpr (MODE == DX) oa.init(a.dS, a.ldp, m0, rows);
  else oa.init(a.X, a.ldx, m0, rows);
  ob.init(w, a.ldw, n0, cols);
  i32x4 ar[2][OA::L], br[2][OB::L];   // two stages under way
  auto fetch = [&](int k, int set) __attribute__((always_inline)) {
    oa.fetch(ar[set], k, kend);
    ob.fetch(br[set], k, kend);
  };
  auto keep = [&](int buf, int set) __attribute__((always_inline)) {
    OA::keep(lds + buf * Cfg::STAGE, ar[set]);
    OB::keep(lds + buf * Cfg::STAGE + OA::BYTES, br[set]);
  };
  typename Ty::Acc acc[TM][TN] = {};
  i32x4 af[2][TM], bf[2][TN];
  auto read = [&](int buf, int q) __attribute__((always_inline)) {
    const char* const st = lds + buf * Cfg::STAGE;
#pragma unroll
    for (int i = 0; i < TM; ++i) af[q & 1][i] = OA::frag(st, wm + i * 16, q, lane);
#pragma unroll
    for (int j = 0; j < TN; ++j) bf[q & 1][j] = OB::frag(st + OA::BYTES, wn + j * 16, q, lane);
  };
  auto multiply = [&](int q) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j) Ty::mma(bf[q & 1][j], af[q & 1][i], acc[i][j]);
  };
  const int stages = (kend - k0 + KE - 1) / KE;
  if (stages > 0) {
    fetch(k0, 0);
    keep(0, 0);
    if (stages > 1) fetch(k0 + KE, 1);
    if (stages > 2) fetch(k0 + 2 * KE, 0);
    lds_sync();
    read(0, 0);
    auto stage = [&](int s, int buf) __attribute__((always_inline)) {
      // nobody reads the other buffer since the barrier of the stage before
      if (s + 1 < stages) keep(buf ^ 1, buf ^ 1);
      if (s + 3 < stages) fetch(k0 + (s + 3) * KE, buf ^ 1);
#pragma unroll
      for (int q = 0; q < Q; ++q) {
        if (q + 1 < Q) {
          read(buf, q + 1);
        } else {
          lds_sync();
          if (s + 1 < stages) read(buf ^ 1, 0);
        }
        multiply(q);
      }
    };
    for (int s = 0; s < stages; s += 2) {
      stage(s, 0);
      if (s + 1 < stages) stage(s + 1, 1);
    }
  }

  epilogue<Ty, BN, TM, TN, MODE>(a, acc, rows, cols, m0, n0, wm, wn, MODE == DX ? (int)blockIdx.y : 0);
}

// Forward for the fewest tokens, TT of them: every wave multiplies kFewRows rows of W by all
// of X on the vector units, 32 rows to a workgroup and its part. Bound by W's bytes: one
// token, 32000 rows of 2048 bf16 that no cache holds 29 us with the join (5.3 TB/s in this
// kernel). The whole 32 KB of a wave's rows are asked for at once: half of them 33 us, four
// rows 30.5 us, four rows by halves 35 us. (Four tokens 41 us, in tiles 36.)
constexpr int kFew = 2, kFewRows = 8, kFewGroup = kThr / 64 * kFewRows;
template <typename Ty, int TT>
__global__ __launch_bounds__(kThr) void vocab_few_kernel(VocabArgs a) {
  constexpr bool F32 = Ty::kSize == 4;
  constexpr int R = kFewRows, U = 4;
  __shared__ float2 red[kThr / 64][TT];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int v0 = (int)blockIdx.x * kFewGroup + wave * R;
  const long long kb = (long long)a.n * Ty::kSize, k = lane * 16;
  const char *w[R], *x[TT];
#pragma unroll
  for (int r = 0; r < R; ++r)
    w[r] = static_cast<const char*>(a.W) + (long long)min(v0 + r, a.V - 1) * a.ldw * Ty::kSize;
#pragma unroll
  for (int t = 0; t < TT; ++t)
    x[t] = static_cast<const char*>(a.X) + min((long long)t, a.T - 1) * a.ldx * Ty::kSize;
  float z[R][TT] = {};
  long long p = 0;
  for (; p + 1024 * U <= kb; p += 1024 * U) {
    i32x4 wv[U][R], xv[U][TT];
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
      for (int r = 0; r < R; ++r) __builtin_memcpy(&wv[u][r], w[r] + p + k + u * 1024, 16);
#pragma unroll
      for (int t = 0; t < TT; ++t) __builtin_memcpy(&xv[u][t], x[t] + p + k + u * 1024, 16);
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int t = 0; t < TT; ++t) Ty::dot(wv[u][r], xv[u][t], z[r][t]);
  }
  for (; p < kb; p += 1024) {
    i32x4 wv[R], xv[TT];
#pragma unroll
    for (int r = 0; r < R; ++r) wv[r] = load16<Ty::kSize>(w[r], p + k, kb);
#pragma unroll
    for (int t = 0; t < TT; ++t) xv[t] = load16<Ty::kSize>(x[t], p + k, kb);
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int t = 0; t < TT; ++t) Ty::dot(wv[r], xv[t], z[r][t]);
  }
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int t = 0; t < TT; ++t)
#pragma unroll
      for (int o = 32; o > 0; o >>= 1) z[r][t] += __shfl_xor(z[r][t], o);
#pragma unroll
  for (int t = 0; t < TT; ++t) {
    float m = -__builtin_inff(), s = 0.0f;
#pragma unroll
    for (int r = 0; r < R; ++r)
      if (v0 + r < a.V) m = fmaxf(m, z[r][t]);
    const float base = m == -__builtin_inff() ? 0.0f : m;
#pragma unroll
    for (int r = 0; r < R; ++r)
      if (v0 + r < a.V) s += exp_of<F32>(z[r][t] - base);
    if (lane == 0) {
      red[wave][t] = float2{m, s};
      if (t < a.T) {
        const long long target = a.target[t];
#pragma unroll
        for (int r = 0; r < R; ++r)
          if (v0 + r == target && target < a.V) a.zt[t] = z[r][t];
      }
    }
  }
  __syncthreads();
  const int t = threadIdx.x;
  if (t >= TT || t >= a.T) return;
  float m = red[0][t].x, s = 0.0f;
#pragma unroll
  for (int i = 1; i < kThr / 64; ++i) m = fmaxf(m, red[i][t].x);
  const float base = m == -__builtin_inff() ? 0.0f : m;
  // an empty or all -inf part has s = 0 and adds 0 exp(-inf); one with a NaN keeps it
#pragma unroll
  for (int i = 0; i < kThr / 64; ++i) s += red[i][t].y * exp_of<F32>(red[i][t].x - base);
  a.part[t * (long long)gridDim.x + blockIdx.x] = float2{m, s};
}

// A row's lse and loss from the parts of its columns, by G lanes a row
template <int G>
__global__ __launch_bounds__(kThr) void vocab_join_kernel(VocabArgs a, int groups) {
  __shared__ float2 red[kThr / 64];
  const long long t = (long long)blockIdx.x * (kThr / G) + threadIdx.x / G;
  if (t >= a.T) return;   // whole workgroups where G = kThr
  const int lane = threadIdx.x % G;
  const float2* const p = a.part + t * groups;
  float m = -__builtin_inff();
  for (int i = lane; i < groups; i += G) m = fmaxf(m, p[i].x);
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor(m, o));
  if constexpr (G > 64) {
    if (threadIdx.x % 64 == 0) red[threadIdx.x / 64].x = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kThr / 64; ++i) m = fmaxf(m, red[i].x);
    __syncthreads();
  }
  // sums of up to 2^24 terms, in 64 bits
  double s = 0.0;
  const float base = m == -__builtin_inff() ? 0.0f : m;
  for (int i = lane; i < groups; i += G) s += (double)p[i].y * (double)expf(p[i].x - base);
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) s += __shfl_xor(s, o);
  if constexpr (G > 64) {
    double* const sums = reinterpret_cast<double*>(red);
    if (threadIdx.x % 64 == 0) sums[threadIdx.x / 64] = s;
    __syncthreads();
    s = sums[0];
#pragma unroll
    for (int i = 1; i < kThr / 64; ++i) s += sums[i];
  }
  if (lane != 0) return;
  const double lse = (double)base + log(s);
  const long long target = a.target[t];
  const bool ignored = target == a.ignore, bad = target < 0 || target >= a.V;
  a.lse_out[t] = (float)lse;
  a.loss[t] = ignored ? 0.0f : bad ? __builtin_nanf("") : (float)(lse - (double)a.zt[t]);
}

// Xm = X with zeros in ignored rows (a padded token's activations may be anything, and
// 0 times infinity would reach dW), once more below itself where d has two halves, columns
// up to ldm and rows up to a.Tm zero too; d's rows behind the last as well, and its columns from vp to a multiple of 64
template <typename E>
__global__ __launch_bounds__(kThr) void vocab_mask_kernel(VocabArgs a) {
  constexpr int N = 16 / sizeof(E);
  const int nv = (int)(a.ldm / N);
  for (long long t = blockIdx.x; t < a.Tm; t += gridDim.x) {
    const long long r = t < a.T ? t : t - a.T;
    const bool none = t >= a.Td || a.target[r] == a.ignore;
    const char* const from = static_cast<const char*>(a.X) + r * a.ldx * (long long)sizeof(E);
    E* const to = static_cast<E*>(a.Xm) + t * a.ldm;
    for (int c = threadIdx.x; c < nv; c += kThr) {
      i32x4 v = {0, 0, 0, 0};
      if (!none) v = load16<sizeof(E)>(from, (long long)c * 16, (long long)a.n * sizeof(E));
      reinterpret_cast<i32x4*>(to)[c] = v;
    }
    if (a.vp % 64 && t < a.Td && threadIdx.x < 64) {
      // behind a single piece's last column
      const int c = a.vp + (int)threadIdx.x;
      if (c < (a.vp + 63) / 64 * 64) static_cast<E*>(a.dS)[t * a.ldp + c] = E(0);
    }
    if (t >= a.Td) {
      i32x4* const d = reinterpret_cast<i32x4*>(static_cast<E*>(a.dS) + t * a.ldp);
      for (int c = threadIdx.x; c < (int)(a.ldp / N); c += kThr) d[c] = i32x4{0, 0, 0, 0};
    }
  }
}

// Zeros in d's columns from vp to a multiple of 64
template <typename E>
__global__ __launch_bounds__(kThr) void vocab_pad_kernel(VocabArgs a) {
  const int vz = (a.vp + 63) / 64 * 64;
  for (long long i = (long long)blockIdx.x * kThr + threadIdx.x; i < a.Td * 64; i += (long long)gridDim.x * kThr) {
    const int c = a.vp + (int)(i & 63);
    if (c < vz) static_cast<E*>(a.dS)[(i >> 6) * a.ldp + c] = E(0);
  }
}

// dX = round(factor * the sum of the splits' parts, and of both halves of d), G threads to 4
// columns of a row, each with every G-th part
template <bool F32, int G>
__global__ __launch_bounds__(kThr) void vocab_finish_kernel(VocabArgs a) {
  __shared__ float4 red[G][kThr / G];
  const int quads = (a.n + 3) / 4, lane = threadIdx.x % (kThr / G), grp = threadIdx.x / (kThr / G);
  const float scale = scale_of(a);
  const long long count = a.T * quads;
  const int halves = a.Td > a.T ? 2 : 1, parts = a.splits * halves;
  for (long long i0 = (long long)blockIdx.x * (kThr / G); i0 < count; i0 += (long long)gridDim.x * (kThr / G)) {
    const long long i = i0 + lane;
    const bool in = i < count;
    const long long t = in ? i / quads : 0;
    const int c = in ? (int)(i - t * quads) * 4 : 0;
    float4 v = {0.0f, 0.0f, 0.0f, 0.0f};
    if (in) {
#pragma unroll 4
      for (int z = grp; z < parts; z += G) {
        const long long row = (z / halves) * a.Td + t + (z % halves) * a.T;
        const float4 b = *reinterpret_cast<const float4*>(a.acc + row * a.lda + c);
        v = float4{v.x + b.x, v.y + b.y, v.z + b.z, v.w + b.w};
      }
    }
    if constexpr (G > 1) {
      red[grp][lane] = v;
      __syncthreads();
      if (grp == 0) {
#pragma unroll
        for (int k = 1; k < G; ++k) {
          const float4 b = red[k][lane];
          v = float4{v.x + b.x, v.y + b.y, v.z + b.z, v.w + b.w};
        }
      }
      __syncthreads();
    }
    if (grp == 0 && in) {
      const float o[4] = {v.x * scale, v.y * scale, v.z * scale, v.w * scale};
      put<F32>(a.GX, t * a.ldgx + c, o, a.n - c);
    }
  }
}
template <bool F32>
hipError_t finish(const VocabArgs& a, hipStream_t s) {
  const long long quads = a.T * ((a.n + 3) / 4);
  // few results of many parts leave the CUs idle otherwise (20 x 1001, 64 parts 20 -> 5 us)
  if (quads < 65536 && a.splits * (a.Td > a.T ? 2 : 1) >= 16) {
    const dim3 grid((unsigned)std::min<long long>((quads + 15) / 16, 1 << 16));
    hipLaunchKernelGGL((vocab_finish_kernel<F32, 16>), grid, dim3(kThr), 0, s, a);
  } else {
    const dim3 grid((unsigned)std::min<long long>((quads + kThr - 1) / kThr, 1 << 16));
    hipLaunchKernelGGL((vocab_finish_kernel<F32, 1>), grid, dim3(kThr), 0, s, a);
  }
  return hipGetLastError();
}

// d W and d^T X of the fewest fp32 tokens, at most TD, in one pass over W: a thread has 4
// columns of X in registers and goes down `per` rows of W, whose d are the same for all of its
// workgroup's; each chunk of rows leaves its part of dX. Bound by memory, W read and dW written
// (8 x 1024 x 32000 48 to 52 us, 5.0 TB/s; in tiles 98; rows of no whole 16 bytes 142 against 299).
// Not for bf16, whose d come in two halves, and for twice as many columns a thread: 4 x 2048 x
// 32000 134 us against 57 in tiles.
template <int TD>
__global__ __launch_bounds__(kThr) void vocab_outer_kernel(VocabArgs a, int per) {
  constexpr int N = 4, U = 4;   // U rows' loads out at a time
  constexpr int kRows = 64;     // of d in LDS at a time
  __shared__ __align__(16) float ds[kRows][TD];
  const int c = ((int)blockIdx.x * kThr + (int)threadIdx.x) * N, left = a.n - c;
  const bool in = left > 0;
  const int first = (int)blockIdx.y * per, end = min(first + per, a.vp);
  const float scale = scale_of(a);
  float x[TD][N] = {}, acc[TD][N] = {};
#pragma unroll
  for (int t = 0; t < TD; ++t)
    // a padded token's activations may be anything
    if (t < a.T && in && a.target[t] != a.ignore)
      row::load_raw<false>(static_cast<const float*>(a.X) + t * a.ldx + c, left, true, x[t]);
  const float* const w = static_cast<const float*>(a.W) + (long long)a.v0 * a.ldw + c;
  float* const gw = a.GW ? static_cast<float*>(a.GW) + (long long)a.v0 * a.ldgw + c : nullptr;
  for (int v0 = first; v0 < end; v0 += kRows) {
    const int rows = min(kRows, end - v0);
    __syncthreads();
    for (int i = threadIdx.x; i < kRows * TD; i += kThr) {
      const int t = i / kRows, v = i % kRows;
      ds[v][t] = t < a.T && v < rows ? static_cast<const float*>(a.dS)[t * a.ldp + v0 + v] : 0.0f;
    }
    __syncthreads();
    if (!in) continue;
    for (int v = 0; v < rows; v += U) {
      float wv[U][N] = {};
      if (a.GX) {
#pragma unroll
        for (int u = 0; u < U; ++u)
          row::load_raw<false>(w + (long long)(v0 + min(v + u, rows - 1)) * a.ldw, left, true, wv[u]);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (v + u >= rows) break;
        float o[N] = {};
#pragma unroll
        for (int t = 0; t < TD; ++t) {
          const float d = ds[v + u][t];
#pragma unroll
          for (int e = 0; e < N; ++e) {
            acc[t][e] = fmaf(d, wv[u][e], acc[t][e]);
            o[e] = fmaf(d, x[t][e], o[e]);
          }
        }
        if (gw) {
#pragma unroll
          for (int e = 0; e < N; ++e) o[e] *= scale;
          row::store_raw<false>(gw + (long long)(v0 + v + u) * a.ldgw, left, o);
        }
      }
    }
  }
  if (!a.GX || !in) return;
  float* const to = a.acc + (long long)blockIdx.y * a.Td * a.lda + c;
#pragma unroll
  for (int t = 0; t < TD; ++t) {
    if (t >= a.T) break;
    // whole vectors: lda is a multiple of 4
    float4* const at = reinterpret_cast<float4*>(to + t * a.lda);
    float4 v = {acc[t][0], acc[t][1], acc[t][2], acc[t][3]};
    if (a.v0 > 0) v = float4{v.x + at->x, v.y + at->y, v.z + at->z, v.w + at->w};
    *at = v;
  }
}
hipError_t outer(const VocabArgs& a, const VocabBackPlan& p, hipStream_t s) {
  const int per = (std::min<int>(p.vp, a.V) + p.chunks - 1) / p.chunks;
  const dim3 grid((unsigned)((a.n + kThr * 4 - 1) / (kThr * 4)), (unsigned)p.chunks);
  if (a.T <= 2) hipLaunchKernelGGL((vocab_outer_kernel<2>), grid, dim3(kThr), 0, s, a, per);
  else if (a.T <= 4) hipLaunchKernelGGL((vocab_outer_kernel<4>), grid, dim3(kThr), 0, s, a, per);
  else hipLaunchKernelGGL((vocab_outer_kernel<8>), grid, dim3(kThr), 0, s, a, per);
  return hipGetLastError();
}
// Tokens up to which, and columns from which, it is taken
constexpr int kOuter = 8, kOuterCols = 4 * kThr;

template <typename Ty, int TT>
hipError_t few(const VocabArgs& a, hipStream_t s) {
  hipLaunchKernelGGL((vocab_few_kernel<Ty, TT>), dim3((unsigned)((a.V + kFewGroup - 1) / kFewGroup)), dim3(kThr), 0, s, a);
  return hipGetLastError();
}
template <typename Ty>
hipError_t few(const VocabArgs& a, hipStream_t s) {
  return a.T == 1 ? few<Ty, 1>(a, s) : few<Ty, 2>(a, s);
}

hipError_t launch_pad(const VocabArgs& a, int bf16, hipStream_t s) {
  const dim3 grid((unsigned)std::min<long long>((a.Td + 3) / 4, 4096));
  if (bf16) hipLaunchKernelGGL((vocab_pad_kernel<uint16_t>), grid, dim3(kThr), 0, s, a);
  else hipLaunchKernelGGL((vocab_pad_kernel<float>), grid, dim3(kThr), 0, s, a);
  return hipGetLastError();
}

// V rows of n elements of zeros (4 or 2 bytes each)
template <typename E>
__global__ __launch_bounds__(kThr) void vocab_zero_kernel(E* p, int V, int n, long long ld) {
  for (long long v = blockIdx.x; v < V; v += gridDim.x)
    for (int c = threadIdx.x; c < n; c += kThr) p[v * ld + c] = E(0);
}

template <typename Ty, int BM, int BN, Mode M>
hipError_t tiles(const VocabArgs& a, hipStream_t s) {
  const int cols = M == DX ? a.n : a.vp;
  hipLaunchKernelGGL((vocab_tile_kernel<Ty, BM, BN, M>),
                     dim3((unsigned)tile_grid(M == DX ? a.Td : a.T, cols, BM, BN), M == DX ? (unsigned)a.splits : 1u), dim3(kThr),
                     (2 * Tile<Ty, BM, BN, M>::STAGE), s, a);
  return hipGetLastError();
}
template <typename Ty, Mode M>
hipError_t tiles(const VocabArgs& a, int tile, hipStream_t s) {
  switch (tile) {
    case VOCAB_TILE_128:
      if constexpr (Ty::kSize == 2) return tiles<Ty, 128, 128, M>(a, s);
      break;
    case VOCAB_TILE_128x64:
      // fp32: two workgroups to a CU, for one wave to a SIMD leaves its matrix unit idle
      if constexpr (Ty::kSize == 4) return tiles<Ty, 128, 64, M>(a, s);
      break;
    case VOCAB_TILE_64: return tiles<Ty, 64, 64, M>(a, s);
    case VOCAB_TILE_32x64: return tiles<Ty, 32, 64, M>(a, s);
  }
  return hipErrorInvalidValue;
}
template <Mode M>
hipError_t tiles(const VocabArgs& a, int bf16, int tile, hipStream_t s) {
  return bf16 ? tiles<TypeBf16, M>(a, tile, s) : tiles<TypeF32, M>(a, tile, s);
}

// How a product is laid out: its tile, and how many workgroups share the sum of one.
// What tiles take in us: for 32 stages of 128 bytes of the sum `first` in a grid of up to 256
// of them, one to a CU, and `round` for every 256 of a grid where the CUs are full; for the
// start and the epilogue `ends` for every 256. kRing, kRingF32: filled by direct-to-LDS loads
// (k_vocab_loss_ring.hip, k_vocab_loss_pipe.hip), the others through registers. Measured at
// 16 to 16384 tokens; e.g. logits of 1003 x 1000 x 10007 bf16 31 us in 256 x 256 tiles (said
// 35), 46 in 128 x 64 (said 43), of 256 x 2048 x 32000 60 in 256 x 256 (58), 50 in 128 x 128 (49).
struct TileCost {
  int tile, bm, bn;
  double first, round, ends;
};
constexpr TileCost kRing[] = {{VOCAB_TILE_256, 256, 256, 46, 46, 9}, {VOCAB_TILE_128, 128, 128, 24, 17, 6},
                              {VOCAB_TILE_128x64, 128, 64, 11, 9.5, 3.3}, {VOCAB_TILE_64, 64, 64, 6.5, 5.8, 1.7},
                              {VOCAB_TILE_32x64, 32, 64, 4.6, 4.3, 1.1}};
constexpr TileCost kRingF32[] = {{VOCAB_TILE_128x64, 128, 64, 33, 30, 4}, {VOCAB_TILE_64, 64, 64, 18, 16.5, 2.2},
                                 {VOCAB_TILE_32x64, 32, 64, 10, 9, 1.3}};
constexpr TileCost kTiles[] = {{VOCAB_TILE_128, 128, 128, 27, 22, 6}, {VOCAB_TILE_64, 64, 64, 24, 19, 2},
                               {VOCAB_TILE_32x64, 32, 64, 20, 15, 1.5}};
constexpr TileCost kTilesF32[] = {{VOCAB_TILE_128x64, 128, 64, 51, 42, 5}, {VOCAB_TILE_64, 64, 64, 32, 24, 2.5},
                                  {VOCAB_TILE_32x64, 32, 64, 25, 18, 2}};
// d W in the ring's tiles, whose loads and reads across the sum do not overlap as well, most
// of all for a workgroup alone on its CU: 1003 x 1000 x 10007 bf16 49 us in 256 tiles of 64 x
// 64, 35 + 5 in 512 shares of tiles of 128 x 64
constexpr double kAcrossFirst = 1.5, kAcrossRound = 1.1;

template <size_t N>
VocabTiles cheapest(const TileCost (&costs)[N], long long rows, long long cols, long long stages, bool wide, bool share) {
  VocabTiles best{-1, 1, 0.0};
  for (const TileCost& c : costs) {
    if (c.tile == VOCAB_TILE_256 && !wide) continue;
    const long long n = ((rows + c.bm - 1) / c.bm) * ((cols + c.bn - 1) / c.bn);
    for (int splits = 1; splits <= (share ? 64 : 1); splits *= 2) {
      const long long per = (stages + splits - 1) / splits, items = n * splits;
      if (splits > 1 && (per < 4 || items > 512)) break;
      // shares are written and read once more, by another launch
      const double extra = splits > 1 ? 3 + 1e-6 * (double)splits * (double)(rows * cols) : 0.0;
      const double rounds = (double)((items + 255) / 256);
      const bool across = share && c.tile != VOCAB_TILE_256;
      const double time = std::max(c.first * (across ? kAcrossFirst : 1.0), c.round * rounds * (across ? kAcrossRound : 1.0));
      const double cost = time * (double)per / 32 + c.ends * rounds + 3 + extra;
      if (best.tile < 0 || cost < best.cost) best = VocabTiles{c.tile, splits, cost};
    }
  }
  return best;
}
// fast: whether the operands' rows are whole 16 bytes; wide: whether 256 x 256 tiles may be taken
VocabTiles tiles_of(long long rows, long long cols, long long sum, int bf16, bool fast, bool wide, bool share = false) {
  const long long stages = (sum * (bf16 ? 2 : 4) + 127) / 128;
  if (fast) {
    return bf16 ? cheapest(kRing, rows, cols, stages, wide, share) : cheapest(kRingF32, rows, cols, stages, false, share);
  }
  return bf16 ? cheapest(kTiles, rows, cols, stages, false, share) : cheapest(kTilesF32, rows, cols, stages, false, share);
}
// Of a product's columns in 256 x 256 tiles those that make whole rounds of the CUs, where the
// others in smaller tiles (`rest`), a launch of their own, take less than one more round: 2048 x
// 4096 x 50021, 1568 tiles, 641 us, in one launch 681. All of them where not.
int whole_rounds(long long rows, int cols, int n, int& rest) {
  const long long tm = (rows + 255) / 256, tn = (cols + 255LL) / 256, full = tm * tn / 256 * 256 / tm;
  if (full < 1 || full >= tn) return cols;
  const int main = (int)full * 256;
  const long long stages = (2LL * n + 127) / 128;
  const TileCost& c = kRing[0];
  const double round = c.round * (double)stages / 32 + c.ends;
  const VocabTiles r = cheapest(kRing, rows, cols - main, stages, false, false);
  if ((double)((tm * full + 255) / 256) * round + 3 + r.cost >= (double)((tm * tn + 255) / 256) * round) return cols;
  rest = r.tile;
  return main;
}
int group_cols(int tile) { return tile == VOCAB_TILE_128 || tile == VOCAB_TILE_256 ? 64 : 32; }

// Parts of a row: 256-column tiles leave those of whole tiles
int groups_of(const VocabPlan& p, int tile, int V) {
  if (tile != VOCAB_TILE_256) return (V + group_cols(tile) - 1) / group_cols(tile);
  return (p.main + 255) / 256 * 4 + (p.main < V ? (V - p.main + group_cols(p.rest) - 1) / group_cols(p.rest) : 0);
}

// Up to this many tokens in bf16 the products take what d loses in rounding too, as rows of
// their own. It shows where tokens have factors of their own: a target's d, about -g, rounds by
// up to half a step, and a row of dX and one of dW with it. Both are off by 0.0024 of their
// 2-norm then, and by 0.0017 with the second rows, as rounding the results alone costs. (One
// factor is left out of d, whose targets are -1 or near it: 0.0017 at any size.) Why not past
// 64: to there memory bounds the products, and its traffic hardly grows (64 x 2048 x 32000
// backward 124 -> 131 us); from some hundred tokens on the matrix units do, and two of the
// three products would double. Nor can g go behind the sums of dX: dW takes the same d and
// would have to round g x instead, a third rounding of its terms.
constexpr long long kHalves = 64;

// Into how many shares the sum of d W goes where it and d^T X are one launch of 256 x 256
// tiles, one to a CU; 0 where one launch after the other is as fast, or their tiles are more
// than the CUs. 1003 x 1000 x 10007 bf16 55 us and 6 for joining the shares, one after the
// other 35 + 30 and 5; 2048 x 1024 x 8192 60 + 8 against 39 + 47 + 12, 300 x 512 x 5000 21 + 4
// against 9 + 13 + 3.
int shares_of_both(const VocabBackPlan& p, int vp, int n) {
  const long long tx = ((p.Td + 255) / 256) * ((n + 255) / 256), tw = ((vp + 255LL) / 256) * ((p.ldm + 255) / 256);
  const long long sx = (vp + 63) / 64, sw = p.Tm / 64, left = 256 - (tw + 7) / 8 * 8;
  const TileCost& c = kRing[0];
  double best = p.dx[1].cost + tiles_of(vp, n, p.Td, 1, true, true).cost;
  int shares = 0;
  for (int s = 1; s <= 64 && (tx * s + 7) / 8 * 8 <= left; ++s) {
    const long long per = (sx + s - 1) / s;
    if (s > 1 && per < 4) break;
    const double extra = s > 1 ? 3 + 1e-6 * (double)s * (double)(p.Td * n) : 0.0;
    const double cost = c.first * (double)std::max(per, sw) / 32 + c.ends + 3 + extra;
    if (cost < best) {
      best = cost;
      shares = (int)((sx + per - 1) / per);
    }
  }
  return shares;
}

constexpr long long kRoom = 256LL << 20;   // bytes that a part of the work may take as workspace
size_t padded(size_t b) { return (b + 255) / 256 * 256; }

}  // namespace

hipError_t launch_vocab_zero(void* p, int V, int n, long long ld, int es, hipStream_t s) {
  const dim3 grid((unsigned)std::min(V, 1 << 16));
  if (es == 4) hipLaunchKernelGGL((vocab_zero_kernel<uint32_t>), grid, dim3(kThr), 0, s, static_cast<uint32_t*>(p), V, n, ld);
  else hipLaunchKernelGGL((vocab_zero_kernel<uint16_t>), grid, dim3(kThr), 0, s, static_cast<uint16_t*>(p), V, n, ld);
  return hipGetLastError();
}

VocabPlan vocab_forward_plan(long long T, int V, int n, int bf16) {
  VocabPlan p{};
  // as the operands' alignment may lead: rows of whole 16 bytes or not
  p.lay[0] = tiles_of(T, V, n, bf16, false, false);
  p.lay[1] = tiles_of(T, V, n, bf16, true, false);
  p.lay[2] = tiles_of(T, V, n, bf16, true, bf16 && T >= 256 && V >= 256);
  p.groups = T <= kFew ? (V + kFewGroup - 1) / kFewGroup : 0;
  p.main = p.lay[2].tile == VOCAB_TILE_256 ? whole_rounds(T, V, n, p.rest) : V;
  for (const VocabTiles& l : p.lay) p.groups = std::max(p.groups, groups_of(p, l.tile, V));
  // tokens of a launch: as many as their parts leave room for, and their tiles can be counted
  const long long most = std::min(kRoom / (8LL * p.groups), (1LL << 33) / V);
  p.rows = std::min(T, std::max(256LL, most / 256 * 256));
  p.bytes = padded((size_t)p.rows * p.groups * 8) + padded((size_t)p.rows * 4);
  return p;
}

hipError_t launch_vocab_forward(const VocabArgs& in, int bf16, void* ws, hipStream_t s) {
  const VocabPlan p = vocab_forward_plan(in.T, in.V, in.n, bf16);
  const int es = bf16 ? 2 : 4;
  for (long long t = 0; t < in.T; t += p.rows) {
    VocabArgs a = in;
    a.T = std::min(p.rows, in.T - t);
    a.X = static_cast<const char*>(in.X) + t * in.ldx * es;
    a.target = in.target + t;
    a.loss = in.loss + t;
    a.lse_out = in.lse_out + t;
    a.part = static_cast<float2*>(ws);
    a.zt = reinterpret_cast<float*>(static_cast<char*>(ws) + padded((size_t)p.rows * p.groups * 8));
    a.v0 = 0;
    a.vp = a.V;
    const VocabTiles& lay = p.lay[!vocab_ring_logits(a, bf16) ? 0 : bf16 && vocab_pipe_logits(a) ? 2 : 1];
    int groups = groups_of(p, lay.tile, a.V);
    a.groups = groups;
    hipError_t e;
    if (in.T <= kFew) {
      groups = (a.V + kFewGroup - 1) / kFewGroup;
      e = bf16 ? few<TypeBf16>(a, s) : few<TypeF32>(a, s);
    } else if (lay.tile == VOCAB_TILE_256) {
      a.vp = p.main;
      e = launch_vocab_pipe_stats(a, s);
      if (e == hipSuccess && p.main < a.V) {
        VocabArgs b = a;
        b.v0 = p.main;
        b.vp = a.V - p.main;
        b.group0 = p.main / 64;
        e = launch_vocab_ring_stats(b, bf16, p.rest, s);
      }
    } else {
      e = &lay == &p.lay[0] ? tiles<STATS>(a, bf16, lay.tile, s) : launch_vocab_ring_stats(a, bf16, lay.tile, s);
    }
    if (e != hipSuccess) return e;
    if (a.T >= 1024)
      hipLaunchKernelGGL((vocab_join_kernel<64>), dim3((unsigned)((a.T + 3) / 4)), dim3(kThr), 0, s, a, groups);
    else
      hipLaunchKernelGGL((vocab_join_kernel<kThr>), dim3((unsigned)a.T), dim3(kThr), 0, s, a, groups);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

VocabBackPlan vocab_backward_plan(long long T, int V, int n, int bf16, bool gx, bool gw) {
  VocabBackPlan p{};
  const int es = bf16 ? 2 : 4;
  p.Td = bf16 && T <= kHalves ? 2 * T : T;
  p.Tm = (p.Td + 63) / 64 * 64;
  p.ldm = (n + 7) / 8 * 8;
  p.lda = (n + 3) / 4 * 4;
  // columns of a piece: those whose d leaves room, in whole tiles, the pieces alike
  const long long most = std::max(256LL, std::min({kRoom / (p.Tm * es), (1LL << 36) / n, 1LL << 19}) / 256 * 256);
  const long long pieces = (V + most - 1) / most;
  p.vp = (int)std::min<long long>(most, ((V + pieces - 1) / pieces + 255) / 256 * 256);
  const int vp = std::min(p.vp, V);
  const bool one = V <= p.vp;
  // as the operands' alignment may lead: rows of whole 16 bytes or not
  p.dx[0] = tiles_of(p.Td, n, vp, bf16, false, false, true);
  p.dx[1] = tiles_of(p.Td, n, vp, bf16, true, bf16 && vocab_pipe_dx(p.Td, n), true);
  // shares none of which is empty in the first piece (the others only add to theirs)
  for (VocabTiles& d : p.dx) {
    const long long stages = (long long)((vp + 63) / 64 * 64) * es / 128, per = (stages + d.splits - 1) / d.splits;
    d.splits = (int)((stages + per - 1) / per);
  }
  if (bf16 && gx && gw && one && vocab_pipe_dx(p.Td, n) && vp >= 256) p.both = shares_of_both(p, vp, n);
  int splits = std::max({p.dx[0].splits, p.dx[1].splits, p.both});
  p.outer = !bf16 && T <= kOuter && n >= kOuterCols;
  if (p.outer) {
    // enough workgroups, whose parts of dX stay an eighth of W
    const long long wide = (n + kOuterCols - 1) / kOuterCols;
    const long long want = std::max(1LL, std::min({2048 / wide, vp / (8 * T), (vp + 63LL) / 64}));
    const long long per = (vp + want - 1) / want;
    splits = p.chunks = (int)((vp + per - 1) / per);
  }
  p.acc = gx && (p.outer || splits > 1 || !one || p.Td > T);
  p.at_x = padded((size_t)p.Tm * p.vp * es);
  p.at_acc = p.at_x + (gw && !p.outer ? padded((size_t)p.Tm * p.ldm * es) : 0);
  p.bytes = p.at_acc + (p.acc ? padded((size_t)splits * p.Td * p.lda * 4) : 0);
  return p;
}

hipError_t launch_vocab_backward(const VocabArgs& in, int bf16, void* ws, hipStream_t s) {
  const VocabBackPlan p = vocab_backward_plan(in.T, in.V, in.n, bf16, in.GX != nullptr, in.GW != nullptr);
  VocabArgs a = in;
  a.dS = ws;
  a.ldp = p.vp;
  a.Xm = static_cast<char*>(ws) + p.at_x;
  a.ldm = p.ldm;
  a.Td = p.Td;
  a.Tm = p.Tm;
  a.lda = p.lda;
  const bool fast = vocab_ring_weight(a, bf16);
  const VocabTiles dx = p.dx[fast ? 1 : 0];
  const bool both = fast && p.both > 0, wide_dx = both || dx.tile == VOCAB_TILE_256;
  a.splits = p.outer ? p.chunks : both ? p.both : dx.splits;
  a.acc = p.outer || a.splits > 1 || a.V > p.vp || a.Td > a.T ? reinterpret_cast<float*>(static_cast<char*>(ws) + p.at_acc) : nullptr;
  hipError_t e;
  if (a.GW && !p.outer) {
    a.vp = a.V <= p.vp ? a.V : p.vp;
    const dim3 grid((unsigned)std::min<long long>(a.Tm, 1 << 16));
    if (bf16) hipLaunchKernelGGL((vocab_mask_kernel<uint16_t>), grid, dim3(kThr), 0, s, a);
    else hipLaunchKernelGGL((vocab_mask_kernel<float>), grid, dim3(kThr), 0, s, a);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  for (long long v = 0; v < a.V; v += p.vp) {
    a.v0 = (int)v;
    a.vp = (int)std::min<long long>(p.vp, a.V - v);
    const bool fast_logits = vocab_ring_logits(a, bf16);
    const VocabTiles grad = tiles_of(a.T, a.vp, a.n, bf16, fast_logits, bf16 && vocab_pipe_logits(a));
    if (grad.tile == VOCAB_TILE_256) {
      VocabArgs b = a;
      int rest = 0;
      b.vp = whole_rounds(a.T, a.vp, a.n, rest);
      e = launch_vocab_pipe_grad(b, s);
      if (e == hipSuccess && b.vp < a.vp) {
        b.v0 = a.v0 + b.vp;
        b.dS = static_cast<uint16_t*>(a.dS) + b.vp;
        b.vp = a.vp - b.vp;
        e = launch_vocab_ring_grad(b, bf16, rest, s);
      }
    } else {
      e = fast_logits ? launch_vocab_ring_grad(a, bf16, grad.tile, s) : tiles<GRAD>(a, bf16, grad.tile, s);
    }
    if (e != hipSuccess) return e;
    if (p.outer) {
      e = outer(a, p, s);
      if (e != hipSuccess) return e;
      continue;
    }
    if (both) {
      // (one piece: vocab_mask_kernel has written the zeros behind d)
      e = launch_vocab_pipe_both(a, s);
      if (e != hipSuccess) return e;
      continue;
    }
    if (a.GX) {
      if (fast && a.vp % 64 && (!a.GW || a.v0 > 0)) {
        e = launch_pad(a, bf16, s);
        if (e != hipSuccess) return e;
      }
      e = wide_dx ? launch_vocab_pipe_dx(a, s)
          : fast  ? launch_vocab_ring_dx(a, bf16, dx.tile, s)
                  : tiles<DX>(a, bf16, dx.tile, s);
      if (e != hipSuccess) return e;
    }
    if (a.GW) {
      // both operands are this call's own: their rows are whole 16 bytes
      const VocabTiles dw = tiles_of(a.vp, a.n, a.Td, bf16, true, bf16 && vocab_pipe_dw(a));
      e = dw.tile == VOCAB_TILE_256 ? launch_vocab_pipe_dw(a, s) : launch_vocab_ring_dw(a, bf16, dw.tile, s);
      if (e != hipSuccess) return e;
    }
  }
  // the last piece of an unshared dX in 256 x 256 tiles writes it whole
  if (!a.GX || !a.acc || (wide_dx && a.splits == 1 && !p.outer)) return hipSuccess;
  return bf16 ? finish<false>(a, s) : finish<true>(a, s);
}

}  // namespace poetx
