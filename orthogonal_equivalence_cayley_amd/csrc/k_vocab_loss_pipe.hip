// The products of the vocabulary's cross entropy (k_vocab_loss.hip) for many tokens in
// bf16: logits with each row's statistics (STATS) or with dL/dz (GRAD) as the epilogue,
// d W (DX) and d^T X (DW). 256 x 256 output tiles by one workgroup to a CU, eight waves of
// 128 x 64 each and one uninterrupted load pipeline over a range of tiles, as in the
// merged-weight product (k_linear_pipe.hip), whose order of loads, barriers and products
// this is: waves 0-3 issue all loads, direct to LDS, the A tile of stage s + 2 behind the
// barrier that frees its buffer, its B tile in halves during stage s + 1; waves 4-7 only
// multiply.
//
// An operand whose rows run across the summed axis (W in d W, both in d^T X) is staged as
// 64 summed rows of 256 columns and read by the transposing LDS read, so nothing is
// transposed in memory: chunk c (16 bytes) of summed row k sits at 32 k + (c ^ 4 (k & 3)),
// and the four rows by 64 bytes that half a wave reads fall in distinct banks.
//
// A last tile that would pass the last row or column is moved back to end there, so that
// every load is inside its operand; what it shares with its neighbour is left to that one.
// Requirements (vocab_pipe_logits and the like): at least one tile of each axis, n a multiple
// of 8, 16-byte rows of X and W.
//
// Bound by the matrix units at the clock that they leave (1.65 to 1.9 GHz), busy for 0.65 to
// 0.79 of the time: 16384 x 2048 x 32000 STATS 1552 us (1380 TFLOP/s), and of 8192 columns GRAD
// 438 (1255), DX 427 (1287), DW 412 (1334).
#include <algorithm>
#include <type_traits>

#include "linear_common.h"
#include "vocab_loss.h"

namespace poetx {
namespace {

using namespace lin;
using namespace vocab;

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short i16x4 __attribute__((ext_vector_type(4)));
typedef short i16x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4), aligned(2)));   // at any element alignment

constexpr int kTile = 256;
constexpr int kThr = 512;
constexpr int kKB = 128;                   // bytes of the summed axis per stage
constexpr int kKE = kKB / 2;               // elements
constexpr int kOp = kTile * kKB;           // bytes of one operand tile
constexpr int kStage = 2 * kOp;
constexpr int kLds = 2 * kStage;
constexpr int kSteps = kKB / 32;
constexpr int kLoads = kTile / 32;         // loads of a lane per operand tile, 4 KB of it each
constexpr int kGroupRows = 4;              // tile-rows per group of the XCD-aware order

// exp(z - m) = 2^(z k - base) corr over the z of a row, one rounding of the exponent: k =
// log2 e, base = m k rounded, and corr = 2^(base - m k) gives back what that lost (2^-12 of the
// exponent, 2e-4 of every term, at m = 4000). Past 2^120, where m k would overflow, two z that
// differ differ by 2^96 and more, so any k will do, and m / 2 is exact.
struct Base {
  float k, base, lost;   // lost: m k - base
};
__device__ __forceinline__ Base base_of(float m) {
  Base b;
  const bool far = fabsf(m) > 0x1p120f;   // infinities too
  b.k = far ? 0.5f : 1.44269504088896340736f;
  b.base = m * b.k;
  b.lost = far ? 0.0f : fmaf(m, b.k, -b.base);
  return b;
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __bf16 a = static_cast<__bf16>(lo), b = static_cast<__bf16>(hi);
  return (uint32_t)__builtin_bit_cast(uint16_t, a) | ((uint32_t)__builtin_bit_cast(uint16_t, b) << 16);
}
// Swaps the upper half of a with the lower half of b
__device__ __forceinline__ void swap_halves(float& a, float& b) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(a), __float_as_uint(b), false, false);
  const uint32_t r0 = r[0], r1 = r[1];
  a = __uint_as_float(r0);
  b = __uint_as_float(r1);
}

// How the lanes load and read an operand tile whose rows run along the summed axis, or
// (ACROSS) across it. `w0`: the wave's first row of it.
template <bool ACROSS>
struct Side;
template <>
struct Side<false> {
  uint32_t base;
  __device__ __forceinline__ void init(int w0, int lane) {
    // chunk c of row r at slot 8 r + (c ^ ((r / 2) & 7)): a step's address is base ^ (step << 5)
    const int r = w0 + (lane & 31), sw = (r / 2) & 7;
    base = (uint32_t)(16 * (r * 8 + ((lane >> 5) ^ (sw & 1)) + 2 * (sw >> 1)));
  }
  __device__ __forceinline__ i32x4 frag(const unsigned char* st, int i, int step) const {
    return *reinterpret_cast<const i32x4*>(st + ((base ^ (uint32_t)(step << 5)) + i * 32 * kKB));
  }
  static __device__ __forceinline__ uint32_t lane_offset(int g, int ld) {
    const int lr = g / 8;
    return (uint32_t)(lr * ld) + (uint32_t)((g & 7) ^ ((lr / 2) & 7)) * 16;
  }
};
template <>
struct Side<true> {
  uint32_t at[4];
  __device__ __forceinline__ void init(int w0, int lane) {
    // 16 lanes read a 4 x 16 block, lane s its 8 bytes of summed row s / 4, and get column s
    const int s = lane & 15, x = s >> 2, col = w0 + (lane >> 4 & 1) * 16 + 4 * (s & 3);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      at[i] = (uint32_t)((8 * (lane >> 5) + x) * 512 + (((col + 32 * i) >> 3) ^ (4 * x)) * 16 + (col & 7) * 2);
  }
  __device__ __forceinline__ i32x4 frag(const unsigned char* st, int i, int step) const {
    const unsigned char* p = st + at[i] + step * 16 * 512;
    const i16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) i16x4*)(p));
    const i16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) i16x4*)(p + 4 * 512));
    const i16x8 v = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    return __builtin_bit_cast(i32x4, v);
  }
  static __device__ __forceinline__ uint32_t lane_offset(int g, int ld) {
    const int k = g >> 5;
    return (uint32_t)(k * ld) + (uint32_t)((g & 31) ^ (4 * (k & 3))) * 16;
  }
};

// TAIL: the last stage of a sum is cut, for n (STATS, GRAD) or the piece of the vocabulary
// (DX) is no multiple of 64 (a branch around the loads parts the products from the reads
// beside them, so it has its own kernel)
// What workgroup `block` of `blocks` does of a product
template <Mode MODE, bool TAIL>
__device__ __forceinline__ void vocab_pipe(const VocabArgs& p, int block, int blocks) {
  constexpr bool AX = MODE == DW, BX = MODE == DX || MODE == DW;   // across the summed axis
  extern __shared__ __align__(16) unsigned char lds[];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm0 = (wave >> 2) * 128, wn0 = (wave & 3) * 64;
  const int cm = lane & 31, half = lane >> 5;

  // The operands: rows along the result's rows and columns, and the summed axis. Of d,
  // columns up to a multiple of 64 exist (zeros behind the piece's last).
  const int vz = (p.vp + 63) / 64 * 64;
  const int rows = MODE == DW ? vz : (int)(MODE == DX ? p.Td : p.T);
  const int cols = MODE == STATS || MODE == GRAD ? p.vp : MODE == DX ? p.n : (int)p.ldm;
  const int sum = MODE == DX ? vz : MODE == DW ? (int)p.Tm : p.n;
  const char* const a_base = static_cast<const char*>(MODE == STATS || MODE == GRAD ? p.X : p.dS);
  const char* const b_base =
      MODE == DW ? static_cast<const char*>(p.Xm) : static_cast<const char*>(p.W) + (long long)p.v0 * p.ldw * 2;
  const int lda = (int)((MODE == STATS || MODE == GRAD ? p.ldx : p.ldp) * 2);   // bytes, 256 of them below 2^31
  const int ldb = (int)((MODE == DW ? p.ldm : p.ldw) * 2);
  // DX of few tiles: p.splits workgroups share the sum of one, `per` stages each
  const int nk_all = (sum + kKE - 1) / kKE;
  const int per = MODE == DX ? (nk_all + p.splits - 1) / p.splits : nk_all;
  const int shares = MODE == DX ? (nk_all + per - 1) / per : 1;

  // XCD x = block % 8 owns the tiles [ntile x / 8, ntile (x + 1) / 8), walked by its
  // workgroups with a stride of their count, in groups of kGroupRows tile-rows
  const int tn = (cols + kTile - 1) / kTile, tm = (rows + kTile - 1) / kTile;
  const int ntile = tn * tm * shares;
  const int x = block % 8, sx = block / 8;
  const int nx = blocks / 8 + (x < blocks % 8 ? 1 : 0);
  const int t_first = (int)((long long)ntile * x / 8) + sx, t_end = (int)((long long)ntile * (x + 1) / 8);
  const int t_count = t_first < t_end ? (t_end - t_first + nx - 1) / nx : 0;
  if (t_count == 0) return;
  auto share = [&](int ti) { return MODE == DX ? __builtin_amdgcn_readfirstlane((t_first + ti * nx) / (tn * tm)) : 0; };
  auto origin = [&](int ti, int& m0, int& n0) {
    const int lin = t_first + ti * nx - share(ti) * (tn * tm);
    const int grp = lin / (kGroupRows * tn);
    const int first = grp * kGroupRows;
    const int gsz = min(kGroupRows, tm - first);
    const int in = lin - grp * (kGroupRows * tn);
    m0 = __builtin_amdgcn_readfirstlane((first + in % gsz) * kTile);
    n0 = __builtin_amdgcn_readfirstlane((in / gsz) * kTile);
  };

  const int g = tid & 255;   // thread of the loading waves
  const uint32_t lds_at = __builtin_amdgcn_readfirstlane(
      (uint32_t)(uintptr_t)(__attribute__((address_space(3))) unsigned char*)lds);
  const uint32_t va = Side<AX>::lane_offset(g, lda), vb = Side<BX>::lane_offset(g, ldb);

  // Where the loads of one operand stand: the stage's tile and its piece of the sum. Past
  // the last stage they repeat it, into buffers nobody reads.
  struct Cursor {
    int ti, kt, end, row;
  };
  auto row_of = [&](int ti, int op) {
    int m0, n0;
    origin(ti, m0, n0);
    return op == 0 ? min(m0, rows - kTile) : min(n0, cols - kTile);
  };
  auto advance = [&](Cursor& c, int op) {
    if (c.kt + 1 < c.end) {
      ++c.kt;
    } else if (c.ti + 1 < t_count) {
      c.row = row_of(++c.ti, op);
      c.kt = share(c.ti) * per;
      c.end = min(c.kt + per, nk_all);
    }
  };
  auto start = [&](int op) { return Cursor{0, share(0) * per, min(share(0) * per + per, nk_all), row_of(0, op)}; };
  // TAIL along n: chunks behind the last column. Their lanes load the stage's first chunk of
  // the row instead, and write zeros over it once it landed
  const uint32_t lc = (uint32_t)((g & 7) ^ ((g / 16) & 7)) * 16;
  constexpr bool CUT = TAIL && !BX;
  auto gone = [&](int kt) { return kt * kKE + (int)lc / 2 >= sum; };
  auto clear = [&](int buf) __attribute__((always_inline)) {
    if (!gone(nk_all - 1)) return;
#pragma unroll
    for (int i = 0; i < 2 * kLoads; ++i)
      *reinterpret_cast<i32x4*>(lds + buf * kStage + i * 4096 + g * 16) = i32x4{0, 0, 0, 0};
  };
  // loads [i0, i1) of operand op (0: A, 1: B) of the cursor's stage into buffer buf
  auto issue = [&](const Cursor& c, int op, int buf, int i0, int i1) __attribute__((always_inline)) {
    const uint32_t st = lds_at + (uint32_t)(buf * kStage + op * kOp + (wave & 3) * 64 * 16);
    const bool across = op == 0 ? AX : BX;
    const int ld = op == 0 ? lda : ldb;
    const char* base = (op == 0 ? a_base : b_base) +
                       (across ? (long long)c.kt * kKE * ld + c.row * 2LL : c.row * (long long)ld);
    // W ends with the vocabulary: behind its last row the last one is loaded again, for d is zero there
    const int there = TAIL && BX && op == 1 ? p.vp - c.kt * kKE : kKE;
    const uint32_t bytes = (uint32_t)(across ? (min(there, kKE) - 1) * ld + kTile * 2 : kTile * ld);
    const int k = across ? 0 : c.kt * kKB, step = across ? 8 * ld : 32 * ld;
    if (TAIL && BX && op == 1 && there < kKE) {
#pragma unroll
      for (int i = i0; i < i1; ++i) {
        const int kr = g >> 5, row = min(kr + 8 * i, there - 1);
        load_lds<BX>(base, bytes, st + i * 256 * 16, (uint32_t)(row * ld) + (uint32_t)((g & 31) ^ (4 * (kr & 3))) * 16, 0);
      }
      return;
    }
    const uint32_t off = (op == 0 ? va : vb) - (CUT && gone(c.kt) ? lc : 0);
#pragma unroll
    for (int i = i0; i < i1; ++i) load_lds<BX>(base, bytes, st + i * 256 * 16, off, (uint32_t)(k + i * step));
  };

  Side<AX> sa;
  Side<BX> sb;
  sa.init(wm0, lane);
  sb.init(wn0, lane);

  // Lane l holds row l & 31, columns 8 q + 4 (l >> 5) .. + 3 of each 32 x 32 tile.
  typedef f32x16 Acc;
  // m0, n0: where the tile lies; m1, n1: the first row and column that are its own
  auto stats = [&](Acc (&acc)[4][2], int m0, int n0, int m1, int n1) __attribute__((always_inline)) {
    const int group = n1 / 64 + (wave & 3);
    const bool whole = n0 == n1;
    float2 out[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int t = m0 + wm0 + i * 32 + cm;
      const long long target = p.target[t];
      if (!whole) {
        // columns of the neighbour's
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int v = 0; v < 16; ++v)
            if (n0 + wn0 + j * 32 + 8 * (v >> 2) + 4 * half + (v & 3) < n1) acc[i][j][v] = -__builtin_inff();
      }
      float m = acc[i][0][0];
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int v = 0; v < 16; ++v) m = fmaxf(m, acc[i][j][v]);
      m = fmaxf(m, __shfl_xor(m, 32));
      // all -inf: each term is exp(-inf), not exp(-inf + inf); a NaN stays one
      const Base b = base_of(m == -__builtin_inff() ? 0.0f : m);
      float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int v = 0; v < 16; ++v) s[v & 3] += __builtin_amdgcn_exp2f(fmaf(acc[i][j][v], b.k, -b.base));
      float sum_ = ((s[0] + s[1]) + (s[2] + s[3])) * __builtin_amdgcn_exp2f(-b.lost);
      sum_ += __shfl_xor(sum_, 32);
      out[i] = float2{m, sum_};
      const long long at = target - (n0 + wn0) - 4 * half;
      const bool mine = t >= m1 && target >= n1 && target < p.vp && at >= 0 && at < 64 && (at & 4) == 0;
      if (__any(mine)) {
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int v = 0; v < 16; ++v)
            if (mine && at == j * 32 + 8 * (v >> 2) + (v & 3)) p.zt[t] = acc[i][j][v];
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int t = m0 + wm0 + i * 32 + cm;
      if (t >= m1 && half == 0) p.part[(long long)t * p.groups + group] = out[i];
    }
  };

  // 8 columns in a row of lane's row: two groups of four with their halves swapped
  auto eight = [&](Acc (&acc)[4][2], int i, int q, float (&v)[8]) __attribute__((always_inline)) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[e] = acc[i][q / 2][8 * (q & 1) + e];
      v[4 + e] = acc[i][q / 2][8 * (q & 1) + 4 + e];
      swap_halves(v[e], v[4 + e]);
    }
  };
  auto column = [&](int n0, int q) { return n0 + wn0 + q * 16 + 8 * half; };   // q = 2 j + h
  // bf16 columns [from, to) of the 8 at `y`
  auto store8 = [&](uint16_t* y, const u32x4& r, int from, int to) __attribute__((always_inline)) {
    if (from <= 0 && to >= 8) {
      *reinterpret_cast<u32x4*>(y) = r;
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (e >= from && e < to) y[e] = (uint16_t)(e & 1 ? r[e / 2] >> 16 : r[e / 2]);
    }
  };
  auto grad = [&](Acc (&acc)[4][2], int m0, int n0, int m1, int n1) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int t = m0 + wm0 + i * 32 + cm;
      const Row r = token_of(p, t);
      // (p - 1) g = (2^(z k - base) - 1 / corr) (corr g)
      const Base b = base_of(r.lse);
      const float one = __builtin_amdgcn_exp2f(b.lost), factor = __builtin_amdgcn_exp2f(-b.lost) * r.factor;
      const uint32_t keep = r.target < 0 && r.factor == 0.0f ? 0u : ~0u;   // an ignored row is zero whatever its logits are
      const long long at = r.target - p.v0 - (n0 + wn0) - 8 * half;
      const bool any = __any(at >= 0 && at < 64);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        float v[8];
        eight(acc, i, q, v);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = __builtin_amdgcn_exp2f(fmaf(v[e], b.k, -b.base));
        if (any) {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (at == q * 16 + e) v[e] -= one;
        }
        u32x4 o;
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] = pack2(v[2 * e] * factor, v[2 * e + 1] * factor) & keep;
        const int c = column(n0, q);
        if (t >= m1 && c + 8 > n1) store8(static_cast<uint16_t*>(p.dS) + t * p.ldp + c, o, n1 - c, 8);
        __builtin_amdgcn_sched_barrier(0);   // one group at a time: registers
      }
    }
  };
  const float scale = MODE == DX || MODE == DW ? scale_of(p) : 1.0f;
  auto dx = [&](Acc (&acc)[4][2], int m0, int n0, int m1, int n1, int ti) __attribute__((always_inline)) {
    const bool first = p.v0 == 0, last = p.v0 + p.vp == p.V && p.splits == 1;
    float* const sums = p.acc + share(ti) * p.Td * p.lda;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const long long t = (long long)m0 + wm0 + i * 32 + cm;
      f32x4 old[4][2];
#pragma unroll
      for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int k = 0; k < 2; ++k)
          old[q][k] = first ? f32x4{0.0f, 0.0f, 0.0f, 0.0f}
                            : *reinterpret_cast<const f32x4*>(sums + t * p.lda + column(n0, q) + 4 * k);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        float v[8];
        eight(acc, i, q, v);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] += old[q][e / 4][e & 3];
        const int c = column(n0, q);
        if (t < m1 || c < n1) continue;
        if (last) {
          u32x4 o;
#pragma unroll
          for (int e = 0; e < 4; ++e) o[e] = pack2(v[2 * e] * scale, v[2 * e + 1] * scale);
          store8(static_cast<uint16_t*>(p.GX) + t * p.ldgx + c, o, 0, 8);
        } else {
#pragma unroll
          for (int k = 0; k < 2; ++k)
            *reinterpret_cast<f32x4*>(sums + t * p.lda + c + 4 * k) =
                f32x4{v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]};
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  auto dw = [&](Acc (&acc)[4][2], int m0, int n0, int m1, int n1) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = m0 + wm0 + i * 32 + cm;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        float v[8];
        eight(acc, i, q, v);
        u32x4 o;
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] = pack2(v[2 * e] * scale, v[2 * e + 1] * scale);
        const int c = column(n0, q);
        if (r >= m1 && r < p.vp && c >= n1)
          store8(static_cast<uint16_t*>(p.GW) + ((long long)p.v0 + r) * p.ldgw + c, o, 0, p.n - c);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  };
  auto finish = [&](Acc (&acc)[4][2], int m0, int n0, int m1, int n1, int ti) __attribute__((always_inline)) {
    if constexpr (MODE == STATS) stats(acc, m0, n0, m1, n1);
    else if constexpr (MODE == GRAD) grad(acc, m0, n0, m1, n1);
    else if constexpr (MODE == DX) dx(acc, m0, n0, m1, n1, ti);
    else dw(acc, m0, n0, m1, n1);
  };

  auto run = [&](auto ld_tag) {
    constexpr bool LD = decltype(ld_tag)::value;
    Cursor ca{}, cw{};   // A stands two stages ahead, B one
    if constexpr (LD) {
      ca = start(0);
      cw = start(1);
      issue(ca, 0, 0, 0, kLoads);
      issue(cw, 1, 0, 0, kLoads);
      advance(ca, 0);
      advance(cw, 1);
      issue(ca, 0, 1, 0, kLoads);   // stage 1's A tile; its B tile goes out in stage 0's first steps
      advance(ca, 0);
      vm_wait<kLoads>();            // stage 0 landed
      if (CUT && nk_all == 1) clear(0);
    }
    lds_sync();
    i32x4 af[2][4], bf[2][2];
    auto read = [&](const unsigned char* st, int set, int step) __attribute__((always_inline)) {
#pragma unroll
      for (int i = 0; i < 4; ++i) af[set][i] = sa.frag(st, i, step);
#pragma unroll
      for (int j = 0; j < 2; ++j) bf[set][j] = sb.frag(st + kOp, j, step);
    };
    read(lds, 0, 0);

    int buf = 0;
    for (int ti = 0; ti < t_count; ++ti) {
      int m1, n1;
      origin(ti, m1, n1);
      const int m0 = min(m1, rows - kTile), n0 = min(n1, cols - kTile);
      Acc acc[4][2];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int v = 0; v < 16; ++v) acc[i][j][v] = 0;
      // The 8 products of a step, and one after another between them the next step's 6
      // fragments from `st` and the loads [i0, i1) of op's cursor, in just this order
      auto step = [&](int set, const unsigned char* next, int kk, const Cursor& c, int op, int into, int i0, int i1)
                      __attribute__((always_inline)) {
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const int i = q / 2, j = q & 1;
          acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, bf[set][j]),
                                                              __builtin_bit_cast(bf16x8, af[set][i]), acc[i][j], 0, 0, 0);
          if (q == 0) af[set ^ 1][0] = sa.frag(next, 0, kk);
          else if (q == 1) bf[set ^ 1][0] = sb.frag(next + kOp, 0, kk);
          else if (q == 2) bf[set ^ 1][1] = sb.frag(next + kOp, 1, kk);
          else if (q < 6) af[set ^ 1][q - 2] = sa.frag(next, q - 2, kk);
          if (i1 - i0 == 8) issue(c, op, into, q, q + 1);
          else if (i1 - i0 == 4 && (q & 1)) issue(c, op, into, i0 + q / 2, i0 + q / 2 + 1);
          __builtin_amdgcn_sched_barrier(0);
        }
      };
      const int nk = MODE == DX ? min(per, nk_all - share(ti) * per) : nk_all;
      for (int kt = 0; kt < nk; ++kt, buf ^= 1) {
        const unsigned char* st = lds + buf * kStage;
#pragma unroll
        for (int kk = 0; kk < kSteps; ++kk) {
          const int cb = kk & 1;
          if (kk + 1 < kSteps) {
            if (LD && kk < 2) step(cb, st, kk + 1, cw, 1, buf ^ 1, kk * (kLoads / 2), (kk + 1) * (kLoads / 2));
            else step(cb, st, kk + 1, cw, 1, 0, 0, 0);
          } else {
            // the next stage landed, and this one no longer read by anyone, once every
            // wave is past this barrier
            if constexpr (LD) {
              vm_wait<0>();
              if (CUT && (kt + 2 == nk || nk == 1)) clear(buf ^ 1);
            }
            lds_sync();
            step(cb, lds + (buf ^ 1) * kStage, 0, ca, 0, buf, 0, LD ? kLoads : 0);
            if constexpr (LD) {
              advance(ca, 0);
              advance(cw, 1);
            }
          }
        }
      }
      finish(acc, m0, n0, m1, n1, ti);
    }
  };
  if (wave < 4) run(std::true_type{});
  else run(std::false_type{});
  // the last iterations loaded the final stage again into buffers nobody reads: let those
  // writes land before the workgroup's LDS is released
  vm_wait<0>();
}

template <Mode MODE, bool TAIL>
__global__ __launch_bounds__(kThr) __attribute__((amdgpu_waves_per_eu(2, 2)))
void vocab_pipe_kernel(VocabArgs p) {
  vocab_pipe<MODE, TAIL>(p, (int)blockIdx.x, (int)gridDim.x);
}
// d W by the first `first` workgroups and d^T X by the others, where a launch of each would
// leave CUs idle
template <bool TAIL>
__global__ __launch_bounds__(kThr) __attribute__((amdgpu_waves_per_eu(2, 2)))
void vocab_pipe_both_kernel(VocabArgs p, int first) {
  if ((int)blockIdx.x < first) vocab_pipe<DX, TAIL>(p, (int)blockIdx.x, first);
  else vocab_pipe<DW, false>(p, (int)blockIdx.x - first, (int)gridDim.x - first);
}

// Tiles of a product, and workgroups for them: a multiple of 8, so that every XCD's range of
// tiles has its own
template <Mode MODE>
long long tiles_for(const VocabArgs& a) {
  const long long rows = MODE == DW ? (a.vp + 63) / 64 * 64 : MODE == DX ? a.Td : a.T;
  const long long cols = MODE == STATS || MODE == GRAD ? a.vp : MODE == DX ? a.n : a.ldm;
  return ((rows + kTile - 1) / kTile) * ((cols + kTile - 1) / kTile) * (MODE == DX ? a.splits : 1);
}
template <Mode MODE>
hipError_t launch(const VocabArgs& a, hipStream_t s) {
  const long long grid = std::min<long long>((tiles_for<MODE>(a) + 7) / 8 * 8, 256);
  const bool tail = MODE == DX ? a.vp % kKE != 0 : MODE != DW && a.n % kKE != 0;
  if (tail)
    hipLaunchKernelGGL((vocab_pipe_kernel<MODE, MODE != DW>), dim3((unsigned)grid), dim3(kThr), kLds, s, a);
  else
    hipLaunchKernelGGL((vocab_pipe_kernel<MODE, false>), dim3((unsigned)grid), dim3(kThr), kLds, s, a);
  return hipGetLastError();
}

bool aligned16(const void* p, long long ld) { return ((uintptr_t)p & 15) == 0 && ld % 8 == 0; }

}  // namespace

bool vocab_pipe_logits(const VocabArgs& a) {
  return a.T >= kTile && a.vp >= kTile && a.n % 8 == 0 && aligned16(a.X, a.ldx) && aligned16(a.W, a.ldw) &&
         a.ldx < (1 << 21) && a.ldw < (1 << 21);
}
bool vocab_pipe_dx(long long T, int n) { return T >= kTile && n >= kTile && n % 8 == 0; }
bool vocab_pipe_dw(const VocabArgs& a) { return a.vp > kTile - 64 && a.ldm >= kTile && a.ldp < (1 << 21); }

hipError_t launch_vocab_pipe_stats(const VocabArgs& a, hipStream_t s) { return launch<STATS>(a, s); }
hipError_t launch_vocab_pipe_grad(const VocabArgs& a, hipStream_t s) { return launch<GRAD>(a, s); }
hipError_t launch_vocab_pipe_dx(const VocabArgs& a, hipStream_t s) { return launch<DX>(a, s); }
hipError_t launch_vocab_pipe_dw(const VocabArgs& a, hipStream_t s) { return launch<DW>(a, s); }
hipError_t launch_vocab_pipe_both(const VocabArgs& a, hipStream_t s) {
  const unsigned first = (unsigned)((tiles_for<DX>(a) + 7) / 8 * 8), rest = (unsigned)((tiles_for<DW>(a) + 7) / 8 * 8);
  if (a.vp % kKE) hipLaunchKernelGGL((vocab_pipe_both_kernel<true>), dim3(first + rest), dim3(kThr), kLds, s, a, (int)first);
  else hipLaunchKernelGGL((vocab_pipe_both_kernel<false>), dim3(first + rest), dim3(kThr), kLds, s, a, (int)first);
  return hipGetLastError();
}

}  // namespace poetx
