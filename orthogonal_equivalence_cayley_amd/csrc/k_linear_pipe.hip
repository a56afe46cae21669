// The merged-weight product (k_linear.hip) for many tokens: 256 x 256 output
// tiles, 8 waves (two per SIMD) of 128 x 64 each as 4 x 2 tiles of the 32 x 32
// matrix instruction, two LDS stages of 128 bytes of every operand row (128 KB),
// one workgroup per CU walking a contiguous, XCD-local range of tiles with one
// uninterrupted load pipeline. bf16 and INT8 rows move alike: a lane feeds the
// matrix unit 16 bytes of a 32-byte slab per step, whatever they hold.
//
// Waves 0-3 issue all loads (direct to LDS): the A tile of stage s + 2 right
// after the barrier that frees its buffer, its B tile in halves during the first
// two steps of stage s + 1. Waves 4-7 only read fragments and multiply, so the
// matrix units stay busy while the loads queue. Each step reads the next step's
// fragments between its own products.
//
// Bound by the matrix units at the clock they hold. 16384 tokens: 2048 to 5632 bf16
// SiLU 331 us (1140 TFLOP/s; a gating operand 20 to 30 us more, its reads in
// bursts between the tiles), 11008 to 4096 INT8 with residual 590 to 615 us (2.4 to
// 2.5 POPS); the vendor library's products alone 350 and 694 us. What it took:
// operands of the epilogue fetched a row tile ahead and all stores last (495 ->
// 387 us), tile numbers in 32 bits and marked uniform (387 -> 361; see origin).
//
// A last tile that would pass the last token or weight row is moved back to end
// there, so that every load is inside its operand; the rows and columns it shares
// with its neighbour are left to that one. Requirements (linear_pipe_supported):
// at least one tile of each, 128-byte multiples of n, m a multiple of 8, 16-byte
// rows of X and W, 256 rows of each below 2 GB.
#include <algorithm>
#include <type_traits>

#include "linear_common.h"

namespace poetx {
namespace {

using namespace lin;

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef int i32x16 __attribute__((ext_vector_type(16)));

constexpr int kTile = 256;
constexpr int kThr = 512;
constexpr int kKB = 128;                   // bytes of a row per stage
constexpr int kOp = kTile * kKB;           // bytes of one operand tile
constexpr int kStage = 2 * kOp;
constexpr int kLds = 2 * kStage + 2 * kTile * 4;
constexpr int kSteps = kKB / 32;
constexpr int kLoads = kTile / 32;         // loads of a lane per operand tile: 32 rows each
constexpr int kGroupRows = 4;              // tile-rows per group of the XCD-aware order

struct PipeBf16 {
  static constexpr int kSize = 2;
  typedef f32x16 Acc;
  typedef float Sum;
  static __device__ __forceinline__ Acc mma(const i32x4& a, const i32x4& b, const Acc& c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b),
                                                   c, 0, 0, 0);
  }
};
struct PipeI8 {
  static constexpr int kSize = 1;
  typedef i32x16 Acc;
  typedef int Sum;
  static __device__ __forceinline__ Acc mma(const i32x4& a, const i32x4& b, const Acc& c) {
    return __builtin_amdgcn_mfma_i32_32x32x32_i8(a, b, c, 0, 0, 0);
  }
};

typedef uint32_t u32x4 __attribute__((ext_vector_type(4), aligned(2)));   // at any element alignment

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __bf16 a = static_cast<__bf16>(lo), b = static_cast<__bf16>(hi);
  return (uint32_t)__builtin_bit_cast(uint16_t, a) | ((uint32_t)__builtin_bit_cast(uint16_t, b) << 16);
}
// Chunk c (16 bytes) of tile row r at slot 8 r + (c ^ ((r / 2) & 7)): the 16 rows
// a quarter of a wave reads at one chunk fall in distinct banks. The swizzle only
// permutes the chunk bits below a row's base, so a fragment's address is
// base ^ (step << 5) + 32 rows i.
__device__ __forceinline__ uint32_t frag_base(int r, int half) {
  const int sw = (r / 2) & 7;
  return (uint32_t)(16 * (r * 8 + (half ^ (sw & 1)) + 2 * (sw >> 1)));
}
__device__ __forceinline__ i32x4 frag(const unsigned char* st, uint32_t base, int i, int step) {
  return *reinterpret_cast<const i32x4*>(st + ((base ^ (uint32_t)(step << 5)) + i * 32 * kKB));
}

// Swaps the upper half of a with the lower half of b
template <typename S>
__device__ __forceinline__ void swap_halves(S& a, S& b) {
  const auto r = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b),
                                                  false, false);
  const uint32_t r0 = r[0], r1 = r[1];   // a bit_cast of r[1] itself reads r[0]
  a = __builtin_bit_cast(S, r0);
  b = __builtin_bit_cast(S, r1);
}

template <typename Ty, bool YBF16, int ACT>
__global__ __launch_bounds__(kThr) __attribute__((amdgpu_waves_per_eu(2, 2)))
void linear_pipe_kernel(LinearArgs p) {
  extern __shared__ __align__(16) unsigned char lds[];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm0 = (wave >> 2) * 128, wn0 = (wave & 3) * 64;

  // XCD x = blockIdx.x % 8 owns the tiles [ntile x / 8, ntile (x + 1) / 8), walked
  // by its workgroups with a stride of their count; a tile index maps to an origin
  // in groups of kGroupRows tile-rows
  const int tn = (p.m + kTile - 1) / kTile, tm = (int)((p.T + kTile - 1) / kTile);
  const int ntile = tn * tm;
  const int x = blockIdx.x % 8, sx = blockIdx.x / 8;
  const int nx = (int)gridDim.x / 8 + (x < (int)gridDim.x % 8 ? 1 : 0);
  const int t_first = (int)((long long)ntile * x / 8) + sx, t_end = (int)((long long)ntile * (x + 1) / 8);
  const int t_count = t_first < t_end ? (t_end - t_first + nx - 1) / nx : 0;
  if (t_count == 0) return;
  // 32-bit throughout, and told to be uniform: a 64-bit division leaves its result
  // in vector registers, and every load would loop over its lanes' descriptors
  auto origin = [&](int ti, int& m0, int& n0) {
    const int lin = t_first + ti * nx;
    const int grp = lin / (kGroupRows * tn);
    const int first = grp * kGroupRows;
    const int gsz = min(kGroupRows, tm - first);
    const int in = lin - grp * (kGroupRows * tn);
    m0 = __builtin_amdgcn_readfirstlane((first + in % gsz) * kTile);
    n0 = __builtin_amdgcn_readfirstlane((in / gsz) * kTile);
  };

  const int lda = (int)(p.ldx * Ty::kSize), ldb = (int)(p.ldw * Ty::kSize);   // bytes, 256 of them below 2^31
  const int g = tid & 255;                  // thread of the loading waves
  const int lr = g / 8;                     // its row among 32
  const uint32_t lc = (uint32_t)((g & 7) ^ ((lr / 2) & 7)) * 16;
  const uint32_t va = (uint32_t)(lr * lda) + lc, vb = (uint32_t)(lr * ldb) + lc;
  const int nk = (int)((long long)p.n * Ty::kSize / kKB);

  // Where the loads of one operand stand: the stage's tile and its piece of n.
  // Past the last stage they repeat it, into buffers nobody reads.
  struct Cursor {
    int ti, kt, row;
  };
  auto row_of = [&](int ti, int op) {
    int m0, n0;
    origin(ti, m0, n0);
    return op == 0 ? min(m0, (int)p.T - kTile) : min(n0, p.m - kTile);
  };
  auto advance = [&](Cursor& c, int op) {
    if (c.kt + 1 < nk) {
      ++c.kt;
    } else if (c.ti + 1 < t_count) {
      c.kt = 0;
      c.row = row_of(++c.ti, op);
    }
  };
  // loads [i0, i1) of operand op (0: X, 1: W) of the cursor's stage into buffer buf
  auto issue = [&](const Cursor& c, int op, int buf, int i0, int i1) {
    unsigned char* st = lds + buf * kStage + op * kOp + (wave & 3) * 64 * 16;
    const int ld = op == 0 ? lda : ldb;
    const char* base = static_cast<const char*>(op == 0 ? p.X : p.W) + c.row * (long long)ld;
    const __amdgpu_buffer_rsrc_t rs =
        __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(base), (short)0, kTile * ld, 0x00020000);
    const int k = c.kt * kKB;
#pragma unroll
    for (int i = i0; i < i1; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          rs, (__attribute__((address_space(3))) void*)(st + i * 256 * 16), 16, op == 0 ? va : vb,
          k + i * 32 * ld, 0, 0);
  };

  const int cm = lane & 31, half = lane >> 5;
  const uint32_t fa = frag_base(wm0 + cm, half), fb = frag_base(wn0 + cm, half) + kOp;
  // The epilogue. Lane l holds row l & 31, columns 8 q + 4 (l >> 5) .. + 3 of each
  // 32 x 32 tile; swapping halves between two groups of columns leaves it 8 in a
  // row, so that operands and results move 16 bytes a lane (fp32: 32). The first
  // of mul and res is fetched a row tile ahead, its first rows before the tile's
  // products; scales of W's rows and bias come from LDS.
  typedef typename std::conditional<YBF16, uint16_t, float>::type E;
  constexpr int NV = sizeof(E) / 2;   // 16-byte vectors of 8 columns
  struct Cols {
    u32x4 v[NV];
  };
  constexpr bool SCALED = std::is_same<typename Ty::Sum, int>::value;
  const E* const opnd = static_cast<const E*>(p.mul ? p.mul : p.res);
  const long long ldo = p.mul ? p.ldm : p.ldr;
  constexpr bool AHEAD = YBF16;   // fp32 operands would take more registers than there are
  Cols pre[2][4];
  float* const colv = reinterpret_cast<float*>(lds + 2 * kStage);   // 256 scales, 256 biases
  auto column = [&](int n0, int q) { return n0 + wn0 + q * 16 + 8 * half; };   // q = 2 j + h
  auto fetch_one = [&](const E* from, long long ld, int m0, int n0, int i, int q) __attribute__((always_inline)) {
    const u32x4* v = reinterpret_cast<const u32x4*>(from + ((long long)m0 + wm0 + i * 32 + cm) * ld + column(n0, q));
    Cols o;
#pragma unroll
    for (int k = 0; k < NV; ++k) o.v[k] = v[k];
    return o;
  };
  auto fetch = [&](const E* from, long long ld, int m0, int n0, int i, Cols (&o)[4])
                   __attribute__((always_inline)) {
#pragma unroll
    for (int q = 0; q < 4; ++q) o[q] = fetch_one(from, ld, m0, n0, i, q);
  };
  auto widen = [](const Cols& v, float (&o)[8]) __attribute__((always_inline)) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if constexpr (YBF16) o[e] = __uint_as_float(e & 1 ? v.v[0][e / 2] & 0xffff0000u : v.v[0][e / 2] << 16);
      else o[e] = __uint_as_float(v.v[e / 4][e & 3]);
    }
  };
  // m0, n0: where the tile lies; m1, n1: the first row and column that are its own
  auto store_tile = [&](typename Ty::Acc (&acc)[4][2], int m0, int n0, int m1, int n1)
                        __attribute__((always_inline)) {
    Cols out[AHEAD ? 4 : 1][4];
    auto put = [&](const Cols& r, int i, int q) __attribute__((always_inline)) {
      const long long t = (long long)m0 + wm0 + i * 32 + cm;
      const int c = column(n0, q);
      if (t >= m1 && c >= n1) {
        u32x4* y = reinterpret_cast<u32x4*>(static_cast<E*>(p.Y) + t * p.ldy + c);
#pragma unroll
        for (int k = 0; k < NV; ++k) y[k] = r.v[k];
      }
    };
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (AHEAD && opnd && i < 3) fetch(opnd, ldo, m0, n0, i + 1, pre[(i + 1) & 1]);
      float sx = 1.0f;
      if constexpr (SCALED) sx = p.sx[(long long)m0 + wm0 + i * 32 + cm];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        typename Ty::Sum w[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          w[e] = acc[i][q / 2][8 * (q & 1) + e];
          w[4 + e] = acc[i][q / 2][8 * (q & 1) + 4 + e];
          swap_halves(w[e], w[4 + e]);
        }
        float v[8], o[8];
        const int lc8 = wn0 + q * 16 + 8 * half;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          v[e] = (float)w[e];
          if constexpr (SCALED) v[e] = v[e] * sx * colv[lc8 + e];
        }
        if (p.bias) {
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] += colv[kTile + lc8 + e];
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = activate<YBF16>(v[e], ACT);
        if (p.mul) {
          widen(AHEAD ? pre[i & 1][q] : fetch_one(static_cast<const E*>(p.mul), p.ldm, m0, n0, i, q), o);
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] *= o[e];
        }
        if (p.res) {
          if (AHEAD && !p.mul) widen(pre[i & 1][q], o);
          else widen(fetch_one(static_cast<const E*>(p.res), p.ldr, m0, n0, i, q), o);
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] += o[e];
        }
        Cols& r = out[AHEAD ? i : 0][q];
        if constexpr (YBF16) {
#pragma unroll
          for (int e = 0; e < 4; ++e) r.v[0][e] = pack2(v[2 * e], v[2 * e + 1]);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) r.v[e / 4][e & 3] = __float_as_uint(v[e]);
          put(r, i, q);
        }
        __builtin_amdgcn_sched_barrier(0);   // one group at a time: registers
      }
    }
    // Stores last: loads and stores of a wave complete in order, so a fetch behind
    // a store would wait for its acknowledgement
    if constexpr (AHEAD) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q) put(out[i][q], i, q);
    }
  };

  auto run = [&](auto ld_tag) {
    constexpr bool LD = decltype(ld_tag)::value;
    Cursor ca{}, cw{};   // X stands two stages ahead, W one
    if constexpr (LD) {
      ca = Cursor{0, 0, row_of(0, 0)};
      cw = Cursor{0, 0, row_of(0, 1)};
      issue(ca, 0, 0, 0, kLoads);
      issue(cw, 1, 0, 0, kLoads);
      advance(ca, 0);
      advance(cw, 1);
      issue(ca, 0, 1, 0, kLoads);   // stage 1's X tile; its W tile goes out in stage 0's first steps
      advance(ca, 0);
      vm_wait<kLoads>();            // stage 0 landed
    }
    lds_sync();
    i32x4 af[2][4], bf[2][2];
#pragma unroll
    for (int i = 0; i < 4; ++i) af[0][i] = frag(lds, fa, i, 0);
#pragma unroll
    for (int j = 0; j < 2; ++j) bf[0][j] = frag(lds, fb, j, 0);

    int buf = 0;
    for (int ti = 0; ti < t_count; ++ti) {
      int m1, n1;
      origin(ti, m1, n1);
      const int m0 = min(m1, (int)p.T - kTile), n0 = min(n1, p.m - kTile);
      float bias = 0.0f, scale = 0.0f;
      if constexpr (!LD) {
        if constexpr (SCALED) scale = p.sw[n0 + g];
        if (p.bias) bias = p.bias[n0 + g];
      }
      if (AHEAD && opnd) fetch(opnd, ldo, m0, n0, 0, pre[0]);
      typename Ty::Acc acc[4][2];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int v = 0; v < 16; ++v) acc[i][j][v] = 0;
      for (int kt = 0; kt < nk; ++kt, buf ^= 1) {
        const unsigned char* sa = lds + buf * kStage;
#pragma unroll
        for (int kk = 0; kk < kSteps; ++kk) {
          const int cb = kk & 1, nb = cb ^ 1;
          if (kk + 1 < kSteps) {
            if (LD && kk < 2) issue(cw, 1, buf ^ 1, kk * (kLoads / 2), (kk + 1) * (kLoads / 2));
#pragma unroll
            for (int i = 0; i < 4; ++i) af[nb][i] = frag(sa, fa, i, kk + 1);
#pragma unroll
            for (int j = 0; j < 2; ++j) bf[nb][j] = frag(sa, fb, j, kk + 1);
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
              for (int j = 0; j < 2; ++j) acc[i][j] = Ty::mma(bf[cb][j], af[cb][i], acc[i][j]);
            // the next step's 6 reads (and the loaders' W tile) go out between
            // the first six products
#pragma unroll
            for (int q = 0; q < 6; ++q) {
              __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
              if (LD && kk < 2) __builtin_amdgcn_sched_group_barrier(0x020, (kLoads / 2 + 5) / 6, 0);
              __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
            }
            __builtin_amdgcn_sched_group_barrier(0x008, 2, 0);
            __builtin_amdgcn_sched_barrier(0);
          } else {
            // the next stage landed, and this one no longer read by anyone, once
            // every wave is past this barrier
            if constexpr (LD) vm_wait<0>();
            lds_sync();
            if constexpr (LD) issue(ca, 0, buf, 0, kLoads);
            const unsigned char* na = lds + (buf ^ 1) * kStage;
#pragma unroll
            for (int i = 0; i < 4; ++i) af[nb][i] = frag(na, fa, i, 0);
#pragma unroll
            for (int j = 0; j < 2; ++j) bf[nb][j] = frag(na, fb, j, 0);
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
              for (int j = 0; j < 2; ++j) acc[i][j] = Ty::mma(bf[cb][j], af[cb][i], acc[i][j]);
#pragma unroll
            for (int q = 0; q < 8; ++q) {
              __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
              if (LD) __builtin_amdgcn_sched_group_barrier(0x020, (kLoads + 7) / 8, 0);
              __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
            }
            __builtin_amdgcn_sched_barrier(0);
            if constexpr (LD) {
              advance(ca, 0);
              advance(cw, 1);
            }
          }
        }
      }
      if (SCALED || p.bias) {
        // the values of the last tile were read before a barrier of this one
        if constexpr (!LD) {
          colv[g] = scale;
          colv[kTile + g] = bias;
        }
        lds_sync();
      }
      store_tile(acc, m0, n0, m1, n1);
    }
  };
  if (wave < 4) run(std::true_type{});
  else run(std::false_type{});
  // the last iterations loaded the final stage again into buffers nobody reads:
  // let those writes land before the workgroup's LDS is released
  vm_wait<0>();
}

template <typename Ty, bool YBF16, int ACT>
hipError_t launch(const LinearArgs& a, hipStream_t s) {
  const long long ntile = ((a.T + kTile - 1) / kTile) * ((a.m + kTile - 1) / kTile);
  // a multiple of 8, so that every XCD's range of tiles has its workgroups
  const long long grid = std::min<long long>((ntile + 7) / 8 * 8, 256);
  hipLaunchKernelGGL((linear_pipe_kernel<Ty, YBF16, ACT>), dim3((unsigned)grid), dim3(kThr), kLds, s, a);
  return hipGetLastError();
}
template <typename Ty, bool YBF16>
hipError_t launch(const LinearArgs& a, hipStream_t s) {
  switch (a.act) {
    case POETX_ACT_RELU: return launch<Ty, YBF16, POETX_ACT_RELU>(a, s);
    case POETX_ACT_SILU: return launch<Ty, YBF16, POETX_ACT_SILU>(a, s);
    case POETX_ACT_GELU: return launch<Ty, YBF16, POETX_ACT_GELU>(a, s);
    case POETX_ACT_GELU_TANH: return launch<Ty, YBF16, POETX_ACT_GELU_TANH>(a, s);
  }
  return launch<Ty, YBF16, POETX_ACT_NONE>(a, s);
}

}  // namespace

bool linear_pipe_supported(const LinearArgs& a, int type) {
  if (type == LINEAR_F32) return false;
  const int es = type == LINEAR_BF16 ? 2 : 1;
  if (a.T < kTile || a.m < kTile || a.m % 8 || (long long)a.n * es % kKB || a.ldx * es % 16 || a.ldw * es % 16) return false;
  if (((uintptr_t)a.X | (uintptr_t)a.W) & 15) return false;
  return a.ldx * es * kTile < (1LL << 31) && a.ldw * es * kTile < (1LL << 31);
}

hipError_t launch_linear_pipe(const LinearArgs& a, int type, hipStream_t s) {
  if (type == LINEAR_BF16) return a.y_bf16 ? launch<PipeBf16, true>(a, s) : launch<PipeBf16, false>(a, s);
  return a.y_bf16 ? launch<PipeI8, true>(a, s) : launch<PipeI8, false>(a, s);
}

}  // namespace poetx
