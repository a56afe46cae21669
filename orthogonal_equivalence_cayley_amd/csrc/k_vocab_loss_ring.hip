// The products of the vocabulary's cross entropy (k_vocab_loss.hip) where 256 x 256 tiles
// would leave CUs idle, and in fp32: smaller tiles, one to a workgroup of four waves, with a
// ring of NS LDS stages of 128 bytes of the summed axis filled by direct-to-LDS loads, as in
// the merged-weight product (k_linear_ring.hip): one barrier a stage, in its middle, so that
// loads, LDS reads and products of three stages overlap.
//
// An operand whose rows run across the summed axis lies in LDS as it comes, 128 bytes' worth
// of summed rows of R columns. bf16 reads it by the transposing LDS read, 8 summed rows by 32
// bytes for half a wave, fp32 by words, 4 summed rows by 64 bytes at a time; the 32-byte
// (64-byte) pieces of a summed row are swizzled by its number so that these fall in distinct
// banks (`turn`; fp32 rows of 32 columns, two to a bank).
//
// Bound by the latency of a stage and, in fp32, by the matrix units: 512 x 512 x 8000 fp32 in
// 128 x 64 tiles STATS 37, GRAD 40, DW 41 us (busy 0.55 to 0.6).
//
// Rows past the last are clamped to it (not stored). Requirements (vocab_ring_logits and the
// like): rows of whole 16 bytes.
#include <algorithm>

#include "linear_common.h"
#include "vocab_loss.h"

namespace poetx {
namespace {

using namespace lin;
using namespace vocab;

typedef short i16x4 __attribute__((ext_vector_type(4)));
typedef short i16x8 __attribute__((ext_vector_type(8)));

constexpr int kThr = 256;
constexpr int kKB = 128;   // bytes of the summed axis a stage

// The 16-byte chunks of summed row k are stored at their number ^ turn(k)
template <int ES, int R>
__device__ __forceinline__ int turn(int k) {
  if constexpr (ES == 4) return ((k >> 2) & (R >= 64 ? 3 : 1)) << 2;
  else if constexpr (R >= 128) return ((k & 3) | (k >> 3 & 1) << 2) << 1;
  else if constexpr (R == 64) return ((k >> 1 & 1) | (k >> 3 & 1) << 1) << 1;
  else return (k >> 3 & 1) << 1;
}

// One operand of a tile: R rows from r0 on, of `rows`
template <typename Ty, int R, bool ACROSS>
struct Side;
template <typename Ty, int R>
struct Side<Ty, R, false> {
  static constexpr int ES = Ty::kSize, L = R / 32;
  const char* base;
  uint32_t off[L], chunk, bytes;
  __device__ __forceinline__ void init(const char* p, long long ld_, int r0, int rows) {
    const int ld = (int)(ld_ * ES), lr = (int)threadIdx.x / 8, last = min(R, rows - r0) - 1;
    chunk = (uint32_t)((threadIdx.x & 7) ^ ((lr / 2) & 7)) * 16;
    base = p + (long long)r0 * ld;
    bytes = (uint32_t)(last + 1) * (uint32_t)ld;
#pragma unroll
    for (int i = 0; i < L; ++i) off[i] = (uint32_t)(min(i * 32 + lr, last) * ld) + chunk;
  }
  // `gone`: this lane's chunk lies behind the sum's end; it loads the stage's first instead
  template <bool WRITTEN>
  __device__ __forceinline__ void issue(uint32_t to, int stage, bool gone, int) const {
#pragma unroll
    for (int i = 0; i < L; ++i)
      load_lds<WRITTEN>(base, bytes, to + i * 4096, off[i] - (gone ? chunk : 0), (uint32_t)(stage * kKB));
  }
  static __device__ __forceinline__ i32x4 frag(const char* st, int r, int q, int lane) {
    const int row = r + (lane & 15), c = q * 4 + (lane >> 4);
    return *reinterpret_cast<const i32x4*>(st + row * kKB + ((c ^ ((row / 2) & 7)) * 16));
  }
};
template <typename Ty, int R>
struct Side<Ty, R, true> {
  static constexpr int ES = Ty::kSize, L = R / 32, KE = kKB / ES;
  static constexpr int CPR = R * ES / 16, RPL = kThr / CPR;   // chunks of a summed row, summed rows a load
  const char* base;
  int ld;
  uint32_t col[L];
  __device__ __forceinline__ void init(const char* p, long long ld_, int r0, int rows) {
    ld = (int)(ld_ * ES);
    base = p + (long long)r0 * ES;
    const int last = min(R, rows - r0) * ES / 16 - 1;   // chunk
#pragma unroll
    for (int i = 0; i < L; ++i)
      col[i] = (uint32_t)min((int)(threadIdx.x % CPR) ^ turn<ES, R>((int)threadIdx.x / CPR + i * RPL), last) * 16;
  }
  // `rows`: summed rows that exist; the last is taken for those of the stage that do not (all
  // of them, where the sum goes on behind it)
  template <bool WRITTEN>
  __device__ __forceinline__ void issue(uint32_t to, int stage, bool, int rows) const {
    const int first = min(stage * KE, rows - 1), there = min(rows - first, KE);
    const char* const at = base + (long long)first * ld;
    const uint32_t bytes = (uint32_t)((there - 1) * ld + R * ES);
#pragma unroll
    for (int i = 0; i < L; ++i)
      load_lds<WRITTEN>(at, bytes, to + i * 4096,
                        (uint32_t)(min((int)threadIdx.x / CPR + i * RPL, there - 1) * ld) + col[i], 0);
  }
  static __device__ __forceinline__ i32x4 frag(const char* st, int r, int q, int lane) {
    if constexpr (ES == 2) {
      // 16 lanes read a 4 x 16 block, lane i its 8 bytes of summed row i / 4, and get column i
      const int k = 32 * q + 8 * (lane >> 4) + (lane >> 2 & 3), c = r + 4 * (lane & 3);
      auto at = [&](int k) {
        return (__attribute__((address_space(3))) i16x4*)(st + k * (R * 2) + ((c >> 3) ^ turn<2, R>(k)) * 16 + (c & 7) * 2);
      };
      const i16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16(at(k));
      const i16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16(at(k + 4));
      const i16x8 v = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
      return __builtin_bit_cast(i32x4, v);
    } else {
      const int k = 16 * q + 4 * (lane >> 4), c = r + (lane & 15);
      i32x4 v;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        v[i] = *reinterpret_cast<const int*>(st + (k + i) * (R * 4) + ((c >> 2) ^ turn<4, R>(k + i)) * 16 + (c & 3) * 4);
      return v;
    }
  }
};

// TAIL: n is no multiple of a stage (STATS, GRAD)
template <typename Ty, int BM, int BN, int NS, Mode MODE, bool TAIL>
__global__ __launch_bounds__(kThr) __attribute__((amdgpu_waves_per_eu(2, 2)))
void vocab_ring_kernel(VocabArgs p) {
  constexpr bool AX = MODE == DW, BX = MODE == DX || MODE == DW;
  // the transposing reads need the written form of the loads (load_lds)
  constexpr bool WRITTEN = BX && Ty::kSize == 2;
  using SA = Side<Ty, BM, AX>;
  using SB = Side<Ty, BN, BX>;
  constexpr int KE = kKB / Ty::kSize;
  constexpr int TM = BM / 32, TN = BN / 32;    // 16 x 16 tiles of a wave (2 x 2 waves)
  constexpr int STAGE = (BM + BN) * kKB, LOADS = SA::L + SB::L;
  static_assert(NS * LOADS <= 63, "loads in flight");
  extern __shared__ __align__(16) char lds[];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = (wave >> 1) * (BM / 2), wn = (wave & 1) * (BN / 2);
  const int rows = MODE == DW ? p.vp : (int)(MODE == DX ? p.Td : p.T), cols = MODE == STATS || MODE == GRAD ? p.vp : p.n;
  int m0, n0;
  if (!tile_origin(rows, cols, BM, BN, m0, n0)) return;
  // d has zeros in its columns up to a multiple of 64 and in its rows up to Tm
  const int sum = MODE == DX ? (p.vp + 63) / 64 * 64 : MODE == DW ? (int)p.Tm : p.n;
  const int stages = (sum + KE - 1) / KE;
  const int per = MODE == DX ? (stages + p.splits - 1) / p.splits : stages;
  const int s0 = MODE == DX ? (int)blockIdx.y * per : 0, nk = min(per, stages - s0);
  const char* const w = static_cast<const char*>(p.W) + (long long)p.v0 * p.ldw * Ty::kSize;
  SA sa;
  SB sb;
  if constexpr (MODE == STATS || MODE == GRAD) {
    sa.init(static_cast<const char*>(p.X), p.ldx, m0, rows);
    sb.init(w, p.ldw, n0, cols);
  } else if constexpr (MODE == DX) {
    sa.init(static_cast<const char*>(p.dS), p.ldp, m0, rows);
    sb.init(w, p.ldw, n0, cols);
  } else {
    sa.init(static_cast<const char*>(p.dS), p.ldp, m0, (int)p.ldp);
    sb.init(static_cast<const char*>(p.Xm), p.ldm, n0, (int)p.ldm);
  }
  const uint32_t lds_at =
      __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(__attribute__((address_space(3))) char*)lds) +
      (uint32_t)(wave * 1024);
  const int lc = ((tid & 7) ^ ((tid / 16) & 7)) * 16 / Ty::kSize;   // this lane's first element of a stage (rows along the sum)
  auto gone = [&](int s) __attribute__((always_inline)) { return TAIL && (s0 + s) * KE + lc >= sum; };
  // stage s (past the end: the last one again, into a buffer nobody reads)
  auto issue = [&](int s, int buf) __attribute__((always_inline)) {
    s = min(s, nk - 1);
    const uint32_t to = lds_at + (uint32_t)(buf * STAGE);
    sa.template issue<WRITTEN>(to, s0 + s, gone(s), sum);
    sb.template issue<WRITTEN>(to + BM * kKB, s0 + s, gone(s), MODE == DX ? p.vp : sum);
  };
  auto clear = [&](int s, int buf) __attribute__((always_inline)) {
    if (!gone(s)) return;
#pragma unroll
    for (int i = 0; i < LOADS; ++i) *reinterpret_cast<i32x4*>(lds + buf * STAGE + tid * 16 + i * 4096) = i32x4{0, 0, 0, 0};
  };
  typename Ty::Acc acc[TM][TN] = {};
  i32x4 af[2][TM], bf[2][TN];
  auto read = [&](int buf, int q) __attribute__((always_inline)) {
    const char* const st = lds + buf * STAGE;
#pragma unroll
    for (int i = 0; i < TM; ++i) af[q][i] = SA::frag(st, wm + i * 16, q, lane);
#pragma unroll
    for (int j = 0; j < TN; ++j) bf[q][j] = SB::frag(st + BM * kKB, wn + j * 16, q, lane);
  };
  auto multiply = [&](int q) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j) Ty::mma(bf[q][j], af[q][i], acc[i][j]);
  };
  if (nk > 0) {   // a later, shorter piece may leave a share empty
#pragma unroll
    for (int s = 0; s < NS; ++s) issue(s, s);
    vm_wait<(NS - 1) * LOADS>();   // this wave's part of stage 0 landed
    if (TAIL) clear(0, 0);
    lds_sync();                    // and everyone's
    read(0, 0);
    int buf = 0;
    for (int s = 0; s < nk; ++s) {
      const int next = buf + 1 == NS ? 0 : buf + 1;
      read(buf, 1);
      multiply(0);
      __builtin_amdgcn_sched_barrier(0);
      vm_wait<(NS - 2) * LOADS>();
      if (TAIL && s + 1 < nk) clear(s + 1, next);
      lds_sync();   // stage s + 1 landed, and nobody reads stage s any more
      read(next, 0);
      issue(s + NS, buf);
      multiply(1);
      __builtin_amdgcn_sched_barrier(0);
      buf = next;
    }
    // the last loads went into buffers nobody reads: let them land before the workgroup's LDS
    // is released
    vm_wait<0>();
  }
  epilogue<Ty, BN, TM, TN, MODE>(p, acc, rows, cols, m0, n0, wm, wn, MODE == DX ? (int)blockIdx.y : 0);
}

template <typename Ty, int BM, int BN, int NS, Mode MODE>
hipError_t launch(const VocabArgs& a, hipStream_t s) {
  const long long rows = MODE == DW ? a.vp : MODE == DX ? a.Td : a.T;
  const int cols = MODE == STATS || MODE == GRAD ? a.vp : a.n;
  const dim3 grid((unsigned)tile_grid(rows, cols, BM, BN), MODE == DX ? (unsigned)a.splits : 1u);
  constexpr int lds = NS * (BM + BN) * kKB;
  constexpr bool along = MODE == STATS || MODE == GRAD;
  if (along && (long long)a.n * Ty::kSize % kKB)
    hipLaunchKernelGGL((vocab_ring_kernel<Ty, BM, BN, NS, MODE, along>), grid, dim3(kThr), lds, s, a);
  else
    hipLaunchKernelGGL((vocab_ring_kernel<Ty, BM, BN, NS, MODE, false>), grid, dim3(kThr), lds, s, a);
  return hipGetLastError();
}
template <typename Ty, Mode MODE>
hipError_t launch(const VocabArgs& a, int tile, hipStream_t s) {
  switch (tile) {
    case VOCAB_TILE_128:
      if constexpr (Ty::kSize == 2) return launch<Ty, 128, 128, 2, MODE>(a, s);
      break;
    case VOCAB_TILE_128x64: return launch<Ty, 128, 64, 3, MODE>(a, s);
    case VOCAB_TILE_64: return launch<Ty, 64, 64, 4, MODE>(a, s);
    case VOCAB_TILE_32x64: return launch<Ty, 32, 64, 4, MODE>(a, s);
  }
  return hipErrorInvalidValue;
}
template <Mode MODE>
hipError_t launch(const VocabArgs& a, int bf16, int tile, hipStream_t s) {
  return bf16 ? launch<TypeBf16, MODE>(a, tile, s) : launch<TypeF32, MODE>(a, tile, s);
}

bool whole(const void* p, long long ld, int es) { return ((uintptr_t)p & 15) == 0 && ld * es % 16 == 0 && ld * es < (1 << 22); }

}  // namespace

bool vocab_ring_weight(const VocabArgs& a, int bf16) {
  const int es = bf16 ? 2 : 4;
  return (long long)a.n * es % 16 == 0 && whole(a.W, a.ldw, es) && a.ldp * es < (1 << 22);
}
bool vocab_ring_logits(const VocabArgs& a, int bf16) {
  return vocab_ring_weight(a, bf16) && whole(a.X, a.ldx, bf16 ? 2 : 4);
}
hipError_t launch_vocab_ring_stats(const VocabArgs& a, int bf16, int tile, hipStream_t s) { return launch<STATS>(a, bf16, tile, s); }
hipError_t launch_vocab_ring_grad(const VocabArgs& a, int bf16, int tile, hipStream_t s) { return launch<GRAD>(a, bf16, tile, s); }
hipError_t launch_vocab_ring_dx(const VocabArgs& a, int bf16, int tile, hipStream_t s) { return launch<DX>(a, bf16, tile, s); }
hipError_t launch_vocab_ring_dw(const VocabArgs& a, int bf16, int tile, hipStream_t s) { return launch<DW>(a, bf16, tile, s); }

}  // namespace poetx
