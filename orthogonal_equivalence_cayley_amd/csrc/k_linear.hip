// Product of activations with a merged weight and its epilogue,
//   Y = act(X W^T + bias) * mul + res,
// X [T, n], W [m, n] both along n: fp32, bf16, or INT8 rows with a scale each
// (z = float(sum q q) sx sw, the sum exact in 32 bits). Sums in fp32 (INT8: in
// integers), the epilogue in fp32, one rounding at the end.
//
// Four kernels:
//  * few tokens (few_rows: one to four), linear_rows: every wave takes a row of W and
//    multiplies on the vector units: bound by the weight's bytes (one token, 2048 to
//    5632 bf16 6.1 us).
//  * linear_pipe (k_linear_pipe.hip) and linear_ring (k_linear_ring.hip): tiles
//    filled by direct-to-LDS loads, for rows of whole 128- and 16-byte pieces.
//  * linear_tile: tiles filled through registers, any sizes and alignment.
// The tile is the one of least cost for the grid it makes (`cheapest`).
#include <algorithm>

#include "linear_common.h"

namespace poetx {
namespace {

using namespace lin;

// ------------------------------------------------------------------ single tokens
constexpr int kRowThr = 256;
// One row of W to a wave (two rows 6.4 against 6.1 us at 2048 to 5632 bf16, 8.9
// against 7.7 at 5632 to 2048; a row split over two waves 8.4 and 7.0); TT tokens.
template <typename Ty, int TT, bool YBF16>
__global__ __launch_bounds__(kRowThr) void linear_rows_kernel(LinearArgs a) {
  const int lane = threadIdx.x & 63;
  const int c = (int)blockIdx.x * (kRowThr / 64) + (threadIdx.x >> 6);
  if (c >= a.m) return;
  const long long kb = (long long)a.n * Ty::kSize;
  const char* const w = static_cast<const char*>(a.W) + (long long)c * a.ldw * Ty::kSize;
  const char* x[TT];
#pragma unroll
  for (int t = 0; t < TT; ++t)
    x[t] = static_cast<const char*>(a.X) + (long long)min((long long)t, a.T - 1) * a.ldx * Ty::kSize;
  typename Ty::Sum acc[TT] = {};
  // pieces of 1 KB, four at a time with all their loads out first
  constexpr int U = 4;
  const long long k = lane * 16;
  long long p = 0;
  for (; p + 1024 * U <= kb; p += 1024 * U) {
    i32x4 wv[U], xv[U][TT];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      __builtin_memcpy(&wv[u], w + p + k + u * 1024, 16);
#pragma unroll
      for (int t = 0; t < TT; ++t) __builtin_memcpy(&xv[u][t], x[t] + p + k + u * 1024, 16);
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int t = 0; t < TT; ++t) Ty::dot(wv[u], xv[u][t], acc[t]);
  }
  for (; p < kb; p += 1024) {
    const i32x4 wv = load16<Ty::kSize>(w, p + k, kb);
    i32x4 xv[TT];
#pragma unroll
    for (int t = 0; t < TT; ++t) xv[t] = load16<Ty::kSize>(x[t], p + k, kb);
#pragma unroll
    for (int t = 0; t < TT; ++t) Ty::dot(wv, xv[t], acc[t]);
  }
#pragma unroll
  for (int t = 0; t < TT; ++t) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) acc[t] += __shfl_xor(acc[t], o);
    const typename Ty::Sum o[1] = {acc[t]};
    if (lane == t && t < a.T) finish<YBF16>(a, o, t, c);
  }
}

// ------------------------------------------------------------------ tiles
// BM tokens x BN rows of W per workgroup, four waves of BM/2 x BN/2 each, any
// sizes and alignment. KB bytes of n per stage, two LDS buffers and one barrier a
// stage; the global loads of the next two stages are under way in registers, and
// the LDS reads of the next 64-byte slab beside the products of one. KS groups of
// four waves take every KS-th stage and add up their sums in LDS, for grids that
// leave CUs idle. 16-byte chunk c of tile row r sits at slot r KB/16 + (c ^ sw(r)),
// so that the 16 rows a quarter of a wave reads at one chunk fall in distinct
// banks. Measured: 1000 x 999 x 1000 bf16 12.5 us, 16384 x 1001 x 2001 137 us
// (480 TFLOP/s), 1531 x 1005 x 707 fp32 39 us (56 TFLOP/s; the matrix units alone
// would take 23 for the three tiles the fullest CU gets).
template <int BM, int BN, int KB, int KS>
constexpr int tile_lds() {
  return KS * 2 * (BM + BN) * KB;
}
template <typename Ty, int BM, int BN, int KB, int KS, bool PART, bool YBF16>
__global__ __launch_bounds__(256 * KS) __attribute__((amdgpu_waves_per_eu(2, 2)))
void linear_tile_kernel(LinearArgs a) {
  constexpr int CPR = KB / 16;
  constexpr int RPL = 256 / CPR;               // rows one load of the group covers
  constexpr int LX = BM / RPL, LW = BN / RPL;
  constexpr int TM = BM / 32, TN = BN / 32;    // 16 x 16 tiles of a wave
  static_assert(BM % RPL == 0 && BN % RPL == 0 && TM > 0 && TN > 0, "whole loads and tiles");
  extern __shared__ __align__(16) i32x4 lds[];
  const int tid = threadIdx.x & 255, lane = tid & 63, wave = tid >> 6;
  const int grp = KS == 1 ? 0 : __builtin_amdgcn_readfirstlane(threadIdx.x >> 8);
  i32x4* const mine = lds + grp * 2 * (BM + BN) * CPR;
  int m0, c0;
  if (!tile_origin(a.T, a.m, BM, BN, m0, c0)) return;
  const long long t0 = m0;
  const int wm = (wave >> 1) * (BM / 2), wn = (wave & 1) * (BN / 2);
  const long long kb = (long long)a.n * Ty::kSize;
  const int lr = tid / CPR, lc = tid % CPR;
  const char* xs[LX];
  const char* ws[LW];
#pragma unroll
  for (int i = 0; i < LX; ++i)
    xs[i] = static_cast<const char*>(a.X) + min(t0 + i * RPL + lr, a.T - 1) * a.ldx * Ty::kSize;
#pragma unroll
  for (int i = 0; i < LW; ++i)
    ws[i] = static_cast<const char*>(a.W) + (long long)min(c0 + i * RPL + lr, a.m - 1) * a.ldw * Ty::kSize;
  i32x4 xr[2][LX], wr[2][LW];   // two stages under way
  auto fetch = [&](long long k0, int set) __attribute__((always_inline)) {
    const long long k = k0 + lc * 16;
    if (k0 + KB <= kb) {   // every chunk of the stage is whole
#pragma unroll
      for (int i = 0; i < LX; ++i) __builtin_memcpy(&xr[set][i], xs[i] + k, 16);
#pragma unroll
      for (int i = 0; i < LW; ++i) __builtin_memcpy(&wr[set][i], ws[i] + k, 16);
    } else {
#pragma unroll
      for (int i = 0; i < LX; ++i) xr[set][i] = load16<Ty::kSize>(xs[i], k, kb);
#pragma unroll
      for (int i = 0; i < LW; ++i) wr[set][i] = load16<Ty::kSize>(ws[i], k, kb);
    }
  };
  auto slot = [](int r, int c) { return r * CPR + (c ^ (CPR == 8 ? (r / 2) & 7 : r & (CPR - 1))); };
  auto keep = [&](int buf, int set) __attribute__((always_inline)) {
    i32x4* const to = mine + buf * (BM + BN) * CPR;
#pragma unroll
    for (int i = 0; i < LX; ++i) to[slot(i * RPL + lr, lc)] = xr[set][i];
#pragma unroll
    for (int i = 0; i < LW; ++i) to[BM * CPR + slot(i * RPL + lr, lc)] = wr[set][i];
  };
  typename Ty::Acc acc[TM][TN] = {};
  // the same number of stages for every group: those behind the end hold zeros
  const long long step = (long long)KB * KS * (PART ? a.splits : 1);
  const int stages = (int)((kb + step - 1) / step);
  const long long first = (long long)((PART ? (int)blockIdx.y * KS : 0) + grp) * KB;
  constexpr int Q = KB / 64;   // slabs of a stage
  static_assert(Q % 2 == 0, "fragment sets alternate across stages");
  i32x4 xf[2][TM], wf[2][TN];
  auto read = [&](int buf, int q) __attribute__((always_inline)) {
    const i32x4* const from = mine + buf * (BM + BN) * CPR;
    const int c = q * 4 + (lane >> 4);
#pragma unroll
    for (int i = 0; i < TM; ++i) xf[q & 1][i] = from[slot(wm + i * 16 + (lane & 15), c)];
#pragma unroll
    for (int j = 0; j < TN; ++j) wf[q & 1][j] = from[BM * CPR + slot(wn + j * 16 + (lane & 15), c)];
  };
  fetch(first, 0);
  keep(0, 0);
  if (stages > 1) fetch(first + step, 1);
  if (stages > 2) fetch(first + 2 * step, 0);
  lds_sync();
  read(0, 0);
  auto stage = [&](int s, int buf) __attribute__((always_inline)) {
    // nobody reads the other buffer since the barrier of the stage before
    if (s + 1 < stages) keep(buf ^ 1, buf ^ 1);
    if (s + 3 < stages) fetch(first + (s + 3) * step, buf ^ 1);
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      if (q + 1 < Q) {
        read(buf, q + 1);
      } else {
        lds_sync();
        if (s + 1 < stages) read(buf ^ 1, 0);
      }
#pragma unroll
      for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j) Ty::mma(wf[q & 1][j], xf[q & 1][i], acc[i][j]);
    }
  };
  for (int s = 0; s < stages; s += 2) {
    stage(s, 0);
    if (s + 1 < stages) stage(s + 1, 1);
  }
  if constexpr (KS > 1) {
    typedef typename Ty::Acc Acc;
    static_assert((KS - 1) * BM * BN * 4 <= tile_lds<BM, BN, KB, KS>(), "sums fit where the stages were");
    __syncthreads();   // the last stage is read
    Acc* const sums = reinterpret_cast<Acc*>(lds);
    if (grp > 0) {
#pragma unroll
      for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j) sums[(((grp - 1) * TM + i) * TN + j) * 256 + tid] = acc[i][j];
    }
    __syncthreads();
    if (grp > 0) return;
#pragma unroll
    for (int g = 0; g < KS - 1; ++g)
#pragma unroll
      for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j) acc[i][j] += sums[((g * TM + i) * TN + j) * 256 + tid];
  }
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j) {
      const long long t = t0 + wm + i * 16 + (lane & 15);
      const int c = c0 + wn + j * 16 + 4 * (lane >> 4);
      if (t < a.T && c < a.m) {
        if constexpr (PART) {
          store_part<Ty>(a, blockIdx.y, t, c, acc[i][j]);
        } else {
          const typename Ty::Sum o[4] = {acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3]};
          finish<YBF16>(a, o, t, c);
        }
      }
    }
}

template <typename Ty, int BM, int BN, int KB, int KS, bool YBF16, bool PART = false>
void tiles(const LinearArgs& a, hipStream_t s) {
  hipLaunchKernelGGL((linear_tile_kernel<Ty, BM, BN, KB, KS, PART, YBF16>),
                     dim3((unsigned)tile_grid(a.T, a.m, BM, BN), PART ? (unsigned)a.splits : 1u), dim3(256 * KS), (tile_lds<BM, BN, KB, KS>()), s, a);
}

template <typename Ty, bool YBF16>
hipError_t launch_tiles(const LinearArgs& a, int tile, hipStream_t s) {
  switch (tile) {
    case LINEAR_TILE_128: tiles<Ty, 128, 128, 128, 1, YBF16>(a, s); break;
    case LINEAR_TILE_128x64: tiles<Ty, 128, 64, 128, 1, YBF16>(a, s); break;
    case LINEAR_TILE_64: tiles<Ty, 64, 64, 256, 1, YBF16>(a, s); break;
    case LINEAR_TILE_32x64: tiles<Ty, 32, 64, 128, 1, YBF16>(a, s); break;
    case LINEAR_TILE_32_SPLIT: tiles<Ty, 32, 32, 256, 2, YBF16>(a, s); break;
    default: return hipErrorInvalidValue;
  }
  return hipGetLastError();
}
hipError_t launch_tiles(const LinearArgs& a, int type, int tile, hipStream_t s) {
  if (a.splits > 1) {   // sums only: the type of Y does not matter
    switch (type) {
      case LINEAR_F32: tiles<TypeF32, 32, 32, 256, 2, false, true>(a, s); break;
      case LINEAR_BF16: tiles<TypeBf16, 32, 32, 256, 2, false, true>(a, s); break;
      default: tiles<TypeI8, 32, 32, 256, 2, false, true>(a, s);
    }
    return hipGetLastError();
  }
  switch (type) {
    case LINEAR_F32: return launch_tiles<TypeF32, false>(a, tile, s);
    case LINEAR_BF16:
      return a.y_bf16 ? launch_tiles<TypeBf16, true>(a, tile, s) : launch_tiles<TypeBf16, false>(a, tile, s);
  }
  return a.y_bf16 ? launch_tiles<TypeI8, true>(a, tile, s) : launch_tiles<TypeI8, false>(a, tile, s);
}

template <typename Ty, int TT, bool YBF16>
hipError_t rows(const LinearArgs& a, hipStream_t s) {
  constexpr int per = kRowThr / 64;
  hipLaunchKernelGGL((linear_rows_kernel<Ty, TT, YBF16>), dim3((unsigned)((a.m + per - 1) / per)), dim3(kRowThr), 0, s,
                     a);
  return hipGetLastError();
}
template <typename Ty, bool YBF16>
hipError_t rows(const LinearArgs& a, hipStream_t s) {
  if (a.T == 1) return rows<Ty, 1, YBF16>(a, s);
  if (a.T == 2) return rows<Ty, 2, YBF16>(a, s);
  return rows<Ty, 4, YBF16>(a, s);
}
hipError_t launch_rows(const LinearArgs& a, int type, hipStream_t s) {
  switch (type) {
    case LINEAR_F32: return rows<TypeF32, false>(a, s);
    case LINEAR_BF16: return a.y_bf16 ? rows<TypeBf16, true>(a, s) : rows<TypeBf16, false>(a, s);
  }
  return a.y_bf16 ? rows<TypeI8, true>(a, s) : rows<TypeI8, false>(a, s);
}

// What a tile costs, in us for 4 KB of every operand row (all of them scale with
// the row): `first` for a grid of up to 256 tiles, one to a CU, and `round` for
// every 256 tiles of a grid where the CUs are full; measured at 2048 x 2048
// weights and 80 to 16384 tokens. bf16 and INT8 cost the same a byte; fp32 is bound
// by its matrix rate, so its cost goes by the tile's area. What a tile takes to start
// and in its epilogue is not counted apart: at n of a few stages the choice can be
// off (2455 x 256 x 3352 bf16 23.8 us, the vendor library 20.5). E.g. bf16 1024 tokens:
// 128 x 128 26.5 us, 128 x 64 15.7, 64 x 64 16.8, 32 x 32 27.9; 16384 tokens: 256 x
// 256 108 us, 128 x 128 141, 128 x 64 173.
struct Cost {
  int tile, bm, bn;
  float first, round;
};
constexpr Cost kRing[] = {
    {LINEAR_TILE_256, 256, 256, 36, 50},      {LINEAR_TILE_128, 128, 128, 24, 17},
    {LINEAR_TILE_128x64, 128, 64, 11, 9.5f},  {LINEAR_TILE_64, 64, 64, 6.5f, 5.8f},
    {LINEAR_TILE_32x64, 32, 64, 4.6f, 4.3f},  {LINEAR_TILE_32, 32, 32, 3.7f, 2.8f},
    {LINEAR_TILE_32_SPLIT, 32, 32, 3.2f, 3.2f}};
constexpr Cost kRingF32[] = {
    {LINEAR_TILE_128, 128, 128, 64, 60},   {LINEAR_TILE_128x64, 128, 64, 33, 30}, {LINEAR_TILE_64, 64, 64, 18, 16.5f},
    {LINEAR_TILE_32x64, 32, 64, 10, 9},    {LINEAR_TILE_32, 32, 32, 6.5f, 5},     {LINEAR_TILE_32_SPLIT, 32, 32, 5, 7.3f}};
constexpr Cost kTiles[] = {
    {LINEAR_TILE_128, 128, 128, 25, 20},     {LINEAR_TILE_128x64, 128, 64, 16.5f, 13}, {LINEAR_TILE_64, 64, 64, 10.5f, 8},
    {LINEAR_TILE_32x64, 32, 64, 5.6f, 5},    {LINEAR_TILE_32_SPLIT, 32, 32, 3.2f, 3.3f}};
constexpr Cost kTilesF32[] = {
    {LINEAR_TILE_128, 128, 128, 75, 65},     {LINEAR_TILE_128x64, 128, 64, 42, 35}, {LINEAR_TILE_64, 64, 64, 23.7f, 18.5f},
    {LINEAR_TILE_32x64, 32, 64, 15.6f, 10.5f}, {LINEAR_TILE_32_SPLIT, 32, 32, 8, 6.6f}};

template <size_t N, typename F>
int cheapest(const Cost (&costs)[N], const LinearArgs& a, F allowed) {
  int best = -1;
  double least = 0.0;
  for (const Cost& c : costs) {
    if (!allowed(c.tile)) continue;
    const long long n = ((a.T + c.bm - 1) / c.bm) * ((a.m + c.bn - 1) / c.bn);
    const double cost = std::max((double)c.first, (double)c.round * (double)((n + 255) / 256));
    if (best < 0 || cost < least) {
      best = c.tile;
      least = cost;
    }
  }
  return best;
}

long long few_rows(int type, bool ring) { return !ring || type == LINEAR_F32 ? 4 : type == LINEAR_BF16 ? 2 : 1; }

// The sums of all splits of 4 columns of a row, in order, and the epilogue
template <typename Ty, bool YBF16>
__global__ __launch_bounds__(256) void linear_join_kernel(LinearArgs a) {
  typedef typename Ty::Acc Acc;
  typedef typename Ty::Sum S;
  const int quads = (a.m + 3) / 4;
  const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
  if (i >= a.T * quads) return;
  const long long t = i / quads;
  const int c = (int)(i - t * quads) * 4;
  Acc v = {0, 0, 0, 0};
#pragma unroll 4
  for (int z = 0; z < a.splits; ++z)
    v += *reinterpret_cast<const Acc*>(static_cast<const S*>(a.part) + part_row(a, z, t) + c);
  const S o[4] = {v[0], v[1], v[2], v[3]};
  finish<YBF16>(a, o, t, c);
}
template <typename Ty, bool YBF16>
hipError_t join(const LinearArgs& a, hipStream_t s) {
  const long long n = a.T * ((a.m + 3) / 4);
  hipLaunchKernelGGL((linear_join_kernel<Ty, YBF16>), dim3((unsigned)((n + 255) / 256)), dim3(256), 0, s, a);
  return hipGetLastError();
}
hipError_t launch_join(const LinearArgs& a, int type, hipStream_t s) {
  switch (type) {
    case LINEAR_F32: return join<TypeF32, false>(a, s);
    case LINEAR_BF16: return a.y_bf16 ? join<TypeBf16, true>(a, s) : join<TypeBf16, false>(a, s);
  }
  return a.y_bf16 ? join<TypeI8, true>(a, s) : join<TypeI8, false>(a, s);
}

hipError_t launch_piece(const LinearArgs& a, int type, hipStream_t s) {
  const bool ring = linear_ring_supported(a, type);
  // Few tokens go by rows (few_rows) while the vector units keep up with the weight: one INT8
  // token (two, 2048 to 5632: 7.1 us by rows, 5.6 in tiles), two bf16 (2048 to 2048
  // 4.4 against 6.6 us; four, 2048 to 5632, 9.1 against 7.2), four fp32 (2048 to 2048
  // 7.5 against 15.8 us), and up to four where rows are ragged.
  if (a.T <= few_rows(type, ring)) return launch_rows(a, type, s);
  if (a.splits > 1) {
    const hipError_t e = ring ? launch_linear_ring(a, type, LINEAR_TILE_32_SPLIT, s)
                              : launch_tiles(a, type, LINEAR_TILE_32_SPLIT, s);
    return e == hipSuccess ? launch_join(a, type, s) : e;
  }
  const bool pipe = ring && linear_pipe_supported(a, type);
  const auto allowed = [&](int tile) {
    return tile == LINEAR_TILE_256 ? pipe : true;
  };
  if (!ring)
    return launch_tiles(a, type, type == LINEAR_F32 ? cheapest(kTilesF32, a, allowed) : cheapest(kTiles, a, allowed), s);
  const int tile = type == LINEAR_F32 ? cheapest(kRingF32, a, allowed) : cheapest(kRing, a, allowed);
  return tile == LINEAR_TILE_256 ? launch_linear_pipe(a, type, s) : launch_linear_ring(a, type, tile, s);
}

}  // namespace

// Where 32 x 32 tiles fill at most a third of the CUs and n is long, several
// workgroups share n: as many as fill the CUs, each with at least 12 stages of 128
// bytes (fp32, whose stages take the matrix units four times as long, 6). It pays for
// the second launch from 48 stages on (bf16 53 x 4624 x 80 13.5 -> 9.4 us, 73 stages;
// 6 x 2816 x 102 7.4 -> 8.6 us, 44), fp32 from 20 (62 x 700 x 256 9.4 -> 8.5 us), and
// not for two workgroups a tile (16 x 11008 x 4096 INT8 11.8 -> 13.9 us).
int linear_splits(const LinearArgs& a, int type) {
  const int es = type == LINEAR_F32 ? 4 : type == LINEAR_BF16 ? 2 : 1;
  const long long stages = ((long long)a.n * es + 127) / 128;
  const long long tiles = ((a.T + 31) / 32) * ((a.m + 31) / 32);
  if (a.T <= 4 || tiles > 85) return 1;
  if (stages < (type == LINEAR_F32 ? 20 : 48)) return 1;
  const long long per = type == LINEAR_F32 ? 6 : 12;
  return (int)std::max(1LL, std::min({32LL, 256 / tiles, stages / per}));
}

hipError_t launch_linear(const LinearArgs& a, int type, hipStream_t s) {
  if (a.T <= 0 || a.m <= 0 || a.n <= 0 || a.m > kLinearMaxRows) return hipErrorInvalidValue;
  if (a.y_bf16 && type == LINEAR_F32) return hipErrorInvalidValue;
  // A launch counts threads in 32 bits: at most 2^22 of the smallest tiles, of 512
  // threads. One launch for any size but results of 2^32 elements and more, the
  // columns counted in whole tiles of 32.
  const long long step = std::max(256LL, (1LL << 22) / ((a.m + 31) / 32) * 32 / 256 * 256);
  const int es = type == LINEAR_F32 ? 4 : type == LINEAR_BF16 ? 2 : 1, ys = a.y_bf16 ? 2 : 4;
  const auto off = [](const void* p, long long bytes) {
    return p ? static_cast<const void*>(static_cast<const char*>(p) + bytes) : nullptr;
  };
  for (long long t = 0; t < a.T; t += step) {
    LinearArgs b = a;
    b.T = std::min(step, a.T - t);
    b.X = off(a.X, t * a.ldx * es);
    b.sx = static_cast<const float*>(off(a.sx, t * 4));
    b.mul = off(a.mul, t * a.ldm * ys);
    b.res = off(a.res, t * a.ldr * ys);
    b.Y = const_cast<void*>(off(a.Y, t * a.ldy * ys));
    const hipError_t e = launch_piece(b, type, s);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace poetx
