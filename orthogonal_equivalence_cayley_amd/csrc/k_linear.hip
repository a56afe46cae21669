// Product of activations with a merged weight and its epilogue,
//   Y = act(X W^T + bias) * mul + res,
// X [T, n], W [m, n] both along n: fp32, bf16, or INT8 rows with a scale each
// (z = float(sum q q) sx sw, the sum exact in 32 bits). Sums in fp32 (INT8: in
// integers), the epilogue in fp32, one rounding at the end.
//
// Three kernels by the number of tokens:
//  * up to 4, linear_rows: every wave takes rows of W whole and multiplies on
//    the vector units: bound by the weight's bytes.
//  * up to 64, linear_few: 16 rows of W to a workgroup, its 8 waves split n and
//    feed the matrix units straight from memory; their sums meet in LDS.
//  * more, linear_tile: tiles staged through LDS, any sizes and alignment.
#include <algorithm>

#include "linear_common.h"

namespace poetx {
namespace {

using namespace lin;

// ------------------------------------------------------------------ single tokens
constexpr int kRowThr = 256;
constexpr int kRowsPerWave = 2;

template <typename Ty, int TT, bool YBF16>
__global__ __launch_bounds__(kRowThr) void linear_rows_kernel(LinearArgs a) {
  constexpr int R = kRowsPerWave;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int c0 = (blockIdx.x * (kRowThr / 64) + wave) * R;
  if (c0 >= a.m) return;
  const long long kb = (long long)a.n * Ty::kSize;
  const char* w[R];
#pragma unroll
  for (int r = 0; r < R; ++r)
    w[r] = static_cast<const char*>(a.W) + (long long)min(c0 + r, a.m - 1) * a.ldw * Ty::kSize;
  const char* x[TT];
#pragma unroll
  for (int t = 0; t < TT; ++t)
    x[t] = static_cast<const char*>(a.X) + (long long)min((long long)t, a.T - 1) * a.ldx * Ty::kSize;
  typename Ty::Sum acc[TT][R] = {};
#pragma unroll 4
  for (long long k = lane * 16; k < kb; k += 1024) {
    i32x4 wv[R], xv[TT];
#pragma unroll
    for (int r = 0; r < R; ++r) wv[r] = load16<Ty::kSize>(w[r] + k, kb - k);
#pragma unroll
    for (int t = 0; t < TT; ++t) xv[t] = load16<Ty::kSize>(x[t] + k, kb - k);
#pragma unroll
    for (int t = 0; t < TT; ++t)
#pragma unroll
      for (int r = 0; r < R; ++r) Ty::dot(wv[r], xv[t], acc[t][r]);
  }
#pragma unroll
  for (int t = 0; t < TT; ++t) {
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int o = 32; o > 0; o >>= 1) acc[t][r] += __shfl_xor(acc[t][r], o);
    if (lane == t && t < a.T) finish<YBF16>(a, acc[t], t, c0);
  }
}

// ------------------------------------------------------------------ few tokens
constexpr int kFewWaves = 8;
constexpr int kFewThr = kFewWaves * 64;

// Wave w takes the 256-byte pieces w, w + 8, .. of n: four slabs of 64 bytes
// whose loads go out together. NT token tiles of 16.
template <typename Ty, int NT, bool YBF16>
__global__ __launch_bounds__(kFewThr) void linear_few_kernel(LinearArgs a) {
  __shared__ typename Ty::Acc red[kFewWaves][NT][64];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int r0 = blockIdx.x * 16;
  const int row = lane & 15, ko = (lane >> 4) * 16;
  const long long kb = (long long)a.n * Ty::kSize;
  const char* w = static_cast<const char*>(a.W) + (long long)min(r0 + row, a.m - 1) * a.ldw * Ty::kSize;
  const char* x[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j)
    x[j] = static_cast<const char*>(a.X) + min((long long)(j * 16 + row), a.T - 1) * a.ldx * Ty::kSize;
  typename Ty::Acc acc[NT] = {};
  for (long long q = (long long)wave * 256; q < kb; q += kFewWaves * 256) {
    i32x4 wv[4], xv[NT][4];
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const long long k = q + s * 64 + ko;
      wv[s] = load16<Ty::kSize>(w + k, kb - k);
#pragma unroll
      for (int j = 0; j < NT; ++j) xv[j][s] = load16<Ty::kSize>(x[j] + k, kb - k);
    }
#pragma unroll
    for (int s = 0; s < 4; ++s)
#pragma unroll
      for (int j = 0; j < NT; ++j) Ty::mma(wv[s], xv[j][s], acc[j]);
  }
#pragma unroll
  for (int j = 0; j < NT; ++j) red[wave][j][lane] = acc[j];
  __syncthreads();
  for (int j = wave; j < NT; j += kFewWaves) {
    typename Ty::Acc v = red[0][j][lane];
#pragma unroll
    for (int i = 1; i < kFewWaves; ++i) v += red[i][j][lane];
    const long long t = j * 16 + (lane & 15);
    const int c = r0 + 4 * (lane >> 4);
    if (t < a.T && c < a.m) {
      const typename Ty::Sum o[4] = {v[0], v[1], v[2], v[3]};
      finish<YBF16>(a, o, t, c);
    }
  }
}

// ------------------------------------------------------------------ tiles
constexpr int kTileThr = 256;
constexpr int kKB = 128;   // bytes of n per stage

// BM tokens x BN rows of W, four waves of BM/2 x BN/2. 16-byte chunk c of tile
// row r sits at slot 8 r + (c ^ ((r / 2) & 7)): the 16 rows a quarter of a wave reads
// at one chunk fall in distinct banks. The next stage's global loads are in
// flight while the current one is multiplied.
template <typename Ty, int BM, int BN, bool YBF16>
__global__ __launch_bounds__(kTileThr) void linear_tile_kernel(LinearArgs a) {
  constexpr int LX = BM * 8 / kTileThr, LW = BN * 8 / kTileThr;
  constexpr int TM = BM / 32, TN = BN / 32;   // 16 x 16 tiles of a wave
  __shared__ __align__(16) i32x4 lds[(BM + BN) * 8];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const long long t0 = (long long)blockIdx.y * BM;
  const int c0 = blockIdx.x * BN;
  const int wm = (wave >> 1) * (BM / 2), wn = (wave & 1) * (BN / 2);
  const long long kb = (long long)a.n * Ty::kSize;
  const char* xs[LX];
  const char* ws[LW];
#pragma unroll
  for (int i = 0; i < LX; ++i) {
    const int r = (i * kTileThr + tid) / 8;
    xs[i] = static_cast<const char*>(a.X) + min(t0 + r, a.T - 1) * a.ldx * Ty::kSize;
  }
#pragma unroll
  for (int i = 0; i < LW; ++i) {
    const int r = (i * kTileThr + tid) / 8;
    ws[i] = static_cast<const char*>(a.W) + (long long)min(c0 + r, a.m - 1) * a.ldw * Ty::kSize;
  }
  const int kc = (tid & 7) * 16;
  i32x4 xr[LX], wr[LW];
  auto fetch = [&](long long k0) {
    const long long k = k0 + kc;
#pragma unroll
    for (int i = 0; i < LX; ++i) xr[i] = load16<Ty::kSize>(xs[i] + k, kb - k);
#pragma unroll
    for (int i = 0; i < LW; ++i) wr[i] = load16<Ty::kSize>(ws[i] + k, kb - k);
  };
  auto slot = [](int r, int c) { return r * 8 + (c ^ ((r / 2) & 7)); };
  typename Ty::Acc acc[TM][TN] = {};
  fetch(0);
  for (long long k0 = 0; k0 < kb; k0 += kKB) {
    __syncthreads();   // the stage before is read
#pragma unroll
    for (int i = 0; i < LX; ++i) lds[slot((i * kTileThr + tid) / 8, tid & 7)] = xr[i];
#pragma unroll
    for (int i = 0; i < LW; ++i) lds[BM * 8 + slot((i * kTileThr + tid) / 8, tid & 7)] = wr[i];
    __syncthreads();
    if (k0 + kKB < kb) fetch(k0 + kKB);
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      i32x4 xf[TM], wf[TN];
      const int c = s * 4 + (lane >> 4);
#pragma unroll
      for (int i = 0; i < TM; ++i) xf[i] = lds[slot(wm + i * 16 + (lane & 15), c)];
#pragma unroll
      for (int j = 0; j < TN; ++j) wf[j] = lds[BM * 8 + slot(wn + j * 16 + (lane & 15), c)];
#pragma unroll
      for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j) Ty::mma(wf[j], xf[i], acc[i][j]);
    }
  }
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j) {
      const long long t = t0 + wm + i * 16 + (lane & 15);
      const int c = c0 + wn + j * 16 + 4 * (lane >> 4);
      if (t < a.T && c < a.m) {
        const typename Ty::Sum o[4] = {acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3]};
        finish<YBF16>(a, o, t, c);
      }
    }
}

template <typename Ty, bool YBF16>
hipError_t launch_typed(const LinearArgs& a, hipStream_t s) {
  if (a.T <= 4) {
    const int per = kRowThr / 64 * kRowsPerWave;
    const dim3 grid((unsigned)((a.m + per - 1) / per));
    if (a.T == 1) hipLaunchKernelGGL((linear_rows_kernel<Ty, 1, YBF16>), grid, dim3(kRowThr), 0, s, a);
    else if (a.T == 2) hipLaunchKernelGGL((linear_rows_kernel<Ty, 2, YBF16>), grid, dim3(kRowThr), 0, s, a);
    else hipLaunchKernelGGL((linear_rows_kernel<Ty, 4, YBF16>), grid, dim3(kRowThr), 0, s, a);
  } else if (a.T <= 64) {
    const dim3 grid((unsigned)((a.m + 15) / 16));
    if (a.T <= 16) hipLaunchKernelGGL((linear_few_kernel<Ty, 1, YBF16>), grid, dim3(kFewThr), 0, s, a);
    else if (a.T <= 32) hipLaunchKernelGGL((linear_few_kernel<Ty, 2, YBF16>), grid, dim3(kFewThr), 0, s, a);
    else hipLaunchKernelGGL((linear_few_kernel<Ty, 4, YBF16>), grid, dim3(kFewThr), 0, s, a);
  } else {
    // grid.y carries the token tiles: at most 65535 per launch
    constexpr int BM = 128, BN = 128;
    const long long step = 65535LL * BM;
    for (long long t = 0; t < a.T; t += step) {
      LinearArgs b = a;
      b.T = std::min(step, a.T - t);
      auto off = [](const void* p, long long bytes) {
        return p ? static_cast<const void*>(static_cast<const char*>(p) + bytes) : nullptr;
      };
      const int ys = YBF16 ? 2 : 4;
      b.X = off(a.X, t * a.ldx * Ty::kSize);
      b.sx = static_cast<const float*>(off(a.sx, t * 4));
      b.mul = off(a.mul, t * a.ldm * ys);
      b.res = off(a.res, t * a.ldr * ys);
      b.Y = const_cast<void*>(off(a.Y, t * a.ldy * ys));
      hipLaunchKernelGGL((linear_tile_kernel<Ty, BM, BN, YBF16>),
                         dim3((unsigned)((a.m + BN - 1) / BN), (unsigned)((b.T + BM - 1) / BM)), dim3(kTileThr),
                         0, s, b);
    }
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_linear(const LinearArgs& a, int type, hipStream_t s) {
  if (a.T <= 0 || a.m <= 0 || a.n <= 0) return hipErrorInvalidValue;
  if (a.T > 256 && linear_pipe_supported(a, type)) return launch_linear_pipe(a, type, s);
  switch (type) {
    case LINEAR_F32: return a.y_bf16 ? hipErrorInvalidValue : launch_typed<TypeF32, false>(a, s);
    case LINEAR_BF16: return a.y_bf16 ? launch_typed<TypeBf16, true>(a, s) : launch_typed<TypeBf16, false>(a, s);
    case LINEAR_I8: return a.y_bf16 ? launch_typed<TypeI8, true>(a, s) : launch_typed<TypeI8, false>(a, s);
  }
  return hipErrorInvalidValue;
}

}  // namespace poetx
