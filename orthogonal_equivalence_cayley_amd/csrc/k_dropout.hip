// Dropout, alone or into the residual stream: y = rnd(keep(t, c) ? x scale : 0) or
// rnd(r + ...), the mask from the generator of dropout_common.h and never stored. Its
// backward is the same call on the gradient.
//
// Bound by memory: x (and r) read and y written once. A thread takes kVecs vectors of
// 16 bytes a workgroup's width apart, all their loads out before the generator runs
// (some 60 cycles of integer products a vector beside them). 16384 x 2048 bf16 with the
// residual 32.4 us (6.2 TB/s), 16384 x 5632 without 65.7 us (5.6 TB/s).
#include <algorithm>

#include "dropout_common.h"
#include "row_common.h"

namespace poetx {
namespace {

using namespace row;

constexpr int kThr = 256;
constexpr int kVecs = 4;

// i / d for 0 <= i < 2^31: (i m) >> shift with m = ceil(2^shift / d), shift = 31 + ceil(log2 d)
struct Divide {
  uint32_t m;
  int shift;
};
Divide divide_by(uint32_t d) {
  int l = 0;
  while ((1u << l) < d) ++l;
  return Divide{(uint32_t)(((1ull << (31 + l)) + d - 1) / d), 31 + l};
}

template <typename E, bool WHOLE, bool RES>
__global__ __launch_bounds__(kThr) void dropout_kernel(DropoutArgs a, int nv, uint32_t count, Divide by) {
  constexpr int N = 16 / sizeof(E);
  const drop::Key key = drop::key_of(a.drop);
  const bool full = a.dim >= N;
  const uint32_t first = blockIdx.x * (uint32_t)(kThr * kVecs) + threadIdx.x;
  E x[kVecs][N], r[kVecs][N];
  uint32_t row[kVecs];
  int col[kVecs];
#pragma unroll
  for (int u = 0; u < kVecs; ++u) {
    const uint32_t i = first + u * kThr;
    if (i >= count) break;
    row[u] = (uint32_t)(((uint64_t)i * by.m) >> by.shift);
    col[u] = (int)(i - row[u] * (uint32_t)nv) * N;
    load_raw<WHOLE>(static_cast<const E*>(a.X) + row[u] * a.ldx + col[u], a.dim - col[u], full, x[u]);
    if constexpr (RES) load_raw<WHOLE>(static_cast<const E*>(a.R) + row[u] * a.ldr + col[u], a.dim - col[u], full, r[u]);
  }
#pragma unroll
  for (int u = 0; u < kVecs; ++u) {
    if (first + u * kThr >= count) break;
    float y[N];
#pragma unroll
    for (int e = 0; e < N; ++e) y[e] = to_f(x[u][e]);
    drop::apply(a.drop, key, a.row0 + row[u], col[u], y);
    if constexpr (RES) {
#pragma unroll
      for (int e = 0; e < N; ++e) y[e] += to_f(r[u][e]);
    }
    store_n<WHOLE>(static_cast<E*>(a.Y) + row[u] * a.ldy + col[u], a.dim - col[u], y);
  }
}

template <typename E>
hipError_t run(DropoutArgs a, hipStream_t s) {
  constexpr int N = 16 / sizeof(E);
  const int nv = (a.dim + N - 1) / N;
  const Divide by = divide_by((uint32_t)nv);
  // vectors of a launch are counted in 31 bits
  const long long rows = std::max(1LL, (1LL << 30) / nv);
  const long long T = a.T;
  const E* const x = static_cast<const E*>(a.X);
  const E* const r = static_cast<const E*>(a.R);
  E* const y = static_cast<E*>(a.Y);
  for (long long t = 0; t < T; t += rows) {
    a.T = std::min(rows, T - t);
    a.X = x + t * a.ldx;
    a.R = r ? r + t * a.ldr : nullptr;
    a.Y = y + t * a.ldy;
    a.row0 = (uint32_t)t;
    const uint32_t count = (uint32_t)(a.T * nv);
    const dim3 grid((count + kThr * kVecs - 1) / (kThr * kVecs));
    const bool whole = a.dim % N == 0;
    if (whole && a.R) hipLaunchKernelGGL((dropout_kernel<E, true, true>), grid, dim3(kThr), 0, s, a, nv, count, by);
    else if (whole) hipLaunchKernelGGL((dropout_kernel<E, true, false>), grid, dim3(kThr), 0, s, a, nv, count, by);
    else if (a.R) hipLaunchKernelGGL((dropout_kernel<E, false, true>), grid, dim3(kThr), 0, s, a, nv, count, by);
    else hipLaunchKernelGGL((dropout_kernel<E, false, false>), grid, dim3(kThr), 0, s, a, nv, count, by);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

hipError_t launch_dropout(const DropoutArgs& a, int bf16, hipStream_t s) {
  if (a.dim <= 0 || a.dim > kNormMaxDim) return hipErrorInvalidValue;
  return bf16 ? run<uint16_t>(a, s) : run<float>(a, s);
}

}  // namespace poetx
