// The global norm over many gradient tensors, and their scaling by it.
//
//   norm = sqrt(sum of all g^2),  c = min(1, max_norm / (norm + 1e-6)),
//   out = rnd(c g)
//
// Bound by memory. The norm has to be known before the first product, so all
// gradients are read twice and written once: the second read comes from the
// caches where they hold the set (256 MB behind the eight L2s). Two launches for
// up to kClipMax tensors: partial sums of squares, one per workgroup, in 64
// bits (no overflow for any fp32 gradient, and no order that shows in the fp32
// result's rounding but in the rarest cases), then the products, where every
// workgroup adds up the few partial sums itself, in the same order, instead of
// waiting for a launch between.
#include <algorithm>

#include "poetx_internal.h"

namespace poetx {
namespace {

constexpr int kThr = 256;
constexpr int kChunk = 8192;        // elements of one step of a workgroup
constexpr int kGrid = 1024;         // workgroups of one launch
constexpr int kFold = 4096;         // partial sums a workgroup adds up itself

__device__ __forceinline__ float bf(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ uint32_t rnd(float v) {
  return __builtin_bit_cast(uint16_t, static_cast<__bf16>(v));
}

__device__ __forceinline__ double block_sum(double v) {
  __shared__ double red[kThr / 64];
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  v = red[0];
#pragma unroll
  for (int i = 1; i < kThr / 64; ++i) v += red[i];
  return v;
}

// entry of chunk q: the last whose first chunk is at or before it
__device__ __forceinline__ int entry_of(const ClipBatch& b, int q) {
  int lo = 0, hi = b.n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (b.e[mid].chunk0 <= q) lo = mid;
    else hi = mid;
  }
  return lo;
}

__global__ __launch_bounds__(kThr) void sum_squares_kernel(ClipBatch b, int chunks, double* part) {
  double s = 0.0;
  for (int q = blockIdx.x; q < chunks; q += gridDim.x) {
    const ClipEntry& e = b.e[entry_of(b, q)];
    const long long i0 = (long long)(q - e.chunk0) * kChunk;
    const int n = (int)min((long long)kChunk, e.n - i0);
    if (e.bf16) {
      const uint16_t* g = static_cast<const uint16_t*>(e.g) + i0;
      for (int i = threadIdx.x * 8; i < n; i += kThr * 8) {
        if (i + 8 <= n) {
          uint4 v;
          __builtin_memcpy(&v, g + i, 16);
          const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const double lo = bf(w[k] & 0xffffu), hi = bf(w[k] >> 16);
            s += lo * lo;
            s += hi * hi;
          }
        } else {
          for (int k = i; k < n; ++k) {
            const double x = bf(g[k]);
            s += x * x;
          }
        }
      }
    } else {
      const float* g = static_cast<const float*>(e.g) + i0;
#pragma unroll 4
      for (int i = threadIdx.x * 4; i < n; i += kThr * 4) {
        if (i + 4 <= n) {
          float4 v;
          __builtin_memcpy(&v, g + i, 16);
          s += (double)v.x * v.x;
          s += (double)v.y * v.y;
          s += (double)v.z * v.z;
          s += (double)v.w * v.w;
        } else {
          for (int k = i; k < n; ++k) s += (double)g[k] * g[k];
        }
      }
    }
  }
  s = block_sum(s);
  if (threadIdx.x == 0) part[blockIdx.x] = s;
}

// more partial sums than the products' workgroups add up themselves: one value
__global__ __launch_bounds__(kThr) void fold_kernel(double* part, int n) {
  double s = 0.0;
  for (int i = threadIdx.x; i < n; i += kThr) s += part[i];
  s = block_sum(s);   // its barrier: every read is over before the write
  if (threadIdx.x == 0) part[0] = s;
}

__global__ __launch_bounds__(kThr) void clip_kernel(ClipBatch b, int chunks, const double* part, int nparts,
                                                    double max_norm, float* norm_out) {
  double s = 0.0;
  for (int i = threadIdx.x; i < nparts; i += kThr) s += part[i];
  const double norm = sqrt(block_sum(s));
  if (norm_out && blockIdx.x == 0 && threadIdx.x == 0) *norm_out = (float)norm;
  const double ratio = max_norm / (norm + 1e-6);
  const float c = ratio >= 1.0 ? 1.0f : (float)ratio;   // NaN stays NaN
  for (int q = blockIdx.x; q < chunks; q += gridDim.x) {
    const ClipEntry& e = b.e[entry_of(b, q)];
    if (c == 1.0f && e.g == e.out) continue;   // in place and within the limit: nothing changes
    const long long i0 = (long long)(q - e.chunk0) * kChunk;
    const int n = (int)min((long long)kChunk, e.n - i0);
    if (e.bf16) {
      const uint16_t* g = static_cast<const uint16_t*>(e.g) + i0;
      uint16_t* o = static_cast<uint16_t*>(e.out) + i0;
      for (int i = threadIdx.x * 8; i < n; i += kThr * 8) {
        if (i + 8 <= n) {
          uint32_t w[4];
          __builtin_memcpy(w, g + i, 16);
#pragma unroll
          for (int k = 0; k < 4; ++k) w[k] = rnd(c * bf(w[k] & 0xffffu)) | rnd(c * bf(w[k] >> 16)) << 16;
          __builtin_memcpy(o + i, w, 16);
        } else {
          for (int k = i; k < n; ++k) o[k] = (uint16_t)rnd(c * bf(g[k]));
        }
      }
    } else {
      const float* g = static_cast<const float*>(e.g) + i0;
      float* o = static_cast<float*>(e.out) + i0;
#pragma unroll 4
      for (int i = threadIdx.x * 4; i < n; i += kThr * 4) {
        if (i + 4 <= n) {
          float v[4];
          __builtin_memcpy(v, g + i, 16);
#pragma unroll
          for (int k = 0; k < 4; ++k) v[k] *= c;
          __builtin_memcpy(o + i, v, 16);
        } else {
          for (int k = i; k < n; ++k) o[k] = c * g[k];
        }
      }
    }
  }
}

// fills b from items [i0, ..) and returns how many it took; `chunks`: their chunks
int fill(const ClipItem* items, int count, int i0, ClipBatch& b, long long& chunks) {
  b.n = 0;
  chunks = 0;
  int i = i0;
  for (; i < count && b.n < kClipMax; ++i) {
    const ClipItem& it = items[i];
    if (it.n <= 0) continue;
    const long long c = (it.n + kChunk - 1) / kChunk;
    if (chunks + c > 0x7fffffffLL) break;
    b.e[b.n++] = ClipEntry{it.g, it.out, it.n, (int)chunks, it.bf16};
    chunks += c;
  }
  return i - i0;
}

}  // namespace

long long clip_parts(long long count) { return (count + kClipMax - 1) / kClipMax * kGrid; }

hipError_t launch_clip(const ClipItem* items, int count, double max_norm, double* part, float* norm_out,
                       bool write, hipStream_t s) {
  ClipBatch b;
  long long chunks = 0;
  int nparts = 0;
  for (int i = 0; i < count;) {
    i += fill(items, count, i, b, chunks);
    if (!b.n) continue;
    const int grid = (int)std::min<long long>(chunks, kGrid);
    hipLaunchKernelGGL(sum_squares_kernel, dim3(grid), dim3(kThr), 0, s, b, (int)chunks, part + nparts);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    nparts += grid;
  }
  if (nparts > kFold) {
    hipLaunchKernelGGL(fold_kernel, dim3(1), dim3(kThr), 0, s, part, nparts);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    nparts = 1;
  }
  bool first = true;
  for (int i = 0; i < count || first;) {
    i += fill(items, count, i, b, chunks);
    if (!b.n && !first) continue;
    if (!write) chunks = 0;   // the norm only
    const int grid = (int)std::max<long long>(1, std::min<long long>(chunks, kGrid));
    hipLaunchKernelGGL(clip_kernel, dim3(grid), dim3(kThr), 0, s, b, (int)chunks, part, nparts, max_norm,
                       first ? norm_out : nullptr);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    first = false;
    if (!write) break;
  }
  return hipSuccess;
}

}  // namespace poetx
