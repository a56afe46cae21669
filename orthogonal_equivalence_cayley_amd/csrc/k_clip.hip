// The global norm over many gradient tensors, and their scaling by it.
//
//   norm = sqrt(sum of all g^2),  c = min(1, max_norm / (norm + 1e-6)),
//   out = rnd(c g)
//
// Bound by memory. The norm has to be known before the first product, so all
// gradients are read twice and written once. Two launches for up to kClipMax
// tensors: partial sums of squares, one per workgroup, in 64 bits (no overflow for
// any fp32 gradient, and an order that does not show in the fp32 norm but in the
// rarest cases), then the products, where every workgroup adds up the few
// partial sums itself, in the same order, instead of waiting for a launch between.
// Workgroups take chunks of 8192 elements, all loads of a chunk out at once.
// Measured: 204 tensors of 1.4 GB in all 730 us (sums 6.1 TB/s, products 5.4
// TB/s); 16 of 20 MB 7.3 + 9.8 us. 2048 workgroups to a launch instead of 1024:
// 752 us.
#include <algorithm>

#include "poetx_internal.h"

namespace poetx {
namespace {

constexpr int kThr = 256;
constexpr int kChunk = 8192;        // elements of one step of a workgroup
constexpr int kGrid = 1024;         // workgroups of one launch
constexpr long long kCached = 256LL << 20;   // bytes of the cache in front of the memory
constexpr int kFold = 4096;         // partial sums a workgroup adds up itself

__device__ __forceinline__ float bf(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ uint32_t rnd(float v) {
  return __builtin_bit_cast(uint16_t, static_cast<__bf16>(v));
}

// 16 bytes at any element alignment
struct __attribute__((packed, aligned(2))) Vec16 {
  uint32_t w[4];
};
typedef uint32_t u32x4 __attribute__((ext_vector_type(4), aligned(2)));

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

__device__ __forceinline__ void add_squares(const Vec16& v, bool bf16, double& s) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if (bf16) {
      const double lo = bf(v.w[k] & 0xffffu), hi = bf(v.w[k] >> 16);
      s += lo * lo;
      s += hi * hi;
    } else {
      const double x = __uint_as_float(v.w[k]);
      s += x * x;
    }
  }
}

// VECS vectors of each thread in one go where the chunk is whole
template <bool BF16>
__device__ __forceinline__ void sum_chunk(const void* p, long long i0, int n, double& s) {
  constexpr int N = BF16 ? 8 : 4, VECS = kChunk / (kThr * N);
  const char* g = static_cast<const char*>(p) + i0 * (16 / N);
  if (n == kChunk) {
    Vec16 v[VECS];
#pragma unroll
    for (int k = 0; k < VECS; ++k) v[k] = *reinterpret_cast<const Vec16*>(g + (k * kThr + threadIdx.x) * 16);
#pragma unroll
    for (int k = 0; k < VECS; ++k) add_squares(v[k], BF16, s);
    return;
  }
  const int whole = n / N;
  for (int k = threadIdx.x; k < whole; k += kThr) add_squares(*reinterpret_cast<const Vec16*>(g + k * 16), BF16, s);
  const int k = whole * N + threadIdx.x;
  if (k < n) {
    const double x = BF16 ? bf(reinterpret_cast<const uint16_t*>(g)[k]) : reinterpret_cast<const float*>(g)[k];
    s += x * x;
  }
}

__global__ __launch_bounds__(kThr) void sum_squares_kernel(ClipBatch b, int chunks, double* part) {
  double s = 0.0;
  for (int q = blockIdx.x; q < chunks; q += gridDim.x) {
    const ClipEntry& e = b.e[entry_of(b, q)];
    const long long i0 = (long long)(q - e.chunk0) * kChunk;
    const int n = (int)min((long long)kChunk, e.n - i0);
    if (e.bf16) sum_chunk<true>(e.g, i0, n, s);
    else sum_chunk<false>(e.g, i0, n, s);
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

__device__ __forceinline__ Vec16 scaled(Vec16 v, bool bf16, float c) {
#pragma unroll
  for (int k = 0; k < 4; ++k)
    v.w[k] = bf16 ? rnd(c * bf(v.w[k] & 0xffffu)) | rnd(c * bf(v.w[k] >> 16)) << 16
                  : __float_as_uint(c * __uint_as_float(v.w[k]));
  return v;
}

template <bool BF16>
__device__ __forceinline__ void clip_chunk(const void* p, void* q, long long i0, int n, float c,
                                           bool stream) {
  constexpr int N = BF16 ? 8 : 4, VECS = kChunk / (kThr * N);
  const char* g = static_cast<const char*>(p) + i0 * (16 / N);
  char* o = static_cast<char*>(q) + i0 * (16 / N);
  if (n == kChunk) {
    Vec16 v[VECS];
#pragma unroll
    for (int k = 0; k < VECS; ++k) v[k] = *reinterpret_cast<const Vec16*>(g + (k * kThr + threadIdx.x) * 16);
#pragma unroll
    for (int k = 0; k < VECS; ++k) {
      const Vec16 r = scaled(v[k], BF16, c);
      char* to = o + (k * kThr + threadIdx.x) * 16;
      if (stream) __builtin_nontemporal_store(u32x4{r.w[0], r.w[1], r.w[2], r.w[3]}, reinterpret_cast<u32x4*>(to));
      else *reinterpret_cast<Vec16*>(to) = r;
    }
    return;
  }
  const int whole = n / N;
  for (int k = threadIdx.x; k < whole; k += kThr)
    *reinterpret_cast<Vec16*>(o + k * 16) = scaled(*reinterpret_cast<const Vec16*>(g + k * 16), BF16, c);
  const int k = whole * N + threadIdx.x;
  if (k < n) {
    if (BF16) reinterpret_cast<uint16_t*>(o)[k] = (uint16_t)rnd(c * bf(reinterpret_cast<const uint16_t*>(g)[k]));
    else reinterpret_cast<float*>(o)[k] = c * reinterpret_cast<const float*>(g)[k];
  }
}

// Chunks from the last to the first: what the sums read last is what the caches
// still hold.
__global__ __launch_bounds__(kThr) void clip_kernel(ClipBatch b, int chunks, const double* part, int nparts,
                                                    double max_norm, float* norm_out, bool stream) {
  double s = 0.0;
  for (int i = threadIdx.x; i < nparts; i += kThr) s += part[i];
  const double norm = sqrt(block_sum(s));
  if (norm_out && blockIdx.x == 0 && threadIdx.x == 0) *norm_out = (float)norm;
  const double ratio = max_norm / (norm + 1e-6);
  const float c = ratio >= 1.0 ? 1.0f : (float)ratio;   // NaN stays NaN
  for (int q = chunks - 1 - (int)blockIdx.x; q >= 0; q -= gridDim.x) {
    const ClipEntry& e = b.e[entry_of(b, q)];
    if (c == 1.0f && e.g == e.out) continue;   // in place and within the limit: nothing changes
    const long long i0 = (long long)(q - e.chunk0) * kChunk;
    const int n = (int)min((long long)kChunk, e.n - i0);
    if (e.bf16) clip_chunk<true>(e.g, e.out, i0, n, c, stream);
    else clip_chunk<false>(e.g, e.out, i0, n, c, stream);
  }
}

// Fills b with the items from i0 on that fit one launch, backward from the one
// before i0 with BACK (still in their order inside b); returns how many it took.
// `chunks`: their chunks.
template <bool BACK>
int fill(const ClipItem* items, int count, int i0, ClipBatch& b, long long& chunks) {
  b.n = 0;
  chunks = 0;
  int took = 0, first = i0;
  // the range first, then the entries in order
  long long total = 0;
  for (int n = 0; BACK ? i0 - took > 0 : i0 + took < count; ++took) {
    const ClipItem& it = items[BACK ? i0 - took - 1 : i0 + took];
    if (it.n <= 0) continue;
    total += (it.n + kChunk - 1) / kChunk;
    if (n == kClipMax || total > 0x7fffffffLL) break;
    ++n;
  }
  if (BACK) first = i0 - took;
  for (int i = first; i < first + took; ++i) {
    const ClipItem& it = items[i];
    if (it.n <= 0) continue;
    b.e[b.n++] = ClipEntry{it.g, it.out, it.n, (int)chunks, it.bf16};
    chunks += (it.n + kChunk - 1) / kChunk;
  }
  return took;
}

}  // namespace

long long clip_parts(long long count) { return (count + kClipMax - 1) / kClipMax * kGrid; }

hipError_t launch_clip(const ClipItem* items, int count, double max_norm, double* part, float* norm_out,
                       bool write, hipStream_t s) {
  ClipBatch b;
  long long chunks = 0;
  int nparts = 0;
  for (int i = 0; i < count;) {
    i += fill<false>(items, count, i, b, chunks);
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
  // Results that the caches cannot hold for their reader go past them: 1.4 GB
  // in 730 instead of 770 us (the sums of the next step find fewer lines to write
  // back). A set that fits stays: it is read next, and 20 MB take 17 us either way.
  long long bytes = 0;
  for (int i = 0; i < count; ++i) bytes += items[i].n * (items[i].bf16 ? 2 : 4);
  const bool stream = bytes > kCached;
  bool first = true;
  for (int i = count; i > 0 || first;) {
    i -= fill<true>(items, count, i, b, chunks);
    if (!b.n && !first) continue;
    if (!write) chunks = 0;   // the norm only
    const int grid = (int)std::max<long long>(1, std::min<long long>(chunks, kGrid));
    hipLaunchKernelGGL(clip_kernel, dim3(grid), dim3(kThr), 0, s, b, (int)chunks, part, nparts, max_norm,
                       first ? norm_out : nullptr, stream);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    first = false;
    if (!write) break;
  }
  return hipSuccess;
}

}  // namespace poetx
