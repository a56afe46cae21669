// Which elements dropout keeps: the counter-based generator Philox 4x32-10 (Salmon,
// Moraes, Dror and Shaw, "Parallel random numbers: as easy as 1, 2, 3", 2011). The
// counter (column / 8, row, site, 0) under the seed gives 128 bits for 8 columns of a
// row, 16 to each, so that a mask is a function of the seed, the site and the place
// alone: the backward makes it again, and no split of the work shows in it. An element
// is dropped where its 16 bits lie below `threshold`, and scaled by 65536 / (65536 -
// threshold) where not, so that the mean stays whatever p was rounded to. 16 bits an
// element make 8 columns cost 20 wide products: at 32 bits the generator, not memory,
// would bound the kernels.
#pragma once

#include "poetx_internal.h"
#include "row_common.h"

namespace poetx {
namespace drop {

struct Key {
  uint32_t k0, k1;
};
// The seed of a launch: the host's, and the device's added where there is one (read by
// the kernel, so that a captured graph may be replayed with another).
__device__ __forceinline__ Key key_of(const DropArgs& d) {
  const uint64_t k = d.seed + (d.seed_dev ? *d.seed_dev : 0);
  return Key{(uint32_t)k, (uint32_t)(k >> 32)};
}

struct Bits {
  uint32_t w[4];
  // of column e of the 8
  __device__ __forceinline__ uint32_t of(int e) const { return e & 1 ? w[e / 2] >> 16 : w[e / 2] & 0xffffu; }
};
__device__ __forceinline__ Bits bits(Key k, uint32_t block, uint32_t row, uint32_t site) {
  uint32_t c0 = block, c1 = row, c2 = site, c3 = 0;
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint64_t a = (uint64_t)c0 * 0xD2511F53u, b = (uint64_t)c2 * 0xCD9E8D57u;
    c0 = (uint32_t)(b >> 32) ^ c1 ^ k.k0;
    c1 = (uint32_t)b;
    c2 = (uint32_t)(a >> 32) ^ c3 ^ k.k1;
    c3 = (uint32_t)a;
    k.k0 += 0x9E3779B9u;
    k.k1 += 0xBB67AE85u;
  }
  return Bits{{c0, c1, c2, c3}};
}

// Which of N (8, or 4: one half of the 8) elements from column c0 of a row on are kept, as bits
template <int N>
__device__ __forceinline__ uint32_t kept(const DropArgs& d, Key k, uint32_t row, int c0) {
  static_assert(N == 8 || N == 4, "whole counters or halves");
  const Bits b = bits(k, (uint32_t)c0 >> 3, row, d.site);
  const bool upper = N == 4 && (c0 & 4);
  const Bits m = upper ? Bits{{b.w[2], b.w[3], 0, 0}} : b;
  uint32_t keep = 0;
#pragma unroll
  for (int e = 0; e < N; ++e) keep |= m.of(e) >= d.threshold ? 1u << e : 0u;
  return keep;
}
// The factor 0 or scale, by selection: a dropped infinity or NaN is 0
template <int N>
__device__ __forceinline__ void apply(const DropArgs& d, uint32_t keep, float (&x)[N]) {
#pragma unroll
  for (int e = 0; e < N; ++e) x[e] = keep >> e & 1 ? x[e] * d.scale : 0.0f;
}
template <int N>
__device__ __forceinline__ void apply(const DropArgs& d, Key k, uint32_t row, int c0, float (&x)[N]) {
  apply(d, kept<N>(d, k, row, c0), x);
}

}  // namespace drop
}  // namespace poetx
