// The merged-weight product (k_linear.hip) where 256 x 256 tiles would leave CUs
// idle: smaller tiles, one to a workgroup of four waves, with a ring of NS LDS
// stages of 128 bytes of every operand row filled by direct-to-LDS loads. One
// barrier a stage, in its middle: the products of a stage's first half run beside
// the LDS reads of its second, those of the second half beside the loads of the
// stage that takes its place and the reads of the next one's first half. (Reads,
// loads and products one after the other: 31 against 22 us a 1024 x 2048 x 2048
// bf16 product in 128 x 128 tiles; more stages in flight changed nothing.) With
// KS = 2 a second group of four waves takes the other half of n, for grids that
// leave CUs idle (bf16, the weight from memory: 16 x 2048 x 5632 10.8 -> 8.9 us, 16 x
// 4096 x 4096 17.5 -> 14.9 us), and with PART several workgroups share n and leave
// their sums to linear_join (k_linear.hip).
//
// Rows past the last token or weight row are clamped to it (not stored).
// Requirements (linear_ring_supported): n and row strides of whole 16 bytes.
#include <algorithm>
#include <type_traits>

#include "linear_common.h"

namespace poetx {
namespace {

using namespace lin;

constexpr int kThr = 256;
constexpr int kKB = 128;          // bytes of a row per stage

// 16 bytes per lane from base + off + k (below `bytes`) to lane * 16 behind `to`
__device__ __forceinline__ void load_lds(const char* base, int bytes, unsigned char* to, uint32_t off, int k) {
  const __amdgpu_buffer_rsrc_t rs =
      __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(base), (short)0, bytes, 0x00020000);
  __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (__attribute__((address_space(3))) void*)to, 16, off, k, 0, 0);
}

// TAIL: n is no multiple of 128 bytes, or its stages none of KS (its own kernel: the
// extra work costs the others 10 %)
template <typename Ty, int BM, int BN, int NS, int KS, bool TAIL, bool PART, bool YBF16>
__global__ __launch_bounds__(kThr * KS)
__attribute__((amdgpu_waves_per_eu(std::max(2, KS), std::max(2, KS))))
void linear_ring_kernel(LinearArgs p) {
  constexpr int LX = BM / 32, LW = BN / 32;    // loads of a lane per stage: 32 rows each
  constexpr int TM = BM / 32, TN = BN / 32;    // 16 x 16 tiles of a wave (2 x 2 waves)
  constexpr int STAGE = (BM + BN) * kKB;
  static_assert(NS * (LX + LW) <= 63, "loads in flight");
  extern __shared__ __align__(16) unsigned char lds[];
  const int tid = threadIdx.x & 255, lane = tid & 63;
  const int grp_k = KS == 1 ? 0 : __builtin_amdgcn_readfirstlane(threadIdx.x >> 8);
  unsigned char* const ring = lds + grp_k * NS * STAGE;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = (wave >> 1) * (BM / 2), wn = (wave & 1) * (BN / 2);

  int m0, n0;
  if (!tile_origin(p.T, p.m, BM, BN, m0, n0)) return;
  const int lda = (int)(p.ldx * Ty::kSize), ldb = (int)(p.ldw * Ty::kSize);
  const int lr = tid / 8;
  const uint32_t lc = (uint32_t)((tid & 7) ^ ((lr / 2) & 7)) * 16;
  const int rx = (int)min((long long)BM, p.T - m0), rw = min(BN, p.m - n0);   // rows that exist
  uint32_t vx[LX], vw[LW];
#pragma unroll
  for (int i = 0; i < LX; ++i) vx[i] = (uint32_t)(min(i * 32 + lr, rx - 1) * lda) + lc;
#pragma unroll
  for (int i = 0; i < LW; ++i) vw[i] = (uint32_t)(min(i * 32 + lr, rw - 1) * ldb) + lc;
  const char* const bx = static_cast<const char*>(p.X) + (long long)m0 * lda;
  const char* const bw = static_cast<const char*>(p.W) + (long long)n0 * ldb;
  const long long kb = (long long)p.n * Ty::kSize;
  const int stages = (int)((kb + kKB - 1) / kKB);
  const int groups = PART ? KS * p.splits : KS;
  const int nk = (stages + groups - 1) / groups;   // stages of a group, a piece of n in a row
  const int k0 = ((PART ? (int)blockIdx.y * KS : 0) + grp_k) * nk * kKB;
  // With TAIL a group's last stages may be cut by the row's end or lie behind it:
  // lanes whose chunks are gone load the row's stage from its start instead (a stage
  // behind the end: the row's first), and write zeros over it once it landed
  auto ends = [&](int s) __attribute__((always_inline)) { return k0 + (long long)(s + 1) * kKB > kb; };
  auto gone = [&](int s) __attribute__((always_inline)) { return k0 + (long long)s * kKB + lc >= kb; };

  // stage s (past the end: the last one again, into a buffer nobody reads)
  auto issue = [&](int s, int buf) __attribute__((always_inline)) {
    s = min(s, nk - 1);
    int k = k0 + s * kKB;
    uint32_t back = 0;
    if (TAIL && ends(s)) {
      back = gone(s) ? lc : 0;
      k = k < kb ? k : 0;
    }
    unsigned char* st = ring + buf * STAGE + wave * 1024;
#pragma unroll
    for (int i = 0; i < LX; ++i) load_lds(bx, rx * lda, st + i * 4096, vx[i] - back, k);
#pragma unroll
    for (int i = 0; i < LW; ++i) load_lds(bw, rw * ldb, st + BM * kKB + i * 4096, vw[i] - back, k);
  };
  auto clear = [&](int s, int buf) __attribute__((always_inline)) {
    if (!gone(s)) return;
    unsigned char* st = ring + buf * STAGE + tid * 16;
#pragma unroll
    for (int i = 0; i < LX + LW; ++i) *reinterpret_cast<i32x4*>(st + i * 4096) = i32x4{0, 0, 0, 0};
  };
  // chunk c of row r at slot 8 r + (c ^ ((r / 2) & 7))
  auto frag = [&](const unsigned char* st, int r, int c) __attribute__((always_inline)) {
    return *reinterpret_cast<const i32x4*>(st + r * kKB + ((c ^ ((r / 2) & 7)) * 16));
  };

  typename Ty::Acc acc[TM][TN] = {};
  i32x4 xf[2][TM], wf[2][TN];
  // fragments of the first (q = 0) or second 64-byte slab of a stage
  auto read = [&](int buf, int q) __attribute__((always_inline)) {
    const unsigned char* st = ring + buf * STAGE;
    const int c = q * 4 + (lane >> 4);
#pragma unroll
    for (int i = 0; i < TM; ++i) xf[q][i] = frag(st, wm + i * 16 + (lane & 15), c);
#pragma unroll
    for (int j = 0; j < TN; ++j) wf[q][j] = frag(st + BM * kKB, wn + j * 16 + (lane & 15), c);
  };
  auto multiply = [&](int q) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j) Ty::mma(wf[q][j], xf[q][i], acc[i][j]);
  };
  // The reads (and loads) of a half stage go out between its products
  constexpr int PM = std::max(1, TM * TN * (Ty::kSize == 4 ? 4 : 1) / (TM + TN));   // products a read
  constexpr int PL = (LX + LW + TM + TN - 1) / (TM + TN);                           // loads a read
  auto spread = [](auto loads) __attribute__((always_inline)) {
#pragma unroll
    for (int r = 0; r < TM + TN; ++r) {
      __builtin_amdgcn_sched_group_barrier(0x008, PM, 0);
      if (decltype(loads)::value) __builtin_amdgcn_sched_group_barrier(0x020, PL, 0);
      __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
    }
  };
#pragma unroll
  for (int s = 0; s < NS; ++s) issue(s, s);
  vm_wait<(NS - 1) * (LX + LW)>();   // this wave's part of stage 0 landed
  if (TAIL && ends(0)) clear(0, 0);
  lds_sync();                        // and everyone's
  read(0, 0);
  int buf = 0;
  for (int s = 0; s < nk; ++s) {
    const int next = buf + 1 == NS ? 0 : buf + 1;
    read(buf, 1);
    multiply(0);
    spread(std::false_type{});
    __builtin_amdgcn_sched_barrier(0);
    vm_wait<(NS - 2) * (LX + LW)>();
    if (TAIL && s + 1 < nk && ends(s + 1)) clear(s + 1, next);
    lds_sync();   // stage s + 1 landed, and nobody reads stage s any more
    issue(s + NS, buf);
    read(next, 0);
    multiply(1);
    spread(std::true_type{});
    __builtin_amdgcn_sched_barrier(0);
    buf = next;
  }
  // the last loads went into buffers nobody reads: let them land before the
  // workgroup's LDS is released
  vm_wait<0>();
  if constexpr (KS > 1) {
    typedef typename Ty::Acc Acc;
    static_assert((KS - 1) * BM * BN * 4 <= KS * NS * STAGE, "sums fit where the stages were");
    __syncthreads();   // every group's loads landed
    Acc* const sums = reinterpret_cast<Acc*>(lds);
    if (grp_k > 0) {
#pragma unroll
      for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j) sums[(((grp_k - 1) * TM + i) * TN + j) * kThr + tid] = acc[i][j];
    }
    __syncthreads();
    if (grp_k > 0) return;
#pragma unroll
    for (int g = 0; g < KS - 1; ++g)
#pragma unroll
      for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j) acc[i][j] += sums[((g * TM + i) * TN + j) * kThr + tid];
  }
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j) {
      const long long t = (long long)m0 + wm + i * 16 + (lane & 15);
      const int c = n0 + wn + j * 16 + 4 * (lane >> 4);
      if (t < p.T && c < p.m) {
        if constexpr (PART) {
          store_part<Ty>(p, blockIdx.y, t, c, acc[i][j]);
        } else {
          const typename Ty::Sum o[4] = {acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3]};
          finish<YBF16>(p, o, t, c);
        }
      }
    }
}

template <typename Ty, int BM, int BN, int NS, int KS, bool YBF16, bool PART = false>
hipError_t tiles(const LinearArgs& a, hipStream_t s) {
  const dim3 grid((unsigned)tile_grid(a.T, a.m, BM, BN), PART ? (unsigned)a.splits : 1u);
  constexpr int lds = KS * NS * (BM + BN) * kKB;
  if ((long long)a.n * Ty::kSize % ((long long)kKB * KS * (PART ? a.splits : 1)))
    hipLaunchKernelGGL((linear_ring_kernel<Ty, BM, BN, NS, KS, true, PART, YBF16>), grid, dim3(kThr * KS), lds, s, a);
  else
    hipLaunchKernelGGL((linear_ring_kernel<Ty, BM, BN, NS, KS, false, PART, YBF16>), grid, dim3(kThr * KS), lds, s, a);
  return hipGetLastError();
}

template <typename Ty, bool YBF16>
hipError_t launch(const LinearArgs& a, int tile, hipStream_t s) {
  switch (tile) {
    case LINEAR_TILE_128: return tiles<Ty, 128, 128, 2, 1, YBF16>(a, s);
    case LINEAR_TILE_128x64: return tiles<Ty, 128, 64, 3, 1, YBF16>(a, s);
    case LINEAR_TILE_64: return tiles<Ty, 64, 64, 4, 1, YBF16>(a, s);
    case LINEAR_TILE_32x64: return tiles<Ty, 32, 64, 4, 1, YBF16>(a, s);
    case LINEAR_TILE_32: return tiles<Ty, 32, 32, 4, 1, YBF16>(a, s);
    case LINEAR_TILE_32_SPLIT: return tiles<Ty, 32, 32, 4, 2, YBF16>(a, s);
  }
  return hipErrorInvalidValue;
}

}  // namespace

bool linear_ring_supported(const LinearArgs& a, int type) {
  const int es = type == LINEAR_F32 ? 4 : type == LINEAR_BF16 ? 2 : 1;
  if ((long long)a.n * es % 16 || a.ldx * es % 16 || a.ldw * es % 16) return false;
  if (((uintptr_t)a.X | (uintptr_t)a.W) & 15) return false;
  // 256 rows within 32-bit offsets
  return a.ldx * es * 256 < (1LL << 31) && a.ldw * es * 256 < (1LL << 31);
}

hipError_t launch_linear_ring(const LinearArgs& a, int type, int tile, hipStream_t s) {
  if (a.splits > 1) {   // sums only: the type of Y does not matter
    switch (type) {
      case LINEAR_F32: return tiles<TypeF32, 32, 32, 4, 2, false, true>(a, s);
      case LINEAR_BF16: return tiles<TypeBf16, 32, 32, 4, 2, false, true>(a, s);
    }
    return tiles<TypeI8, 32, 32, 4, 2, false, true>(a, s);
  }
  switch (type) {
    case LINEAR_F32: return launch<TypeF32, false>(a, tile, s);
    case LINEAR_BF16: return a.y_bf16 ? launch<TypeBf16, true>(a, tile, s) : launch<TypeBf16, false>(a, tile, s);
  }
  return a.y_bf16 ? launch<TypeI8, true>(a, tile, s) : launch<TypeI8, false>(a, tile, s);
}

}  // namespace poetx
