// Launch shapes of the calls that train around the linears at their documented limits. The
// runtime's launch entry is defined here and takes its place, so nothing runs: it writes down
// each grid. A dispatch counts threads in 32 bits, so a launch of 2^32 threads or more along
// an axis would be refused by the runtime.
#include <hip/hip_runtime.h>

#include <cstdint>
#include <cstdio>
#include <vector>

#include "../../orthogonal_equivalence_cayley_amd/csrc/poetx_internal.h"
#include "poetx.h"

static int failures = 0;
static const char* where = "";
static long long c_T, c_m, c_n, c_type;
#define EXPECT(cond)                                                                            \
  do {                                                                                          \
    if (!(cond)) {                                                                              \
      if (failures < 40)                                                                        \
        std::printf("FAILED line %d: %s (%s T=%lld m=%lld n=%lld type=%lld)\n", __LINE__, #cond, \
                    where, c_T, c_m, c_n, c_type);                                              \
      ++failures;                                                                               \
    }                                                                                           \
  } while (0)

struct Launch {
  dim3 grid, block;
  size_t lds;
};
static std::vector<Launch> launches;
static Launch pending;

extern "C" {
hipError_t __hipPushCallConfiguration(dim3 grid, dim3 block, size_t lds, hipStream_t) {
  pending = Launch{grid, block, lds};
  return hipSuccess;
}
hipError_t __hipPopCallConfiguration(dim3* grid, dim3* block, size_t* lds, hipStream_t* s) {
  *grid = pending.grid;
  *block = pending.block;
  *lds = pending.lds;
  *s = nullptr;
  return hipSuccess;
}
hipError_t hipLaunchKernel(const void*, dim3 grid, dim3 block, void**, size_t lds, hipStream_t) {
  launches.push_back(Launch{grid, block, lds});
  return hipSuccess;
}
hipError_t hipGetLastError(void) { return hipSuccess; }
}

namespace {

char* dev(uintptr_t i) { return reinterpret_cast<char*>(i << 58); }
float* fdev(uintptr_t i) { return reinterpret_cast<float*>(dev(i)); }

void shapes_ok() {
  EXPECT(!launches.empty());
  for (const Launch& l : launches) {
    const uint32_t threads = l.block.x * l.block.y * l.block.z;
    EXPECT(threads >= 64 && threads <= 1024 && l.lds <= 160 * 1024);
    EXPECT(l.grid.x >= 1 && (uint64_t)l.grid.x * l.block.x < (1ull << 32));
    EXPECT(l.grid.y >= 1 && (uint64_t)l.grid.y * l.block.y <= (1ull << 20));
    EXPECT(l.grid.z == 1);
  }
  launches.clear();
}

constexpr int64_t kMaxT = 0x7fffffff;

void norms() {
  for (int type : {POETX_FP32, POETX_BF16})
    for (int dim : {1, 8, 64, 100, 1000, 1024, 2048, 4096, 5000, 8192, 20000, 40000, 1 << 24})
      for (int64_t T : {int64_t(1), int64_t(1023), int64_t(1024), int64_t(1) << 21, (int64_t(1) << 23) + 1, kMaxT})
        for (double p : {0.0, 0.1}) {
          if (T * dim > (int64_t(1) << 48)) continue;   // thousands of pieces
          c_T = T, c_m = dim, c_n = 0, c_type = type;
          const poetx_dropout_rule rule{p, 1, nullptr, 2};
          where = "dropout";
          poetx_dropout_desc q{T, dim, type, dim, dim, dim, rule};
          EXPECT(poetx_dropout(&q, dev(1), dev(2), dev(3), nullptr) == POETX_OK);
          shapes_ok();
          where = "norm";
          for (int y : {type, (int)POETX_INT8}) {
            poetx_layer_norm_desc d{T, dim, type, y, dim, dim, dim, dim, 1e-6, rule};
            EXPECT(poetx_add_layer_norm(&d, dev(1), dev(2), fdev(3), fdev(9), dev(4), dev(5),
                                        y == POETX_INT8 ? fdev(6) : nullptr, fdev(7), fdev(8), nullptr) == POETX_OK);
            shapes_ok();
          }
          where = "norm backward";
          poetx_layer_norm_backward_desc b{T, dim, type, dim, dim, dim, dim, dim, rule};
          const size_t ws = poetx_layer_norm_backward_workspace(T, dim);
          EXPECT(poetx_layer_norm_backward(&b, dev(1), dev(2), dev(3), fdev(4), fdev(5), fdev(6), dev(7),
                                           p > 0 ? dev(8) : nullptr, fdev(9), fdev(10), dev(11), ws, nullptr) == POETX_OK);
          shapes_ok();
        }
}

void losses() {
  where = "cross entropy";
  for (int type : {POETX_FP32, POETX_BF16})
    for (int64_t T : {1, 2, 3, 31, 64, 255, 256, 1000, 16384, 70000, 1 << 20, 1 << 24})
      for (int V : {1, 2, 63, 256, 257, 1000, 32000, 50021, 300000, 1 << 20, 1 << 24})
        for (int n : {1, 7, 64, 100, 1000, 2048, 4097, 16384, 65536}) {
          c_T = T, c_m = V, c_n = n, c_type = type;
          const bool fits = T * n <= (int64_t(1) << 36) && (int64_t)V * n <= (int64_t(1) << 36);
          for (int off : {0, 1}) {   // aligned rows, and rows that are not
            poetx_cross_entropy_desc d{T, V, n, type, n + off, n + off, n, n, 1, -100};
            const size_t ws = poetx_linear_cross_entropy_workspace(&d);
            EXPECT((ws > 0) == fits);
            EXPECT(poetx_linear_cross_entropy(&d, dev(1), dev(2), reinterpret_cast<int64_t*>(dev(3)), fdev(4), fdev(5),
                                              dev(6), ws, nullptr) == (fits ? POETX_OK : POETX_ERR_SHAPE));
            if (fits) shapes_ok();
            // thousands of pieces
            if (!fits || T * V > (int64_t(1) << 38)) continue;
            for (int need : {1, 2, 3}) {
              const size_t bs = poetx_linear_cross_entropy_backward_workspace(&d, need & 1, need & 2);
              EXPECT(poetx_linear_cross_entropy_backward(&d, fdev(7), dev(1), dev(2), reinterpret_cast<int64_t*>(dev(3)),
                                                         fdev(5), need & 1 ? dev(8) : nullptr, need & 2 ? dev(9) : nullptr,
                                                         dev(6), bs, nullptr) == POETX_OK);
              shapes_ok();
            }
          }
        }
}

}  // namespace

int main() {
  norms();
  losses();
  std::printf("%s (%d failed checks)\n", failures ? "FAIL" : "OK", failures);
  return failures ? 1 : 0;
}
