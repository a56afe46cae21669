// Host-side checks of the calls that train around the linears (include/poetx.h) for a build of
// the library's host code under AddressSanitizer and UndefinedBehaviorSanitizer. It runs only
// where no GPU is visible: calls that pass their checks then go on to choose their kernels and
// fail at the first launch (POETX_ERR_HIP), so the host code in front of the launch runs too.
// Device pointers are fake.
#include <cstdint>
#include <cstdio>

#include <hip/hip_runtime.h>

#include "poetx.h"

static int failures = 0;
#define EXPECT(cond)                                        \
  do {                                                      \
    if (!(cond)) {                                          \
      std::printf("FAILED line %d: %s\n", __LINE__, #cond); \
      ++failures;                                           \
    }                                                       \
  } while (0)

namespace {

char* dev(uintptr_t i) { return reinterpret_cast<char*>(0x7f0000000000ull + (i << 44)); }
float* fdev(uintptr_t i) { return reinterpret_cast<float*>(dev(i)); }
int64_t* idev(uintptr_t i) { return reinterpret_cast<int64_t*>(dev(i)); }

void norms() {
  for (int dtype : {POETX_FP32, POETX_BF16})
    for (int64_t T : {1, 7, 5000, 9000000})
      for (int dim : {1, 33, 512, 2048, 4096, 7000, 20000, 70000})
        for (double p : {0.0, 0.3, 1.0}) {
          const poetx_dropout_rule rule{p, UINT64_MAX, reinterpret_cast<uint64_t*>(dev(12)), UINT32_MAX};
          poetx_dropout_desc q{T, dim, dtype, dim, dim + 5, dim, rule};
          EXPECT(poetx_dropout(&q, dev(1), dev(2), dev(3), nullptr) == POETX_ERR_HIP);
          EXPECT(poetx_dropout(&q, dev(1), nullptr, dev(1), nullptr) == POETX_ERR_HIP);
          EXPECT(poetx_dropout(&q, dev(1), dev(2), dev(12), nullptr) == POETX_ERR_INVALID_ARG);
          poetx_layer_norm_desc d{T, dim, dtype, dtype, dim, dim + 5, dim, dim, 1e-6, rule};
          EXPECT(poetx_add_layer_norm(&d, dev(1), dev(2), fdev(3), fdev(4), dev(5), dev(6), nullptr, fdev(7), fdev(8),
                                      nullptr) == POETX_ERR_HIP);
          EXPECT(poetx_add_layer_norm(&d, dev(1), dev(2), fdev(3), nullptr, dev(1), dev(6), nullptr, nullptr, nullptr,
                                      nullptr) == POETX_ERR_HIP);
          d.y_dtype = POETX_INT8;
          EXPECT(poetx_add_layer_norm(&d, dev(1), nullptr, fdev(3), nullptr, nullptr, dev(6), fdev(7), nullptr, nullptr,
                                      nullptr) == POETX_ERR_HIP);
          poetx_layer_norm_backward_desc b{T, dim, dtype, dim, dim, dim + 3, dim, dim, rule};
          const size_t ws = poetx_layer_norm_backward_workspace(T, dim);
          EXPECT(ws > 0);
          void* const gr = p > 0 ? dev(9) : nullptr;
          EXPECT(poetx_layer_norm_backward(&b, dev(1), dev(2), dev(3), fdev(4), fdev(5), fdev(6), dev(7), gr, fdev(8),
                                           fdev(10), dev(11), ws, nullptr) == POETX_ERR_HIP);
          EXPECT(poetx_layer_norm_backward(&b, dev(1), nullptr, dev(3), fdev(4), fdev(5), fdev(6), dev(1), gr, fdev(8),
                                           fdev(10), dev(11), ws - 1, nullptr) == POETX_ERR_WORKSPACE);
          b.T = 0;
          EXPECT(poetx_layer_norm_backward(&b, dev(1), nullptr, dev(3), fdev(4), fdev(5), fdev(6), dev(1), gr, nullptr,
                                           fdev(10), dev(11), ws, nullptr) == POETX_ERR_INVALID_ARG);
        }
}

void losses() {
  for (int dtype : {POETX_FP32, POETX_BF16})
    for (int64_t T : {1, 3, 20, 130, 700, 16384, 70000, 1 << 24})
      for (int V : {1, 31, 264, 5003, 32000, 1 << 24})
        for (int n : {1, 70, 256, 1001, 4096, 65536}) {
          if (T * n > (int64_t(1) << 36) || (int64_t)V * n > (int64_t(1) << 36)) continue;
          poetx_cross_entropy_desc d{T, V, n, dtype, n + 8, n, n, n, 1, INT64_MIN};
          const size_t ws = poetx_linear_cross_entropy_workspace(&d);
          EXPECT(poetx_linear_cross_entropy(&d, dev(1), dev(2), idev(3), fdev(4), fdev(5), dev(6), ws, nullptr) ==
                 POETX_ERR_HIP);
          EXPECT(poetx_linear_cross_entropy(&d, dev(1), dev(2), idev(3), fdev(4), fdev(5), dev(6), ws - 1, nullptr) ==
                 POETX_ERR_WORKSPACE);
          for (int need : {1, 2, 3}) {
            d.g_count = need == 2 ? T : 1;
            const size_t bs = poetx_linear_cross_entropy_backward_workspace(&d, need & 1, need & 2);
            void* const gx = need & 1 ? dev(8) : nullptr;
            void* const gw = need & 2 ? dev(9) : nullptr;
            EXPECT(poetx_linear_cross_entropy_backward(&d, fdev(7), dev(1), dev(2), idev(3), fdev(5), gx, gw, dev(6), bs,
                                                       nullptr) == POETX_ERR_HIP);
            EXPECT(poetx_linear_cross_entropy_backward(&d, fdev(7), dev(1), dev(2), idev(3), fdev(5), gx, gw, dev(6),
                                                       bs - 1, nullptr) == POETX_ERR_WORKSPACE);
          }
        }
  poetx_cross_entropy_desc d{1 << 24, 1, 1, POETX_BF16, INT64_MAX, 1, 1, 1, 1, 0};
  EXPECT(poetx_linear_cross_entropy(&d, dev(1), dev(2), idev(3), fdev(4), fdev(5), dev(6), 1 << 30, nullptr) ==
         POETX_ERR_SHAPE);
}

}  // namespace

int main() {
  int ndev = 0;
  if (hipGetDeviceCount(&ndev) == hipSuccess && ndev > 0) {
    std::printf("skipped: a GPU is visible\n");
    return 77;
  }
  norms();
  losses();
  std::printf("%s (%d failed checks)\n", failures ? "FAIL" : "OK", failures);
  return failures ? 1 : 0;
}
