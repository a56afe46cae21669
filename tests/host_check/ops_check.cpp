// Host-side checks of the calls around the linears (include/poetx.h) for a build
// of the library's host code under AddressSanitizer and UndefinedBehaviorSanitizer.
// It runs only where no GPU is visible: calls that pass their checks then go on
// to choose their kernels and fail at the first launch (POETX_ERR_HIP), so the
// host code in front of the launch runs too. Device pointers are fake.
#include <cstdint>
#include <cstdio>
#include <random>
#include <vector>

#include <hip/hip_runtime.h>

#include "poetx.h"

static int failures = 0;
#define EXPECT(cond)                                                            \
  do {                                                                          \
    if (!(cond)) {                                                              \
      std::printf("FAILED line %d: %s\n", __LINE__, #cond);                     \
      ++failures;                                                               \
    }                                                                           \
  } while (0)

namespace {

char* dev(uintptr_t i) { return reinterpret_cast<char*>(0x7f0000000000ull + (i << 44)); }
float* fdev(uintptr_t i) { return reinterpret_cast<float*>(dev(i)); }

void norms() {
  for (int dtype : {POETX_FP32, POETX_BF16})
    for (int64_t T : {1, 7, 5000, 9000000})
      for (int dim : {1, 33, 512, 2048, 4096, 20000}) {
        poetx_norm_desc d{T, dim, dtype, dtype, dim, dim + 5, dim, dim, 1e-6};
        EXPECT(poetx_add_rms_norm(&d, dev(1), dev(2), fdev(3), dev(4), dev(5), nullptr, fdev(6), nullptr) ==
               POETX_ERR_HIP);
        EXPECT(poetx_add_rms_norm(&d, dev(1), dev(2), fdev(3), dev(1), dev(5), nullptr, nullptr, nullptr) ==
               POETX_ERR_HIP);
        // four bytes behind r: past its end only where it is one element
        EXPECT(poetx_add_rms_norm(&d, dev(1), dev(2), fdev(3), dev(2) + 4, dev(5), nullptr, nullptr, nullptr) ==
               (T * dim == 1 ? POETX_ERR_HIP : POETX_ERR_INVALID_ARG));
        d.y_dtype = POETX_INT8;
        EXPECT(poetx_add_rms_norm(&d, dev(1), nullptr, fdev(3), nullptr, dev(5), fdev(6), nullptr, nullptr) ==
               POETX_ERR_HIP);
        poetx_norm_backward_desc b{T, dim, dtype, dim, dim, dim + 3, dim};
        const size_t ws = poetx_rms_norm_backward_workspace(T, dim);
        EXPECT(ws > 0);
        EXPECT(poetx_rms_norm_backward(&b, dev(1), dev(2), dev(3), fdev(4), fdev(5), dev(6), fdev(7), dev(8), ws,
                                       nullptr) == POETX_ERR_HIP);
        EXPECT(poetx_rms_norm_backward(&b, dev(1), nullptr, dev(3), fdev(4), fdev(5), dev(1), fdev(7), dev(8),
                                       ws - 1, nullptr) == POETX_ERR_WORKSPACE);
        b.T = 0;
        EXPECT(poetx_rms_norm_backward(&b, dev(1), nullptr, dev(3), fdev(4), fdev(5), dev(1), nullptr, dev(8), ws,
                                       nullptr) == POETX_ERR_INVALID_ARG);
      }
}

void products() {
  for (int dtype : {POETX_FP32, POETX_BF16, POETX_INT8})
    for (int64_t T : {1, 3, 20, 130, 700, 16384, 70000})
      for (int n : {1, 70, 256, 4096, 30000})
        for (int m : {1, 31, 264, 4096, 1 << 24})
          for (int act = POETX_ACT_NONE; act <= POETX_ACT_GELU_TANH; ++act) {
            const int y = dtype == POETX_FP32 ? POETX_FP32 : POETX_BF16;
            poetx_linear_desc d{T, m, n, dtype, y, act, n, n, m, m, m + 3};
            const float* s = dtype == POETX_INT8 ? fdev(3) : nullptr;
            const size_t wsb = poetx_linear_workspace(&d);
            char* const ws = wsb ? dev(8) : nullptr;
            EXPECT(poetx_linear(&d, dev(1), dev(2), s, s, fdev(4), dev(5), dev(6), dev(7), ws, wsb, nullptr) ==
                   POETX_ERR_HIP);
            EXPECT(poetx_linear(&d, dev(1), dev(2), s, s, nullptr, dev(5), nullptr, dev(5), ws, wsb, nullptr) ==
                   POETX_ERR_HIP);
            EXPECT(poetx_linear(&d, dev(1), dev(2), s, s, nullptr, nullptr, dev(6), dev(2), ws, wsb, nullptr) ==
                   POETX_ERR_INVALID_ARG);
          }
  poetx_linear_desc d{0x7fffffff, 1, 1, POETX_BF16, POETX_BF16, 0, INT64_MAX, 1, 1, 1, 1};
  EXPECT(poetx_linear(&d, dev(1), dev(2), nullptr, nullptr, nullptr, nullptr, nullptr, dev(3), nullptr, 0,
                      nullptr) == POETX_ERR_SHAPE);
}

void clips() {
  std::mt19937 rng(1);
  for (int count : {1, 2, 119, 120, 121, 1000}) {
    std::vector<const void*> g;
    std::vector<void*> o;
    std::vector<int64_t> n;
    std::vector<int32_t> t;
    uintptr_t at = 1 << 20;
    for (int i = 0; i < count; ++i) {
      n.push_back(rng() % 7 == 0 ? 0 : rng() % 100000);
      t.push_back((int32_t)(rng() % 2));
      g.push_back(dev(1) + at);
      o.push_back(rng() % 3 ? const_cast<void*>(g.back()) : dev(2) + at);
      at += (uintptr_t)n.back() * 4;
    }
    const size_t ws = poetx_clip_grads_workspace(count);
    EXPECT(ws > 0);
    auto call = [&](double limit) {
      return poetx_clip_grads(count, g.data(), n.data(), t.data(), o.data(), limit, fdev(4), dev(3), ws, nullptr);
    };
    EXPECT(call(1.0) == POETX_ERR_HIP);
    EXPECT(call(-1.0) == POETX_ERR_INVALID_ARG);
    EXPECT(poetx_clip_grads(count, g.data(), n.data(), t.data(), nullptr, 1.0, nullptr, dev(3), ws, nullptr) ==
           POETX_ERR_HIP);
    n[0] = 8;
    o[0] = const_cast<void*>(g[0]);
    g.push_back(g[0]);   // the first tensor once more: clipped twice
    o.push_back(o[0]);
    n.push_back(8);
    t.push_back(t[0]);
    EXPECT(poetx_clip_grads(count + 1, g.data(), n.data(), t.data(), o.data(), 1.0, fdev(4), dev(3),
                            poetx_clip_grads_workspace(count + 1), nullptr) == POETX_ERR_INVALID_ARG);
  }
}

}  // namespace

int main() {
  int ndev = 0;
  if (hipGetDeviceCount(&ndev) == hipSuccess && ndev > 0) {
    std::printf("skipped: a GPU is visible\n");
    return 77;
  }
  norms();
  products();
  clips();
  std::printf("%s (%d failed checks)\n", failures ? "FAIL" : "OK", failures);
  return failures ? 1 : 0;
}
