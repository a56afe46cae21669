// Launch shapes of the calls around the linears at their documented limits. The
// runtime's launch entry is defined here and takes its place, so nothing runs: it
// writes down each grid and, for the product and the norm, the rows of its
// arguments. A dispatch counts threads in 32 bits, so a launch of 2^32 threads or
// more along an axis would be refused by the runtime.
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
  void* args;   // first argument, valid during the launch only
};
static std::vector<Launch> launches;
static void (*on_launch)(const Launch&) = nullptr;
static Launch pending;

extern "C" {
hipError_t __hipPushCallConfiguration(dim3 grid, dim3 block, size_t lds, hipStream_t) {
  pending = Launch{grid, block, lds, nullptr};
  return hipSuccess;
}
hipError_t __hipPopCallConfiguration(dim3* grid, dim3* block, size_t* lds, hipStream_t* s) {
  *grid = pending.grid;
  *block = pending.block;
  *lds = pending.lds;
  *s = nullptr;
  return hipSuccess;
}
hipError_t hipLaunchKernel(const void*, dim3 grid, dim3 block, void** args, size_t lds, hipStream_t) {
  const Launch l{grid, block, lds, args[0]};
  launches.push_back(l);
  if (on_launch) on_launch(l);
  return hipSuccess;
}
hipError_t hipGetLastError(void) { return hipSuccess; }
}

namespace {

constexpr int64_t kMaxT = 0x7fffffff;
char* dev(uintptr_t i) { return reinterpret_cast<char*>(i << 59); }
float* fdev(uintptr_t i) { return reinterpret_cast<float*>(dev(i)); }

void shapes_ok() {
  for (const Launch& l : launches) {
    const uint32_t threads = l.block.x * l.block.y * l.block.z;
    EXPECT(threads >= 64 && threads <= 1024 && l.lds <= 160 * 1024);
    EXPECT(l.grid.x >= 1 && (uint64_t)l.grid.x * l.block.x < (1ull << 32));
    EXPECT(l.grid.y >= 1 && (uint64_t)l.grid.y * l.block.y <= 65535);
    EXPECT(l.grid.z == 1);
  }
}

int64_t rows_seen, row_bytes;
const char* next_row;
// Rows of the product's activations: piece after piece, none left out or taken twice
void product_rows(const Launch& l) {
  const poetx::LinearArgs& a = *static_cast<const poetx::LinearArgs*>(l.args);
  EXPECT(a.T > 0);
  if (a.X != next_row) return;   // the join of split sums, over the rows of its product
  rows_seen += a.T;
  next_row += a.T * row_bytes;
}

void products() {
  where = "product";
  on_launch = product_rows;
  for (int type : {POETX_FP32, POETX_BF16, POETX_INT8})
    for (int m : {1, 2, 4, 7, 8, 15, 16, 17, 31, 32, 33, 40, 63, 64, 65, 100, 127, 129, 256, 257, 1000, 4096, 65537,
                  (1 << 24) - 1, 1 << 24})
      for (int n : {1, 3, 16, 64, 70, 256, 1000})
        for (int64_t T : {int64_t(1), int64_t(5), int64_t(1000), int64_t(100000), int64_t(1) << 22, int64_t(1) << 26,
                          (int64_t(1) << 27) + 1, int64_t(1) << 28, int64_t(1) << 29, kMaxT}) {
          if (T > (int64_t(1) << 42) / m) continue;   // millions of pieces
          const int es = type == POETX_FP32 ? 4 : type == POETX_BF16 ? 2 : 1;
          poetx_linear_desc d{T, m, n, type, type == POETX_FP32 ? POETX_FP32 : POETX_BF16, POETX_ACT_SILU,
                              n, n, m, m, m};
          c_T = T, c_m = m, c_n = n, c_type = type;
          const float* s = type == POETX_INT8 ? fdev(3) : nullptr;
          const size_t wsb = poetx_linear_workspace(&d);
          launches.clear();
          rows_seen = 0, row_bytes = (int64_t)n * es, next_row = dev(1);
          EXPECT(poetx_linear(&d, dev(1), dev(2), s, s, fdev(4), dev(5), dev(6), dev(7), wsb ? dev(8) : nullptr, wsb,
                              nullptr) == POETX_OK);
          EXPECT(rows_seen == T);
          shapes_ok();
          // results below 2^32 elements with whole column tiles need no second piece
          if (m % 32 == 0 && T <= (int64_t(1) << 32) / m / 256 * 256) EXPECT(launches.size() <= 2);
        }
  on_launch = nullptr;
}

void norm_rows(const Launch& l) {
  const poetx::NormArgs& a = *static_cast<const poetx::NormArgs*>(l.args);
  EXPECT(a.X == next_row && a.T > 0);
  rows_seen += a.T;
  next_row += a.T * row_bytes;
}
void norms() {
  for (int type : {POETX_FP32, POETX_BF16})
    for (int dim : {1, 8, 64, 100, 1000, 1024, 4096, 5000, 20000, 1 << 24})
      for (int64_t T : {int64_t(1), int64_t(1023), int64_t(1024), int64_t(1) << 23, (int64_t(1) << 23) + 1, kMaxT}) {
        c_T = T, c_m = dim, c_n = 0, c_type = type;
        where = "norm";
        const int es = type == POETX_FP32 ? 4 : 2;
        for (int y : {type, (int)POETX_INT8}) {
          poetx_norm_desc d{T, dim, type, y, dim, dim, dim, dim, 1e-6};
          launches.clear();
          rows_seen = 0, row_bytes = (int64_t)dim * es, next_row = dev(1);
          on_launch = norm_rows;
          EXPECT(poetx_add_rms_norm(&d, dev(1), dev(2), fdev(3), dev(4), dev(5), y == POETX_INT8 ? fdev(6) : nullptr,
                                    fdev(7), nullptr) == POETX_OK);
          on_launch = nullptr;
          EXPECT(rows_seen == T);
          shapes_ok();
        }
        where = "norm backward";
        poetx_norm_backward_desc b{T, dim, type, dim, dim, dim, dim};
        const size_t ws = poetx_rms_norm_backward_workspace(T, dim);
        launches.clear();
        EXPECT(poetx_rms_norm_backward(&b, dev(1), dev(2), dev(3), fdev(4), fdev(5), dev(6), fdev(7), dev(8), ws,
                                       nullptr) == POETX_OK);
        EXPECT(!launches.empty());
        shapes_ok();
      }
}

void clips() {
  where = "clip";
  for (int count : {0, 1, 120, 121, 5000})
    for (int64_t n : {int64_t(0), int64_t(1), int64_t(1) << 24, int64_t(1) << 33, int64_t(1) << 37}) {
      std::vector<void*> g;
      std::vector<int64_t> ns;
      std::vector<int32_t> types;
      for (int i = 0; i < count; ++i) {
        g.push_back(dev(1) + (uintptr_t)i * ((uintptr_t)n * 4 + 256));
        ns.push_back(n);
        types.push_back(i & 1);
      }
      c_T = count, c_m = n, c_n = 0, c_type = -1;
      for (bool write : {false, true}) {
        launches.clear();
        EXPECT(poetx_clip_grads(count, g.data(), ns.data(), types.data(),
                                write ? g.data() : nullptr, 1.0, fdev(9), dev(10),
                                poetx_clip_grads_workspace(count), nullptr) == POETX_OK);
        EXPECT(!launches.empty());
        shapes_ok();
      }
    }
}

}  // namespace

int main() {
  products();
  norms();
  clips();
  std::printf("%s (%d failed checks)\n", failures ? "FAIL" : "OK", failures);
  return failures ? 1 : 0;
}
