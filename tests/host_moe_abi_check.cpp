// Host-side check of the expert-layer entry points (fp8q_moe_api.cpp), built
// for the CPU with AddressSanitizer and UndefinedBehaviorSanitizer by
// tests/test_moe_abi.py: launchers and the two HIP runtime queries are stubs.
// Prints "host MoE ABI checks passed" and returns 0 when every check holds.
#include <cstdint>
#include <cstdio>
#include <cstring>
#include <limits>
#include <string>

#include "fp8q.h"
#include "fp8q_internal.h"

namespace {
int g_failures = 0;
#define CHECK(cond)                                                        \
  do {                                                                     \
    if (!(cond)) {                                                         \
      std::printf("%s:%d: check failed: %s\n", __FILE__, __LINE__, #cond); \
      ++g_failures;                                                        \
    }                                                                      \
  } while (0)

int g_dev = 0;
std::string g_name;
int64_t g_a = 0, g_b = 0, g_c = 0, g_d = 0;
int g_calls = 0;
hipError_t g_result = hipSuccess;
hipError_t record(const char* n, int64_t a, int64_t b, int64_t c, int64_t d) {
  g_name = n; g_a = a; g_b = b; g_c = c; g_d = d;
  ++g_calls;
  return g_result;
}
}  // namespace

extern "C" hipError_t hipGetDevice(int* device) {
  if (g_dev < 0) return hipErrorNoDevice;
  *device = g_dev;
  return hipSuccess;
}
extern "C" hipError_t hipGetDeviceProperties(hipDeviceProp_t* prop, int device) {
  std::memset(prop, 0, sizeof(*prop));
  std::strncpy(prop->gcnArchName, device == 1 ? "gfx942" : "gfx950", sizeof(prop->gcnArchName) - 1);
  return hipSuccess;
}

namespace fp8q {
hipError_t launch_moe_sort(const void*, bool i64, int pairs, int topk, int64_t, int64_t, int groups, int, int cap, int*, int*,
                           int*, int* hist, hipStream_t) {
  return record("sort", pairs, topk, groups * 2 + i64, hist ? cap : -cap);
}
hipError_t launch_moe_combine(const void*, bool yf, int cap, int n, int64_t, const int*, const float*, int tokens, int topk,
                              bool of, void*, int64_t, hipStream_t) {
  return record("combine", yf * 2 + of, cap, n, (int64_t)tokens * topk);
}
hipError_t launch_moe_combine_backward(const void*, bool df, int tokens, int n, int64_t, const void* y, bool yf, int cap,
                                       int64_t, const int*, const float*, int topk, const int*, uint16_t*, int64_t, bool pow2,
                                       uint8_t*, int64_t, float*, float*, hipStream_t) {
  return record("backward", (y ? 8 : 0) + df * 4 + yf * 2 + pow2, cap, n, (int64_t)tokens * topk);
}
hipError_t launch_swiglu_backward(const void*, const float*, int rows, int inter, int64_t, const uint16_t*, int64_t, uint16_t*,
                                  int64_t, bool pow2, uint8_t*, int64_t, float*, uint16_t*, int64_t, hipStream_t) {
  return record("swiglu", rows, inter, pow2, 0);
}
hipError_t launch_grouped_wgrad(const uint8_t*, const float*, const uint8_t*, const float*, const int32_t*, int groups, int cap,
                                int nout, int kin, int acc, float*, int64_t, hipStream_t) {
  return record("wgrad", groups, cap, nout * 10000 + kin, acc);
}
}  // namespace fp8q

int main() {
  void* P = reinterpret_cast<void*>(4096);
  int32_t* I = static_cast<int32_t*>(P);
  float* F = static_cast<float*>(P);
  uint8_t* U = static_cast<uint8_t*>(P);
  const int64_t big = (int64_t(1) << 31) - 1, huge = std::numeric_limits<int64_t>::max();

  // sort: the largest products neither overflow nor pass
  CHECK(fp8q_moe_sort(P, 1, 1024, 8, 8, 3, 16, 128, 10240, I, I, I, P, 1 << 20, nullptr) == FP8Q_OK);
  CHECK(g_name == "sort" && g_a == 8192 && g_b == 8 && g_c == 33 && g_d == 10240);
  CHECK(fp8q_moe_sort(P, 0, big, big, big, 0, 16, 1, 16, I, I, I, P, huge, nullptr) == FP8Q_ERR_SHAPE);
  CHECK(fp8q_moe_sort(P, 0, big, 1, 1, 0, 1, 1, 16, I, I, I, P, huge, nullptr) == FP8Q_ERR_SHAPE);  // pairs + G * align
  CHECK(fp8q_moe_sort(P, 0, 4, 1, 1, 0, 512, std::numeric_limits<int32_t>::max(), 0, I, I, I, P, 0, nullptr) == FP8Q_ERR_SHAPE);
  CHECK(fp8q_moe_sort(P, 0, huge, 1, 1, 0, 1, 1, 16, I, I, I, P, 0, nullptr) == FP8Q_ERR_INVALID_ARG);
  CHECK(fp8q_moe_sort_workspace(huge, huge, 3) == 0 && fp8q_moe_sort_workspace(big, big, 3) == 0);
  CHECK(fp8q_moe_sort_workspace(1, 8, 256) == 0 && fp8q_moe_sort_workspace(-1, 8, 4) == 0);
  const int64_t need = fp8q_moe_sort_workspace(16384, 8, 16);
  CHECK(need > 0 && need % 64 == 0);
  CHECK(fp8q_moe_sort(P, 0, 16384, 8, 8, 0, 16, 1, 16, I, I, I, P, need - 1, nullptr) == FP8Q_ERR_INVALID_ARG);
  CHECK(fp8q_moe_sort(P, 0, 16384, 8, 8, 0, 16, 1, 16, I, I, I, nullptr, need, nullptr) == FP8Q_ERR_INVALID_ARG);
  CHECK(fp8q_moe_sort(P, 0, 16384, 8, 8, 0, 16, 1, 16, I, I, I, P, need, nullptr) == FP8Q_OK);
  // the walk over padding rows ends at the largest rows that are accepted, for every lane and step of the kernel
  CHECK(fp8q_moe_sort(P, 0, 1, 1, 1, 0, 1, (int32_t)big - 1, big - 1, I, I, I, nullptr, 0, nullptr) == FP8Q_OK);
  CHECK(fp8q_moe_sort(P, 0, big - 2, 1, 1, 0, 1, 2, big - 1, I, I, I, P, 1 << 20, nullptr) == FP8Q_OK);
  for (int first : {(int)big - 2, (int)big - 1100, (int)big - 1})
    for (int lanes : {64, 1024, 256 * 1024}) {
      int64_t seen = 0;
      bool inside = true;
      for (int lane = 0; lane < lanes; ++lane)
        fp8q::for_rows(first, lane, lanes, (int)big - 1, [&](int64_t r) {
          inside = inside && r >= first && r < big - 1;
          ++seen;
        });
      CHECK(inside && seen == big - 1 - first);
    }
  // no tokens: the table is still written
  CHECK(fp8q_moe_sort(nullptr, 0, 0, 8, 8, 0, 16, 1, 16, I, I, nullptr, nullptr, 0, nullptr) == FP8Q_OK && g_a == 0);

  // combine
  CHECK(fp8q_moe_combine(P, FP8Q_OUT_BF16, 100, 64, 64, I, F, 10, 4, FP8Q_OUT_F32, P, 64, nullptr) == FP8Q_OK);
  CHECK(g_name == "combine" && g_a == 1 && g_b == 100 && g_c == 64 && g_d == 40);
  CHECK(fp8q_moe_combine(P, 0, 100, big, big, I, F, big, 1, 0, P, big, nullptr) == FP8Q_ERR_SHAPE);
  CHECK(fp8q_moe_combine(P, 0, 100, 8, 8, I, F, big, big, 0, P, 8, nullptr) == FP8Q_ERR_SHAPE);
  CHECK(fp8q_moe_combine(P, 0, 100, 512, 512, I, F, 1 << 24, 1, 0, P, 512, nullptr) == FP8Q_ERR_SHAPE);
  CHECK(fp8q_moe_combine(P, 0, 100, 512, 512, I, F, (1 << 24) - 1, 1, 0, P, 512, nullptr) == FP8Q_OK);
  CHECK(fp8q_moe_combine(P, 0, 1, 1 << 30, 1 << 30, I, F, 1, 1, 0, P, 1 << 30, nullptr) == FP8Q_ERR_SHAPE);
  CHECK(fp8q_moe_combine(P, 0, 1, (1 << 30) - 1, 1 << 30, I, F, 1, 1, 0, P, 1 << 30, nullptr) == FP8Q_OK);
  CHECK(fp8q_moe_combine_backward(P, 0, 1, 1 << 30, 1 << 30, P, 0, 1, 1 << 30, I, F, 1, I, P, 1 << 30, 0, nullptr, 0, nullptr, F, nullptr) == FP8Q_ERR_SHAPE);
  CHECK(fp8q_moe_combine(nullptr, 0, 0, 64, 0, I, nullptr, 10, 4, 0, P, 64, nullptr) == FP8Q_OK);  // no rows: zeros
  // ... and the rule that the launch asks takes an input of no bytes
  CHECK(fp8q::input_stays_cached(0, 0) && fp8q::input_stays_cached(big, 0) && fp8q::input_stays_cached(0, 4 * big));
  CHECK(fp8q::input_stays_cached(96, 1 << 20) && !fp8q::input_stays_cached(97, 1 << 20) && !fp8q::input_stays_cached(big, 4 * big));

  // backward: y is handed over only for the weight gradient
  CHECK(fp8q_moe_combine_backward(P, 1, 10, 64, 64, P, 1, 100, 64, I, F, 4, I, P, 64, 1, U, 64, F, F, nullptr) == FP8Q_OK);
  CHECK(g_name == "backward" && g_a == 9 && g_b == 100 && g_c == 64 && g_d == 40);
  CHECK(fp8q_moe_combine_backward(P, 0, 10, 64, 64, P, 0, 100, 64, I, F, 4, I, P, 64, 0, nullptr, 0, nullptr, nullptr, nullptr) == FP8Q_OK);
  CHECK(g_a == 6);
  g_calls = 0;
  CHECK(fp8q_moe_combine_backward(P, 0, 10, 64, 64, P, 0, 100, 64, I, F, 4, I, nullptr, 0, 0, nullptr, 0, nullptr, nullptr, nullptr) == FP8Q_OK);
  CHECK(fp8q_moe_combine_backward(P, 0, 0, 64, 64, P, 0, 100, 64, I, F, 4, nullptr, P, 64, 0, nullptr, 0, nullptr, F, nullptr) == FP8Q_OK);
  CHECK(g_calls == 0);
  CHECK(fp8q_moe_combine_backward(P, 0, big, 64, 64, P, 0, 100, 64, I, F, big, I, P, 64, 0, nullptr, 0, nullptr, F, nullptr) == FP8Q_ERR_SHAPE);
  CHECK(fp8q_moe_combine_backward(P, 0, 10, 64, 64, P, 0, big, 64, I, F, 4, I, P, 64, 0, nullptr, 0, nullptr, F, nullptr) == FP8Q_ERR_SHAPE);

  // rows of no columns have weight gradients (zeros) all the same ...
  g_calls = 0;
  for (int64_t tokens : {int64_t(1), int64_t(10), int64_t(3000)})
    CHECK(fp8q_moe_combine_backward(nullptr, 0, tokens, 0, 0, nullptr, 0, 100, 0, I, F, 4, I, nullptr, 0, 0, nullptr, 0, nullptr, F, nullptr) == FP8Q_OK &&
          g_c == 0 && g_d == 4 * tokens);
  CHECK(g_calls == 3);
  // ... and every width that is accepted gets whole waves, no more than 256 threads, on both sides of the rule
  for (int pairs : {1, 2048, 2049, 1 << 23})
    for (int n : {0, 1, 8, 9, 511, 512, 513, 1030, 2047, 2048, 2049, 6259, 7168, (1 << 30) - 1}) {
      const int threads = fp8q::combine_backward_threads(pairs, n);
      CHECK(threads >= 64 && threads <= 256 && threads % 64 == 0);
      if (pairs <= 2048 && n > 0) CHECK((int64_t)threads * 8 * ((n + 2047) / 2048) >= n);  // in the fewest steps
    }
  CHECK(fp8q::combine_backward_threads(8, 6259) == 256 && fp8q::combine_backward_threads(1 << 15, 7168) == 128);

  // swiglu, grouped wgrad
  CHECK(fp8q_swiglu_backward(P, F, 10, 128, 256, P, 128, P, 256, 1, U, 256, F, P, 128, nullptr) == FP8Q_OK && g_name == "swiglu" && g_c == 1);
  CHECK(fp8q_swiglu_backward(P, nullptr, big, big / 2, big, P, big, P, big, 0, nullptr, 0, nullptr, nullptr, 0, nullptr) == FP8Q_ERR_SHAPE);
  CHECK(fp8q_grouped_wgrad_ex(U, F, U, F, I, 3, 256, 20, 30, 3, F, 30, nullptr) == FP8Q_OK && g_name == "wgrad" && g_a == 3 && g_b == 256 && g_c == 200030 && g_d == 3);
  CHECK(fp8q_grouped_wgrad(U, F, U, F, I, std::numeric_limits<int32_t>::max(), 256, 20, 30, F, 30, nullptr) == FP8Q_ERR_SHAPE);
  CHECK(fp8q_grouped_wgrad(U, F, U, F, I, 2, big - 127, big, big, F, big, nullptr) == FP8Q_ERR_SHAPE);
  CHECK(fp8q_grouped_wgrad(U, F, U, F, I, 2, 1 << 24, 20, 30, F, 30, nullptr) == FP8Q_ERR_SHAPE);
  CHECK(fp8q_grouped_wgrad(U, F, U, F, I, 2, (1 << 24) - 128, 20, 30, F, 30, nullptr) == FP8Q_OK);
  CHECK(fp8q_grouped_wgrad(U, F, U, F, I, 2, 0, 20, 30, F, 30, nullptr) == FP8Q_OK);  // no rows: zeros

  g_result = hipErrorInvalidValue;
  CHECK(fp8q_moe_combine(P, 1, 100, 64, 64, I, F, 10, 4, 0, P, 64, nullptr) == FP8Q_ERR_LAUNCH);
  for (g_dev = -1; g_dev <= 1; g_dev += 2)
    CHECK(fp8q_moe_combine(P, 1, 100, 64, 64, I, F, 10, 4, 0, P, 64, nullptr) == FP8Q_ERR_DEVICE);
  if (g_failures == 0) std::printf("host MoE ABI checks passed\n");
  return g_failures != 0;
}
