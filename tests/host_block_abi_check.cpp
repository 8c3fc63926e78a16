// Host-side check of the entry points between a block's linear layers
// (fp8q_block_api.cpp), built for the CPU with AddressSanitizer and
// UndefinedBehaviorSanitizer by tests/test_block_abi.py: launchers and the two
// HIP runtime queries are stubs.  Prints "host block ABI checks passed" and
// returns 0 when every check holds.
#include <cstdint>
#include <cstdio>
#include <cstring>
#include <limits>

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

int g_dev = 0, g_calls = 0;
hipError_t g_result = hipSuccess;
fp8q::NormArgs g_norm;
fp8q::NormBwdArgs g_bwd;
fp8q::NormTokenArgs g_token;
fp8q::GateArgs g_gate;
fp8q::GateBwdArgs g_gate_bwd;
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
hipError_t launch_norm(const NormArgs& a, hipStream_t) { ++g_calls; g_norm = a; return g_result; }
hipError_t launch_norm_backward(const NormBwdArgs& a, hipStream_t) { ++g_calls; g_bwd = a; return g_result; }
hipError_t launch_norm_token(const NormTokenArgs& a, hipStream_t) { ++g_calls; g_token = a; return g_result; }
hipError_t launch_gate(GateArgs a, hipStream_t) { ++g_calls; g_gate = a; return g_result; }
hipError_t launch_gate_backward(const GateBwdArgs& a, hipStream_t) { ++g_calls; g_gate_bwd = a; return g_result; }
}  // namespace fp8q

int main() {
  void* P = reinterpret_cast<void*>(4096);
  void* R = reinterpret_cast<void*>(8192);
  float* F = static_cast<float*>(P);
  uint8_t* U = static_cast<uint8_t*>(P);
  int32_t* I = static_cast<int32_t*>(P);
  const int64_t big = (int64_t(1) << 31) - 1, huge = std::numeric_limits<int64_t>::max(), row = int64_t(1) << 30;

  // every argument of the norm arrives where it belongs
  CHECK(fp8q_rmsnorm_quantize(P, 0, 10, 64, 65, R, 1, 66, P, 67, R, 0, 0.5, P, 68, 1, U, 69, F, F, nullptr) == FP8Q_OK);
  CHECK(g_norm.x == P && g_norm.ldx == 65 && g_norm.res == R && g_norm.ldr == 66 && g_norm.h == P && g_norm.ldh == 67 && g_norm.weight == R);
  CHECK(g_norm.ldy == 68 && g_norm.ldc == 69 && g_norm.eps == 0.5 && g_norm.rows == 10 && g_norm.n == 64);
  CHECK(g_norm.xf32 && !g_norm.sf32 && g_norm.wf32 && g_norm.pow2);
  CHECK(fp8q_rmsnorm_quantize(P, 1, big, row - 1, big, R, 0, big, nullptr, 0, R, 1, 1e-6, nullptr, 0, 0, U, big, F, nullptr, nullptr) == FP8Q_OK);
  CHECK(g_norm.rows == big && g_norm.n == row - 1 && !g_norm.xf32 && g_norm.sf32 && !g_norm.wf32 && !g_norm.pow2);
  CHECK(fp8q_rmsnorm_quantize(P, 1, 1, row, row, nullptr, 1, 0, nullptr, 0, P, 1, 1e-6, nullptr, 0, 0, nullptr, 0, nullptr, F, nullptr) == FP8Q_ERR_SHAPE);
  CHECK(fp8q_rmsnorm_quantize(P, 1, huge, 8, 8, nullptr, 1, 0, nullptr, 0, P, 1, 1e-6, nullptr, 0, 0, nullptr, 0, nullptr, F, nullptr) == FP8Q_ERR_INVALID_ARG);
  // in place: at its own stride, any stride for a single row
  CHECK(fp8q_rmsnorm_quantize(P, 1, 2, 8, 8, R, 1, 8, R, 8, P, 1, 1e-6, nullptr, 0, 0, nullptr, 0, nullptr, nullptr, nullptr) == FP8Q_OK);
  CHECK(fp8q_rmsnorm_quantize(P, 1, 2, 8, 8, R, 1, 8, R, 9, P, 1, 1e-6, nullptr, 0, 0, nullptr, 0, nullptr, nullptr, nullptr) == FP8Q_ERR_SHAPE);
  CHECK(fp8q_rmsnorm_quantize(P, 1, 1, 8, 8, R, 1, 8, R, 9, P, 1, 1e-6, nullptr, 0, 0, nullptr, 0, nullptr, nullptr, nullptr) == FP8Q_OK);

  // backward: the workspace is what the launch will write, for every size that is accepted
  for (int64_t rows : {int64_t(0), int64_t(1), int64_t(31), int64_t(33), int64_t(5000), big})
    for (int64_t n : {int64_t(1), int64_t(7), int64_t(512), int64_t(513), int64_t(1024), int64_t(2048), int64_t(2049), int64_t(7168), int64_t(8192), int64_t(8193), int64_t(16384),
                      int64_t(16385), int64_t(32768), int64_t(32769), row - 1}) {
      const int64_t need = fp8q_rmsnorm_backward_workspace(rows, n);
      CHECK(need % 16 == 0 && (need > 0) == (rows > 0));
      for (bool f32 : {false, true}) {
        if (rows == 0) break;
        const fp8q::NormBwdShape s = fp8q::norm_bwd_shape((int)rows, (int)n, f32);
        CHECK(need >= s.blocks * fp8q::norm_partial_ld((int)n) * 4 && s.blocks >= 1 && s.blocks <= rows && fp8q::norm_partial_ld((int)n) >= n);
        CHECK(s.threads >= 64 && s.threads <= (s.chunks ? s.wave ? 256 : 512 : 1024) && s.threads % 64 == 0);
        CHECK(s.chunks == 0 ? n > (f32 ? 8192 : 16384) : (int64_t)(s.wave ? 64 : s.threads) * s.chunks * 8 >= n);  // a row fits
        CHECK(s.chunks <= (f32 ? 2 : 4) && (s.wave || s.chunks == 0 || s.chunks == (f32 ? 2 : 4)));  // the kernels there are
      }
      if (need > 0) {
        CHECK(fp8q_rmsnorm_backward(P, 1, rows, n, n, P, 1, n, F, P, 1, nullptr, 0, P, 1, n, 0, nullptr, 0, nullptr, F, P, need - 1, nullptr) == FP8Q_ERR_INVALID_ARG);
        CHECK(fp8q_rmsnorm_backward(P, 1, rows, n, n, P, 1, n, F, P, 1, nullptr, 0, P, 1, n, 0, nullptr, 0, nullptr, F, nullptr, need, nullptr) == FP8Q_ERR_INVALID_ARG);
      }
      CHECK(fp8q_rmsnorm_backward(P, 1, rows, n, n, P, 1, n, F, P, 1, nullptr, 0, P, 1, n, 0, nullptr, 0, nullptr, F, P, need, nullptr) == FP8Q_OK);
      CHECK(g_bwd.rows == rows && g_bwd.n == n && g_bwd.dweight == F);
      CHECK(fp8q_rmsnorm_backward(P, 1, rows, n, n, P, 1, n, F, P, 1, nullptr, 0, P, 1, n, 0, nullptr, 0, nullptr, nullptr, nullptr, 0, nullptr) == FP8Q_OK);
    }
  CHECK(fp8q_rmsnorm_backward_workspace(huge, 8) == 0 && fp8q_rmsnorm_backward_workspace(8, row) == 0 && fp8q_rmsnorm_backward_workspace(-1, 8) == 0);
  CHECK(fp8q_rmsnorm_backward(P, 0, 10, 64, 65, R, 1, 66, F, R, 0, R, 67, P, 1, 68, 1, U, 69, F, nullptr, nullptr, 0, nullptr) == FP8Q_OK);
  CHECK(g_bwd.dy == P && g_bwd.lddy == 65 && g_bwd.h == R && g_bwd.ldh == 66 && g_bwd.weight == R && g_bwd.dres == R && g_bwd.lddr == 67 && g_bwd.lddx == 68 &&
        g_bwd.ldc == 69 && g_bwd.df32 && !g_bwd.hf32 && g_bwd.wf32 && !g_bwd.of32 && g_bwd.pow2);
  CHECK(fp8q_rmsnorm_backward(P, 0, 1, row, row, R, 1, row, F, R, 0, nullptr, 0, P, 1, row, 0, nullptr, 0, nullptr, nullptr, nullptr, 0, nullptr) == FP8Q_ERR_SHAPE);

  // the forward pass: every width is held by the threads, or goes to the kernel of long rows
  for (int rows : {1, 4095, 4096, (int)big})
    for (int n : {0, 1, 512, 2048, 2049, 4096, 4097, 7168, 16384, 16385, 32768, 32769, (int)row - 1}) {
      const int chunks = fp8q::norm_chunks(rows, n), threads = fp8q::norm_threads(n, chunks);
      CHECK((chunks == 1 || chunks == 2 || chunks == 4) && threads % 64 == 0 && threads <= (chunks == 4 ? 512 : 1024));
      CHECK(threads ? (int64_t)threads * chunks * 8 >= n : n > 16384);
    }

  // token tiles: the number of workgroups neither overflows nor passes
  CHECK(fp8q_rmsnorm_quantize_t(P, 0, 10, 64, 65, F, P, 1, I, 300, 1, U, 304, F, nullptr) == FP8Q_OK);
  CHECK(g_token.rows == 300 && g_token.src_rows == 10 && g_token.n == 64 && g_token.ldh == 65 && g_token.ldc == 304 && g_token.hf32 && !g_token.wf32 && g_token.pow2);
  CHECK(fp8q_rmsnorm_quantize_t(P, 0, big, big, big, F, P, 1, nullptr, big, 1, U, big, F, nullptr) == FP8Q_ERR_SHAPE);
  CHECK(fp8q_rmsnorm_quantize_t(P, 0, big, 64, 64, F, P, 1, nullptr, big, 1, U, big, F, nullptr) == FP8Q_ERR_SHAPE);
  CHECK(fp8q_rmsnorm_quantize_t(P, 0, (1 << 24) * 128ll - 128, 64, 64, F, P, 1, nullptr, (1 << 24) * 128ll - 128, 1, U, big, F, nullptr) == FP8Q_OK);

  // route
  CHECK(fp8q_moe_route(P, 1, 10, 256, 257, F, 0, 8, 4, 0, 6, 5, 2.5, 1, R, F, F, I, nullptr) == FP8Q_OK);
  CHECK(g_gate.logits == P && g_gate.ld == 257 && g_gate.chosen == R && g_gate.tokens == 10 && g_gate.experts == 256 && g_gate.topk == 6 && g_gate.groups == 8 &&
        g_gate.top_groups == 4 && g_gate.scale == 2.5 && !g_gate.lf32 && g_gate.i64 && !g_gate.sigmoid && !g_gate.two_best && g_gate.renormalize);
  CHECK(fp8q_moe_route(P, 1, big, 512, big, nullptr, 1, 64, 8, 1, 64, 0, -1.0, 0, R, F, nullptr, nullptr, nullptr) == FP8Q_OK && g_gate.tokens == big && g_gate.two_best);
  CHECK(fp8q_moe_route(P, 1, 10, huge, huge, F, 0, 8, 4, 0, 6, 5, 2.5, 1, R, F, F, I, nullptr) == FP8Q_ERR_INVALID_ARG);
  CHECK(fp8q_moe_route(P, 1, 10, 256, 257, F, 0, std::numeric_limits<int32_t>::max(), 4, 0, 6, 5, 2.5, 1, R, F, F, I, nullptr) == FP8Q_ERR_SHAPE);
  CHECK(fp8q_moe_route_backward(F, P, 0, 10, 6, R, 0, 256, 257, 1, 1, 0.5, F, P, 1, 258, nullptr) == FP8Q_OK);
  CHECK(g_gate_bwd.logits == R && g_gate_bwd.ld == 257 && g_gate_bwd.ldd == 258 && g_gate_bwd.topk == 6 && g_gate_bwd.lf32 && !g_gate_bwd.of32 && !g_gate_bwd.i64 &&
        g_gate_bwd.sigmoid && g_gate_bwd.renormalize && g_gate_bwd.scale == 0.5);

  g_result = hipErrorInvalidValue;
  CHECK(fp8q_moe_route(P, 1, 10, 256, 256, F, 0, 8, 4, 0, 6, 1, 2.5, 1, R, F, F, I, nullptr) == FP8Q_ERR_LAUNCH);
  g_calls = 0;
  for (g_dev = -1; g_dev <= 1; g_dev += 2) {
    CHECK(fp8q_moe_route(P, 1, 10, 256, 256, F, 0, 8, 4, 0, 6, 1, 2.5, 1, R, F, F, I, nullptr) == FP8Q_ERR_DEVICE);
    CHECK(fp8q_rmsnorm_quantize_t(P, 0, 10, 64, 65, F, P, 1, I, 300, 1, U, 304, F, nullptr) == FP8Q_ERR_DEVICE);
  }
  CHECK(g_calls == 0);
  if (g_failures == 0) std::printf("host block ABI checks passed\n");
  return g_failures != 0;
}
