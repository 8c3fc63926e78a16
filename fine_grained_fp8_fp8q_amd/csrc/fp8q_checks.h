// Argument and device checks shared by the host entry points (fp8q_api.cpp,
// fp8q_moe_api.cpp).  Not part of the public ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <atomic>
#include <cstring>

#include "fp8q.h"

namespace fp8q {
namespace checks {

constexpr int64_t kMaxDim = (int64_t(1) << 31) - 1;
constexpr int64_t kMaxGroups = int64_t(1) << 24;  // 256-thread workgroups per launch
// 128x128 weight blocks per launch (one workgroup each; with the activation
// part of fp8q_quantize_linear, at most 2^20 more, still below kMaxGroups)
constexpr int64_t kMaxWeightBlocks = int64_t(1) << 23;
// GEMM kernels address an operand with 32-bit byte offsets.
constexpr int64_t kMaxOperandBytes = int64_t(1) << 31;
// 512-thread GEMM workgroups per launch (work items must fit in 32 bits)
constexpr int64_t kMaxGemmTiles = int64_t(1) << 23;

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool dim_ok(int64_t v) { return v >= 0 && v <= kMaxDim; }

// Per-device cache of "is gfx950": 0 unknown, 1 yes, 2 no.
constexpr int kMaxDevices = 64;
inline std::atomic<int> g_arch_ok[kMaxDevices];

inline fp8q_status check_device() {
  int dev = -1;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0) return FP8Q_ERR_DEVICE;
  if (dev < kMaxDevices) {
    const int cached = g_arch_ok[dev].load(std::memory_order_relaxed);
    if (cached) return cached == 1 ? FP8Q_OK : FP8Q_ERR_DEVICE;
  }
  hipDeviceProp_t prop;
  if (hipGetDeviceProperties(&prop, dev) != hipSuccess) return FP8Q_ERR_DEVICE;
  const bool ok = std::strncmp(prop.gcnArchName, "gfx950", 6) == 0;
  if (dev < kMaxDevices) g_arch_ok[dev].store(ok ? 1 : 2, std::memory_order_relaxed);
  return ok ? FP8Q_OK : FP8Q_ERR_DEVICE;
}

inline fp8q_status launched(hipError_t e) { return e == hipSuccess ? FP8Q_OK : FP8Q_ERR_LAUNCH; }

inline bool acc_ok(int acc) {
  return acc == FP8Q_ACC_FP32 || acc == FP8Q_ACC_FP8_MFMA || acc == FP8Q_ACC_FP8_MFMA_SCALED ||
         acc == FP8Q_ACC_FP32_POW2;
}

inline int64_t tiles256(int64_t rows, int64_t cols, int64_t width) {
  return ((rows + 255) / 256) * ((cols + width - 1) / width);
}

inline fp8q_status check_gemm_common(int64_t K, int out_dtype, const void* c, int64_t ld_c, int64_t N) {
  if (out_dtype != FP8Q_OUT_F32 && out_dtype != FP8Q_OUT_BF16) return FP8Q_ERR_INVALID_ARG;
  if (K % 128) return FP8Q_ERR_SHAPE;
  if (!c) return FP8Q_ERR_INVALID_ARG;
  if (ld_c < N) return FP8Q_ERR_SHAPE;
  if (!aligned16(c)) return FP8Q_ERR_ALIGN;
  return FP8Q_OK;
}

}  // namespace checks
}  // namespace fp8q
