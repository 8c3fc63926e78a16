// What the RMS norm's kernels share (gfx950): the products of a normalised
// row, rounded the same way everywhere, and sums over a wave.
//
// With r = 1 / sqrt(mean(h^2) + eps), the sum in 64 bits and r rounded once to
// float32, a row's output is y = bf16(fl(fl(h r) w)).  A 64-bit sum differs
// between two orders of addition by some 2^-50, so r, and with it every bit of
// y, of its codes and of its scales, is the same whichever way the row is
// split over threads, in the forward pass and wherever y is formed again.  (A
// float32 sum moves r by a step now and then, and with it a tile's scale by a
// step of BF16.)  The 64-bit additions are hidden behind the row's loads.
#pragma once

#include "chunk8.h"

namespace fp8q {

// Eight columns of a row of n, as they come; those past its end are +0.  A
// row's last chunk is read as its last eight columns and moved down, so that
// it costs no load after another (column by column a row of 1030 took twice
// the time of one of 1024).
__device__ __forceinline__ Raw<false, 8> moved_down(Raw<false, 8> r, int s) {
  if (s & 4) r = Raw<false, 8>{{r.w[2], r.w[3], 0, 0}};
  if (s & 2) r = Raw<false, 8>{{r.w[1], r.w[2], r.w[3], 0}};
  if (s & 1) {
    r = Raw<false, 8>{{__builtin_amdgcn_alignbit(r.w[1], r.w[0], 16), __builtin_amdgcn_alignbit(r.w[2], r.w[1], 16),
                       __builtin_amdgcn_alignbit(r.w[3], r.w[2], 16), r.w[3] >> 16}};
  }
  return r;
}
__device__ __forceinline__ Raw<true, 8> moved_down(Raw<true, 8> r, int s) {
  if (s & 4) r = Raw<true, 8>{{r.w[4], r.w[5], r.w[6], r.w[7], 0, 0, 0, 0}};
  if (s & 2) r = Raw<true, 8>{{r.w[2], r.w[3], r.w[4], r.w[5], r.w[6], r.w[7], 0, 0}};
  if (s & 1) r = Raw<true, 8>{{r.w[1], r.w[2], r.w[3], r.w[4], r.w[5], r.w[6], r.w[7], 0}};
  return r;
}
template <bool F32, bool VEC, bool KEEP>
__device__ __forceinline__ Raw<F32, 8> ld_row8(const void* base, int64_t row_at, int col, int n) {
  if constexpr (VEC) {
    return ld_raw<F32, 8, KEEP>(base, row_at + col, 8, true);
  } else {
    if (n < 8) return ld_raw<F32, 8, true>(base, row_at + col, n - col, false);
    const Raw<F32, 8> r = ld_raw<F32, 8, true>(base, row_at + min(col, n - 8), 8, false);
    return n - col < 8 ? moved_down(r, 8 - (n - col)) : r;
  }
}

// Eight columns of the gain, float32 (lo, hi) or BF16 (lo), as they come.  The
// type is a matter of uniform branches, which cost less than twice the kernels.
struct Gain8 {
  uint4 lo, hi;
};
template <bool VEC>
__device__ __forceinline__ Gain8 ld_gain8(const void* p, bool f32, int col, int n) {
  Gain8 g;
  g.hi = make_uint4(0, 0, 0, 0);
  if (f32) {
    const auto r = ld_row8<true, VEC, true>(p, 0, col, n);
    g.lo = make_uint4(r.w[0], r.w[1], r.w[2], r.w[3]);
    g.hi = make_uint4(r.w[4], r.w[5], r.w[6], r.w[7]);
  } else {
    const auto r = ld_row8<false, VEC, true>(p, 0, col, n);
    g.lo = make_uint4(r.w[0], r.w[1], r.w[2], r.w[3]);
  }
  return g;
}
__device__ __forceinline__ void widen_gain8(const Gain8& g, bool f32, float* v) {
  v[0] = f32 ? __uint_as_float(g.lo.x) : bf16_lo(g.lo.x);
  v[1] = f32 ? __uint_as_float(g.lo.y) : bf16_hi(g.lo.x);
  v[2] = f32 ? __uint_as_float(g.lo.z) : bf16_lo(g.lo.y);
  v[3] = f32 ? __uint_as_float(g.lo.w) : bf16_hi(g.lo.y);
  v[4] = f32 ? __uint_as_float(g.hi.x) : bf16_lo(g.lo.z);
  v[5] = f32 ? __uint_as_float(g.hi.y) : bf16_hi(g.lo.z);
  v[6] = f32 ? __uint_as_float(g.hi.z) : bf16_lo(g.lo.w);
  v[7] = f32 ? __uint_as_float(g.hi.w) : bf16_hi(g.lo.w);
}

// y before its rounding to BF16.
__device__ __forceinline__ float normalised(float h, float r, float w) { return (h * r) * w; }

// A double of the lane that a DPP control names.
template <int CTRL>
__device__ __forceinline__ double dpp_double(double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)u, CTRL, 0xF, 0xF, false);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(u >> 32), CTRL, 0xF, 0xF, false);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ double lane_double(double v, int lane) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)u, lane), hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(u >> 32), lane);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

// Sum over the wave, the same in every lane: within rows of 16 lanes by DPP
// (as dpp_max16), then the four rows' sums.  All 64 lanes must be active.
__device__ __forceinline__ double wave_sum(double v) {
  v += dpp_double<0xB1>(v);
  v += dpp_double<0x4E>(v);
  v += dpp_double<0x141>(v);
  v += dpp_double<0x140>(v);
  return (lane_double(v, 0) + lane_double(v, 16)) + (lane_double(v, 32) + lane_double(v, 48));
}

// Sum over the workgroup, the same in every thread; `part` holds one value a
// wave.  All threads take part, and none may write `part` again before the
// next barrier.
__device__ __forceinline__ double block_sum(double v, double* part) {
  v = wave_sum(v);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
  __syncthreads();
  double t = part[0];
  for (int i = 1; i < (int)blockDim.x >> 6; ++i) t += part[i];
  return t;
}

// 1 / sqrt(sum / n + eps), rounded once: the hardware's estimate and two
// Newton steps in 64 bits, a tenth of the instructions of a division and a root
// (every wave of a row works it out).  The limits keep the steps finite; beyond
// them the result is 0 or infinite in float32 either way, and a NaN stays one.
__device__ __forceinline__ float reciprocal_rms(double sum, double inv_n, double eps) {
  double m = __builtin_fma(sum, inv_n, eps);
  m = m < 0x1p-1000 ? 0x1p-1000 : m > 0x1p1000 ? 0x1p1000 : m;
  double y = __builtin_amdgcn_rsq(m);
#pragma unroll
  for (int i = 0; i < 2; ++i) y = __builtin_fma(0.5 * y, __builtin_fma(-m * y, y, 1.0), y);
  return (float)y;
}

}  // namespace fp8q
