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

// Eight columns of the gain, float32 or BF16; those past `left` are 0.
__device__ __forceinline__ void ld_weight8(const void* w, bool f32, int col, int left, float* v) {
  if (f32) {
    const auto r = ld_raw<true, 8, true>(w, col, left, false);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = r.at(i);
  } else {
    const auto r = ld_raw<false, 8, true>(w, col, left, false);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = r.at(i);
  }
}

// y before its rounding to BF16.
__device__ __forceinline__ float normalised(float h, float r, float w) { return (h * r) * w; }

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int d = 32; d; d >>= 1) v += __shfl_xor(v, d);
  return v;
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

__device__ __forceinline__ float reciprocal_rms(double sum, int n, double eps) {
  return (float)(1.0 / __builtin_sqrt((n ? sum / (double)n : 0.0) + eps));
}

}  // namespace fp8q
