// The exponential of the SwiGLU kernels, forward and backward (gfx950).
#pragma once

#include <hip/hip_runtime.h>

namespace fp8q {

// e^x for x <= 0: x log2(e) = n + f with |f| <= 1/2, reduced with log2(e)
// carried as a float32 head and a small tail (Cody and Waite's two-constant
// argument reduction, taken in base 2), 2^f from the hardware exp2, scaled by
// 2^n with ldexp (which also rounds subnormal results); below -104 the
// result is 0.
__device__ __forceinline__ float exp_nonpos(float x) {
  x = __builtin_fmaxf(x, -104.0f);
  const float l2e_hi = 1.44269502162933349609375f;  // RN32(log2 e)
  const float l2e_lo = 1.92596298909109e-8f;        // log2 e - l2e_hi
  const float n = __builtin_rintf(x * l2e_hi);
  const float f = __builtin_fmaf(x, l2e_lo, __builtin_fmaf(x, l2e_hi, -n));
  return __builtin_ldexpf(__builtin_amdgcn_exp2f(f), (int)n);
}

}  // namespace fp8q
