// Residual addition, RMS norm and 1x128 quantization in one pass, and the
// norm's gradient, gfx950.
//
// Forward, per row of n columns (norm_common.h has the roundings):
//   h = rn(x + res),  r = rn32(1 / sqrt(mean(h^2) + eps)),  y = bf16((h r) w),
// y in BF16 and / or as E4M3 codes with 1x128 scales, what the quantizer would
// make of that BF16 tensor.
//
// Backward, with g = dy w, c = rn32(mean(g h) r) (the sum in 64 bits):
//   dx = (g - (h r) c) r + dres,   dw = sum over rows of dy (h r).
#include "fp8q_internal.h"
#include "norm_common.h"

namespace fp8q {
namespace {

constexpr int kNormThreads = 256;
constexpr int kMaxNormGrid = 1 << 20;  // workgroups; more rows go round

// Eight values of the row that is normalised.
template <bool F32>
__device__ __forceinline__ void widen(const Raw<F32, 8>& r, float* v) {
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = r.at(i);
}

// Eight values as the row's type holds them, and rounded to it in place.
template <bool F32>
__device__ __forceinline__ void st_row8(void* base, int64_t at, float* v, int left) {
  if constexpr (F32) {
    st_float4(static_cast<float*>(base) + at, v, left, false);
    st_float4(static_cast<float*>(base) + at + 4, v + 4, left - 4, false);
  } else {
    st_bf16x8(static_cast<uint16_t*>(base) + at, pack_bf16x8(v), left, false);
  }
}
template <bool F32>
__device__ __forceinline__ void round_row8(float* v) {
  if constexpr (!F32) {
    const uint4 c = pack_bf16x8(v);
    const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = bf16_lo(w[i]);
      v[2 * i + 1] = bf16_hi(w[i]);
    }
  }
}

// Eight BF16 values of one lane quantized with the 16-lane DPP row that holds
// their 1x128 tile; every lane of the wave takes part.
__device__ __forceinline__ void quantize_chunk(uint4 d, bool pow2, bool in, int col, int left, int row, int nb, uint8_t* codes, int64_t ldc,
                                               float* scales) {
  const uint32_t amax = dpp_max16(absmax8(d));
  TileScale ts;
  uint2 c;
  if (pow2) {
    ts = tile_scale<true>(amax);
    c = encode8<true>(d, ts);
  } else {
    ts = tile_scale<false>(amax);
    c = encode8<false>(d, ts);
  }
  if (in) {
    st_codes8(codes + (int64_t)row * ldc + col, c, left, false);
    if ((threadIdx.x & 15) == 0) scales[(int64_t)row * nb + (col >> 7)] = ts.s;
  }
}

// -------------------------------------------------------------- forward ---
// One workgroup per row, which it goes over twice.
template <bool XF32, bool SF32, bool RES>
__global__ __launch_bounds__(kNormThreads) void norm_kernel(NormArgs a) {
  __shared__ double part[kNormThreads / 64];
  const int step = (int)blockDim.x * 8, tid = threadIdx.x;
  const int nb = (a.n + 127) >> 7;
  // eight values of h: of x, or of the stream rounded to its type
  auto load_h = [&](int row, int col, int left, float* v) {
    widen(ld_raw<XF32, 8>(a.x, (int64_t)row * a.ldx + col, left, false), v);
    if constexpr (RES) {
      float s[8];
      widen(ld_raw<SF32, 8>(a.res, (int64_t)row * a.ldr + col, left, false), s);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] += s[i];
      round_row8<SF32>(v);
    }
  };
  for (int row = blockIdx.x; row < a.rows; row += (int)gridDim.x) {
    double sum = 0.0;
    for (int col = tid * 8; col < a.n; col += step) {
      float v[8];
      load_h(row, col, a.n - col, v);
      if (RES && a.h) st_row8<SF32>(a.h, (int64_t)row * a.ldh + col, v, a.n - col);
#pragma unroll
      for (int i = 0; i < 8; ++i) sum = __builtin_fma((double)v[i], (double)v[i], sum);
    }
    const float r = reciprocal_rms(block_sum(sum, part), a.n, a.eps);
    if (tid == 0 && a.rstd) a.rstd[row] = r;
    if (a.y || a.codes) {
      for (int c0 = 0; c0 < a.n; c0 += step) {
        const int col = c0 + tid * 8, left = a.n - col;
        float v[8] = {}, w[8] = {};
        if (left > 0) {
          // (the stream may have been written over its own input)
          if (RES && a.h) {
            widen(ld_raw<SF32, 8, true>(a.h, (int64_t)row * a.ldh + col, left, false), v);
          } else {
            load_h(row, col, left, v);
          }
          ld_weight8(a.weight, a.wf32, col, left, w);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = normalised(v[i], r, w[i]);
        const uint4 d = pack_bf16x8(v);
        if (a.y && left > 0) st_bf16x8(a.y + (int64_t)row * a.ldy + col, d, left, false);
        if (a.codes) quantize_chunk(d, a.pow2, left > 0, col, left, row, nb, a.codes, a.ldc, a.scales);
      }
    }
    __syncthreads();  // (part is written again)
  }
}

// ------------------------------------------------------------- backward ---
template <bool DF32, bool HF32, bool OF32>
__global__ __launch_bounds__(kNormThreads) void norm_bwd_kernel(NormBwdArgs a) {
  __shared__ double part[kNormThreads / 64];
  const int step = (int)blockDim.x * 8, tid = threadIdx.x;
  const int nb = (a.n + 127) >> 7;
  for (int row = blockIdx.x; row < a.rows; row += (int)gridDim.x) {
    const float r = a.rstd[row];
    auto load = [&](int col, int left, float* g, float* h) {
      float w[8];
      widen(ld_raw<DF32, 8, true>(a.dy, (int64_t)row * a.lddy + col, left, false), g);
      widen(ld_raw<HF32, 8, true>(a.h, (int64_t)row * a.ldh + col, left, false), h);
      ld_weight8(a.weight, a.wf32, col, left, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) g[i] *= w[i];
    };
    double sum = 0.0;
    for (int col = tid * 8; col < a.n; col += step) {
      float g[8], h[8];
      load(col, a.n - col, g, h);
#pragma unroll
      for (int i = 0; i < 8; ++i) sum = __builtin_fma((double)g[i], (double)h[i], sum);
    }
    const float c = (float)(block_sum(sum, part) * (double)r / (double)a.n);
    for (int c0 = 0; c0 < a.n; c0 += step) {
      const int col = c0 + tid * 8, left = a.n - col;
      float g[8] = {}, h[8] = {}, s[8] = {};
      if (left > 0) {
        load(col, left, g, h);
        if (a.dres) widen(ld_raw<OF32, 8>(a.dres, (int64_t)row * a.lddr + col, left, false), s);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        g[i] = (g[i] - (h[i] * r) * c) * r;
        if (a.dres) g[i] += s[i];
      }
      if (a.dx && left > 0) st_row8<OF32>(a.dx, (int64_t)row * a.lddx + col, g, left);
      if (a.codes) quantize_chunk(pack_bf16x8(g), a.pow2, left > 0, col, left, row, nb, a.codes, a.ldc, a.scales);
    }
    __syncthreads();  // (part is written again)
  }
}

// dw over the rows of one block (blockIdx.y), one column a thread.
template <bool DF32, bool HF32>
__global__ __launch_bounds__(kNormThreads) void norm_dw_kernel(NormBwdArgs a, int per) {
  const int col = blockIdx.x * kNormThreads + (int)threadIdx.x;
  if (col >= a.n) return;
  const int64_t lo = (int64_t)blockIdx.y * per, hi = min(lo + per, (int64_t)a.rows);
  auto at = [&](const void* p, bool f32, int64_t i) {
    return f32 ? static_cast<const float*>(p)[i] : __uint_as_float((uint32_t)static_cast<const uint16_t*>(p)[i] << 16);
  };
  float sum = 0.0f;
  for (int64_t t = lo; t < hi; ++t) sum = __builtin_fmaf(at(a.dy, DF32, t * a.lddy + col), at(a.h, HF32, t * a.ldh + col) * a.rstd[t], sum);
  a.partial[(int64_t)blockIdx.y * a.n + col] = sum;
}

// The blocks' sums added in their order.
__global__ __launch_bounds__(kNormThreads) void norm_dw_sum_kernel(const float* partial, int blocks, int n, float* dw) {
  const int col = blockIdx.x * kNormThreads + (int)threadIdx.x;
  if (col >= n) return;
  float sum = 0.0f;
  for (int b = 0; b < blocks; ++b) sum += partial[(int64_t)b * n + col];
  dw[col] = sum;
}

}  // namespace

static int norm_grid(int rows) { return rows < kMaxNormGrid ? rows : kMaxNormGrid; }

hipError_t launch_norm(const NormArgs& a, hipStream_t stream) {
  auto kernel = !a.res ? (a.xf32 ? norm_kernel<true, true, false> : norm_kernel<false, false, false>)
                : a.xf32 ? (a.sf32 ? norm_kernel<true, true, true> : norm_kernel<true, false, true>)
                         : (a.sf32 ? norm_kernel<false, true, true> : norm_kernel<false, false, true>);
  hipLaunchKernelGGL(kernel, dim3(norm_grid(a.rows)), dim3(kNormThreads), 0, stream, a);
  return hipGetLastError();
}

hipError_t launch_norm_backward(const NormBwdArgs& a, hipStream_t stream) {
  if (a.rows > 0 && (a.dx || a.codes)) {
    auto kernel = a.df32 ? (a.hf32 ? (a.of32 ? norm_bwd_kernel<true, true, true> : norm_bwd_kernel<true, true, false>)
                                   : (a.of32 ? norm_bwd_kernel<true, false, true> : norm_bwd_kernel<true, false, false>))
                         : (a.hf32 ? (a.of32 ? norm_bwd_kernel<false, true, true> : norm_bwd_kernel<false, true, false>)
                                   : (a.of32 ? norm_bwd_kernel<false, false, true> : norm_bwd_kernel<false, false, false>));
    hipLaunchKernelGGL(kernel, dim3(norm_grid(a.rows)), dim3(kNormThreads), 0, stream, a);
  }
  if (a.dweight) {
    const int blocks = norm_dw_blocks(a.rows), per = blocks ? (a.rows + blocks - 1) / blocks : 0;
    const int cols = (a.n + kNormThreads - 1) / kNormThreads;
    auto kernel = a.df32 ? (a.hf32 ? norm_dw_kernel<true, true> : norm_dw_kernel<true, false>)
                         : (a.hf32 ? norm_dw_kernel<false, true> : norm_dw_kernel<false, false>);
    if (blocks) hipLaunchKernelGGL(kernel, dim3(cols, blocks), dim3(kNormThreads), 0, stream, a, per);
    hipLaunchKernelGGL(norm_dw_sum_kernel, dim3(cols), dim3(kNormThreads), 0, stream, a.partial, blocks, a.n, a.dweight);
  }
  return hipGetLastError();
}

}  // namespace fp8q
