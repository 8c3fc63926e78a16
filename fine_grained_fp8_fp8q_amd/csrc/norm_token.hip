// The rows of an RMS norm formed again from its kept input and 1 / rms, in
// 128x1 token-axis tiles: the operand of a weight gradient (gfx950).
//
// y[t] = bf16((h[index[t]] r[index[t]]) w), bit for bit what the forward pass
// quantized (norm_common.h), then transposed tiles as the token-axis quantizer
// makes them of that BF16 tensor (token_tile.h).  With an index (the token
// list of a routing table) the rows come in expert order and its padding, rows
// outside the source, is zero.
#include "fp8q_internal.h"
#include "norm_common.h"
#include "token_tile.h"

namespace fp8q {
namespace {

// Workgroup tile: 128 tokens x 64 features; the token block varies fastest.
template <bool HF32, bool POW2>
__global__ __launch_bounds__(256) void norm_token_kernel(NormTokenArgs a, int ntb) {
  __shared__ TokenTileLds sh;
  const int tid = threadIdx.x;
  const int c8 = tid & 7;
  const int q = tid >> 3;
  const int logical = xcd_block(blockIdx.x, gridDim.x);
  const int tb = logical % ntb, t0 = tb * 128, f0 = logical / ntb * 64;
  const int col = f0 + 8 * c8, left = a.n - col;
  uint4 v[4];
  float w[8] = {};
  if (left > 0) widen_gain8<false>(ld_gain8<false>(a.weight, a.wf32, col, a.n), a.wf32, col, a.n, w);
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    const int t = t0 + 4 * q + p;
    int row = t < a.rows ? t : -1;
    if (a.index && row >= 0) row = a.index[t];
    v[p] = make_uint4(0, 0, 0, 0);
    if ((unsigned)row < (unsigned)a.src_rows && left > 0) {
      const auto h = ld_raw<HF32, 8>(a.h, (int64_t)row * a.ldh + col, left, false);
      const float r = a.rstd[row];
      float y[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = normalised(h.at(i), r, w[i]);
      v[p] = pack_bf16x8(y);
    }
  }
  const bool full = a.ldc % 16 == 0 && t0 + 128 <= a.rows && f0 + 64 <= a.n;
  token_tile<POW2>(v, sh, t0, f0, tb, ntb, a.rows, a.n, full, a.codes, a.ldc, a.scales);
}

}  // namespace

hipError_t launch_norm_token(const NormTokenArgs& a, hipStream_t stream) {
  const int ntb = (a.rows + 127) / 128;
  const dim3 grid(ntb * ((a.n + 63) / 64)), block(256);
  auto kernel = a.pow2 ? (a.hf32 ? norm_token_kernel<true, true> : norm_token_kernel<false, true>)
                       : (a.hf32 ? norm_token_kernel<true, false> : norm_token_kernel<false, false>);
  hipLaunchKernelGGL(kernel, grid, block, 0, stream, a, ntb);
  return hipGetLastError();
}

}  // namespace fp8q
