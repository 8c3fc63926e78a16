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
// rot4 as in the token-axis quantizer.  VEC: rows and columns allow whole
// aligned loads, n a multiple of 8; rows outside the source are then read as
// row 0 and dropped, so that all loads of a thread go out together (16384 x
// 7168 BF16: 72 -> 68 us, 5.2 TB/s; the token-axis quantizer of a BF16 tensor,
// which this adds two products per value to, 66 us).  Rows that are read once
// pass the caches by (68 us against 70); those an index may name again, and
// float32 rows, whose 16-byte loads each cover half of their lines, are kept
// there (12288 of 4096 rows x 2048: 19.6 us passing by, 14.8 kept; 8192 x 7168
// float32: 61.8 and 58.9).
template <bool HF32, bool POW2, bool VEC>
__global__ __launch_bounds__(256) void norm_token_kernel(NormTokenArgs a, int ntb, bool rot4) {
  __shared__ TokenTileLds sh;
  const int tid = threadIdx.x;
  const int c8 = tid & 7;
  const int q = tid >> 3;
  const int logical = xcd_block(blockIdx.x, gridDim.x);
  int fg = logical / ntb;
  const int tb = logical - fg * ntb, t0 = tb * 128;
  if (rot4) fg = (fg & ~3) | ((fg + tb) & 3);
  const int f0 = fg * 64, col = f0 + 8 * c8, left = a.n - col;
  int row[4];
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    const int t = t0 + 4 * q + p;
    row[p] = t < a.rows ? t : -1;
    if (a.index && t < a.rows) row[p] = a.index[t];
    if ((unsigned)row[p] >= (unsigned)a.src_rows || left <= 0) row[p] = -1;
  }
  uint4 v[4];
  if constexpr (VEC) {
    const int at = left > 0 ? col : 0;
    Raw<HF32, 8> h[4];
    float r[4], w[8];
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      const int64_t from = (int64_t)max(row[p], 0) * a.ldh + at;
      h[p] = HF32 || a.index ? ld_raw<HF32, 8, true>(a.h, from, 8, true) : ld_raw<HF32, 8, false>(a.h, from, 8, true);
      r[p] = a.rstd[max(row[p], 0)];
    }
    widen_gain8<true>(ld_gain8<true>(a.weight, a.wf32, at, a.n), a.wf32, at, a.n, w);
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      float y[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = normalised(h[p].at(i), r[p], w[i]);
      v[p] = pack_bf16x8(y);
      if (row[p] < 0) v[p] = make_uint4(0, 0, 0, 0);
    }
  } else {
    float w[8] = {};
    if (left > 0) widen_gain8<false>(ld_gain8<false>(a.weight, a.wf32, col, a.n), a.wf32, col, a.n, w);
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      v[p] = make_uint4(0, 0, 0, 0);
      if (row[p] >= 0) {
        const auto h = ld_raw<HF32, 8>(a.h, (int64_t)row[p] * a.ldh + col, left, false);
        const float r = a.rstd[row[p]];
        float y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = normalised(h.at(i), r, w[i]);
        v[p] = pack_bf16x8(y);
      }
    }
  }
  const bool full = a.ldc % 16 == 0 && t0 + 128 <= a.rows && f0 + 64 <= a.n;
  token_tile<POW2>(v, sh, t0, f0, tb, ntb, a.rows, a.n, full, a.codes, a.ldc, a.scales);
}

}  // namespace

template <bool VEC>
static auto norm_token_kernel_of(const NormTokenArgs& a) {
  return a.pow2 ? (a.hf32 ? norm_token_kernel<true, true, VEC> : norm_token_kernel<false, true, VEC>)
                : (a.hf32 ? norm_token_kernel<true, false, VEC> : norm_token_kernel<false, false, VEC>);
}

hipError_t launch_norm_token(const NormTokenArgs& a, hipStream_t stream) {
  const int ntb = (a.rows + 127) / 128, nblk = ntb * ((a.n + 63) / 64);
  const int unit = a.hf32 ? 4 : 8;
  const bool vec = a.src_rows > 0 && a.n % 8 == 0 && a.ldh % unit == 0 && reinterpret_cast<uintptr_t>(a.h) % 16 == 0 && reinterpret_cast<uintptr_t>(a.weight) % 16 == 0;
  const bool rot4 = nblk % 8 == 0 && (nblk / 8) % (4 * ntb) == 0;
  hipLaunchKernelGGL(vec ? norm_token_kernel_of<true>(a) : norm_token_kernel_of<false>(a), dim3(nblk), dim3(256), 0, stream, a, ntb, rot4);
  return hipGetLastError();
}

}  // namespace fp8q
