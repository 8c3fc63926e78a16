// Residual addition, RMS norm and 1x128 quantization in one pass, gfx950.
//
// Per row of n columns (norm_common.h has the roundings):
//   h = rn(x + res),  r = rn32(1 / sqrt(mean(h^2) + eps)),  y = bf16((h r) w),
// y in BF16 and / or as E4M3 codes with 1x128 scales, what the quantizer would
// make of that BF16 tensor.
#include "fp8q_internal.h"
#include "norm_common.h"

namespace fp8q {
namespace {

constexpr int kMaxNormThreads = 1024;
enum { kNoStream = 0, kStreamBF16 = 1, kStreamF32 = 2 };

// One workgroup per row, CH chunks of eight columns a thread (norm_shape), the
// row kept in registers: every byte is moved once.  SPLIT: the threads hold
// halves of what those of many rows hold (split_sum).  With a residual HBM bounds
// it: 16384 x 7168 BF16 to E4M3 137-139 us, 6.0 TB/s at 4:3 reads to writes (127 us
// at the rates of plain reads and fills).  Without one the vector instructions
// do, 20 a value: 76-79 us, where the bytes take 55; BF16 out 79, the bytes 73.
// One row takes 3.6 us, 2.6 of them the launch: of the rest most is two loads
// and a barrier in a row, one after another.
template <bool XF32, int STREAM, bool VEC, bool KEEP, int CH, bool SPLIT>
__global__ __launch_bounds__(CH == 4 ? kMaxNormThreads / 2 : kMaxNormThreads) void norm_row_kernel(NormArgs a) {
  static_assert(VEC || KEEP, "loads of unaligned rows are plain ones");
  constexpr bool RES = STREAM != kNoStream, HF32 = RES ? STREAM == kStreamF32 : XF32;
  __shared__ double part[kMaxNormThreads / 64];
  const int tid = SPLIT ? split_thread<CH>() : (int)threadIdx.x, step = (int)blockDim.x * 8;
  const bool out = a.y || a.codes;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    Raw<HF32, 8> h[CH];
    Gain8 w[CH];
    {
      const Row<XF32, VEC, KEEP> rx(a.x, row * a.ldx, a.n);
      const Row<HF32, VEC, KEEP> rs(RES ? a.res : a.x, RES ? row * a.ldr : 0, a.n);
      Raw<XF32, 8> x[CH];
      Raw<HF32, 8> s[CH];
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        x[c] = rx.load(c * step + tid * 8);
        if constexpr (RES) s[c] = rs.load(c * step + tid * 8);
      }
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        w[c] = {};
        if (out) w[c] = ld_gain8<VEC>(a.weight, a.wf32, c * step + tid * 8, a.n);
      }
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        rx.settle(c * step + tid * 8, x[c]);
        if constexpr (RES) {
          rs.settle(c * step + tid * 8, s[c]);
          float v[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] = x[c].at(i) + s[c].at(i);
          h[c] = as_raw<HF32>(v);
        } else {
          h[c] = x[c];
        }
      }
    }
    const Row<HF32, VEC> rh(a.h, row * a.ldh, a.n);
    double sums[CH];
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      sums[c] = 0.0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const double v = (double)h[c].at(i);
        sums[c] = __builtin_fma(v, v, sums[c]);
      }
      forget(h[c]);
      if (RES && a.h) rh.store(c * step + tid * 8, h[c]);
    }
    // (the halves of the row's threads apart, as few rows have them)
    double sum = sums[0];
    if constexpr (CH == 2) sum += sums[1];
    if constexpr (CH == 4) sum = (sums[0] + sums[2]) + (sums[1] + sums[3]);
    const float r = reciprocal_rms(SPLIT ? split_sum<CH>(sum, part) : block_sum(sum, part), a.inv_n, a.eps);
    if (tid == 0 && a.rstd) a.rstd[row] = r;
    if (out) {
      const Row<false, VEC> ry(a.y, row * a.ldy, a.n);
      uint4 d[CH];
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const int col = c * step + tid * 8;
        float g[8], v[8];
        widen_gain8<VEC>(w[c], a.wf32, col, a.n, g);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = normalised(h[c].at(i), r, g[i]);
        d[c] = pack_bf16x8(v);
        if (a.y) ry.store(col, as_raw<false>(v));
      }
      if (a.codes) quantize_chunks<VEC, CH>(d, a.pow2, row, tid * 8, step, a.n, a.codes, a.ldc, a.scales);
    }
    if (row + (int)gridDim.x < a.rows) __syncthreads();  // (part is written again)
  }
}

// Rows of more columns than a workgroup's registers hold: the row is read
// twice, the second time from the stream just written (which may be the
// residual itself) where there is one.  (512 x 20000 23 us, the bytes 11; the
// second reading comes from the caches, but a workgroup's loads wait for one
// another: 512 x 16384 in registers 14 us, the bytes 9.)
template <bool XF32, int STREAM>
__global__ __launch_bounds__(kMaxNormThreads) void norm_long_kernel(NormArgs a) {
  constexpr bool RES = STREAM != kNoStream, HF32 = RES ? STREAM == kStreamF32 : XF32;
  __shared__ double part[kMaxNormThreads / 64];
  const int tid = threadIdx.x, step = (int)blockDim.x * 8;
  auto load = [&](int64_t row, int col) {
    const auto x = Row<XF32, false>(a.x, row * a.ldx, a.n).settled(col);
    if constexpr (RES) {
      const auto s = Row<HF32, false>(a.res, row * a.ldr, a.n).settled(col);
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = x.at(i) + s.at(i);
      return as_raw<HF32>(v);
    } else {
      return x;
    }
  };
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    double sum = 0.0;
    for (int col = tid * 8; col < a.n; col += step) {
      const auto h = load(row, col);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const double v = (double)h.at(i);
        sum = __builtin_fma(v, v, sum);
      }
      if (RES && a.h) Row<HF32, false>(a.h, row * a.ldh, a.n).store(col, h);
    }
    const float r = reciprocal_rms(block_sum(sum, part), a.inv_n, a.eps);
    if (tid == 0 && a.rstd) a.rstd[row] = r;
    if (a.y || a.codes) {
      for (int c0 = 0; c0 < a.n; c0 += step) {
        const int col = c0 + tid * 8;
        Raw<HF32, 8> h = {};
        float w[8] = {}, v[8];
        if (col < a.n) {
          h = RES && a.h ? Row<HF32, false>(a.h, row * a.ldh, a.n).settled(col) : load(row, col);
          widen_gain8<false>(ld_gain8<false>(a.weight, a.wf32, col, a.n), a.wf32, col, a.n, w);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = normalised(h.at(i), r, w[i]);
        const uint4 d[1] = {pack_bf16x8(v)};
        if (a.y) Row<false, false>(a.y, row * a.ldy, a.n).store(col, as_raw<false>(v));
        if (a.codes) quantize_chunks<false, 1>(d, a.pow2, row, col, 0, a.n, a.codes, a.ldc, a.scales);
      }
    }
    __syncthreads();  // (part is written again)
  }
}

}  // namespace

static int norm_grid(int rows) { return rows < kMaxNormGrid ? rows : kMaxNormGrid; }

template <bool XF32, int STREAM, bool VEC, bool KEEP>
static void launch_norm_rows(const NormArgs& a, const NormShape& s, hipStream_t stream) {
  auto kernel = s.split ? (s.chunks == 1 ? norm_row_kernel<XF32, STREAM, VEC, KEEP, 1, true> : norm_row_kernel<XF32, STREAM, VEC, KEEP, 2, true>)
                : s.chunks == 1 ? norm_row_kernel<XF32, STREAM, VEC, KEEP, 1, false>
                : s.chunks == 2 ? norm_row_kernel<XF32, STREAM, VEC, KEEP, 2, false>
                                : norm_row_kernel<XF32, STREAM, VEC, KEEP, 4, false>;
  hipLaunchKernelGGL(kernel, dim3(norm_grid(a.rows)), dim3(s.threads), 0, stream, a);
}

template <bool XF32, int STREAM>
static void launch_norm_typed(const NormArgs& a, hipStream_t stream) {
  const bool vec = a.n % 8 == 0 && a.ldx % 8 == 0 && (!a.res || a.ldr % 8 == 0) && (!a.h || a.ldh % 8 == 0) && (!a.y || a.ldy % 8 == 0) &&
                   (!a.codes || a.ldc % 8 == 0);
  const NormShape s = norm_shape(a.rows, a.n);
  if (s.threads == 0) {
    hipLaunchKernelGGL((norm_long_kernel<XF32, STREAM>), dim3(norm_grid(a.rows)), dim3(kMaxNormThreads), 0, stream, a);
    return;
  }
  if constexpr (!XF32 && STREAM != kStreamF32) {
    if (vec && !input_stays_cached(a.rows, (int64_t)a.n * (STREAM == kNoStream ? 2 : 4))) {
      launch_norm_rows<XF32, STREAM, true, false>(a, s, stream);
      return;
    }
  }
  if (vec) {
    launch_norm_rows<XF32, STREAM, true, true>(a, s, stream);
  } else {
    launch_norm_rows<XF32, STREAM, false, true>(a, s, stream);
  }
}

hipError_t launch_norm(const NormArgs& a, hipStream_t stream) {
  const int kind = !a.res ? kNoStream : a.sf32 ? kStreamF32 : kStreamBF16;
  if (a.xf32) {
    kind == kNoStream ? launch_norm_typed<true, kNoStream>(a, stream)
    : kind == kStreamF32 ? launch_norm_typed<true, kStreamF32>(a, stream) : launch_norm_typed<true, kStreamBF16>(a, stream);
  } else {
    kind == kNoStream ? launch_norm_typed<false, kNoStream>(a, stream)
    : kind == kStreamF32 ? launch_norm_typed<false, kStreamF32>(a, stream) : launch_norm_typed<false, kStreamBF16>(a, stream);
  }
  return hipGetLastError();
}

}  // namespace fp8q
