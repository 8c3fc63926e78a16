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
constexpr int kMaxNormThreads = 1024;
constexpr int kMaxNormGrid = 1 << 20;  // workgroups; more rows go round
enum { kNoStream = 0, kStreamBF16 = 1, kStreamF32 = 2 };

// Eight values of a row.
template <bool F32>
__device__ __forceinline__ void widen(const Raw<F32, 8>& r, float* v) {
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = r.at(i);
}
// Makes the compiler forget what it knows of r, so that a second use widens it
// again: eight widened values kept between two uses take twice the registers
// of eight BF16 ones.
template <bool F32>
__device__ __forceinline__ void forget(Raw<F32, 8>& r) {
  if constexpr (!F32) asm volatile("" : "+v"(r.w[0]), "+v"(r.w[1]), "+v"(r.w[2]), "+v"(r.w[3]));
}
template <bool F32>
__device__ __forceinline__ Raw<F32, 8> as_raw(const float* v) {
  Raw<F32, 8> r;
  if constexpr (F32) {
#pragma unroll
    for (int i = 0; i < 8; ++i) r.w[i] = __float_as_uint(v[i]);
  } else {
    const uint4 c = pack_bf16x8(v);
    r.w[0] = c.x;
    r.w[1] = c.y;
    r.w[2] = c.z;
    r.w[3] = c.w;
  }
  return r;
}
template <bool F32>
__device__ __forceinline__ void st_raw(void* base, int64_t at, const Raw<F32, 8>& r, int left, bool aligned) {
  if constexpr (F32) {
    float v[8];
    widen(r, v);
    st_float4(static_cast<float*>(base) + at, v, left, aligned);
    st_float4(static_cast<float*>(base) + at + 4, v + 4, left - 4, aligned);
  } else {
    st_bf16x8(static_cast<uint16_t*>(base) + at, make_uint4(r.w[0], r.w[1], r.w[2], r.w[3]), left, aligned);
  }
}

// Chunks of eight BF16 values, each quantized with the 16-lane DPP row that
// holds its 1x128 tile; every lane of the wave takes part.  The scales of a
// DPP row's CH tiles are worked out once, by lane u for tile u, as in the row
// quantizer.
template <bool POW2, int CH>
__device__ __forceinline__ void encode_chunks(const uint4 (&d)[CH], uint32_t mine, int row, int col0, int step, int n, bool vec,
                                              uint8_t* codes, int64_t ldc, float* scales) {
  static_assert(CH == 1 || CH == 2 || CH == 4, "tiles u = 0 .. CH - 1 of a DPP row");
  const int sub = threadIdx.x & 15, nb = (n + 127) >> 7;
  const TileScale tm = tile_scale<POW2>(mine);
  {
    const int col = col0 - 8 * sub + sub * step;  // first column of tile `sub`
    if (sub < CH && col < n) scales[(int64_t)row * nb + (col >> 7)] = tm.s;
  }
  auto store = [&](int u, const TileScale& ts, auto enc) {
    const uint2 c = enc(d[u], ts);
    const int col = col0 + u * step, left = n - col;
    if (left > 0) st_codes8(codes + (int64_t)row * ldc + col, c, vec ? 8 : left, vec);
  };
  auto all = [&](auto enc) {
    store(0, row_tile_scale<POW2, 0>(tm), enc);
    if constexpr (CH > 1) store(1, row_tile_scale<POW2, 1>(tm), enc);
    if constexpr (CH > 2) {
      store(2, row_tile_scale<POW2, 2>(tm), enc);
      store(3, row_tile_scale<POW2, 3>(tm), enc);
    }
  };
  if constexpr (POW2) {
    all([](uint4 x, const TileScale& t) { return encode8<true>(x, t); });
  } else if (__builtin_amdgcn_ballot_w64(sub < CH && tm.slow) == 0) {  // (one wave-uniform decision)
    all([](uint4 x, const TileScale& t) { return encode8_markstein<false>(x, t); });
  } else {
    all([](uint4 x, const TileScale& t) { return encode8_markstein<true>(x, t); });
  }
}

// col0: the lane's first column, chunk u is u * step further.
template <int CH>
__device__ __forceinline__ void quantize_chunks(const uint4 (&d)[CH], bool pow2, int row, int col0, int step, int n, bool vec, uint8_t* codes,
                                                int64_t ldc, float* scales) {
  uint32_t mine = 0;  // lane u: tile u's max-abs
#pragma unroll
  for (int u = 0; u < CH; ++u) {
    const uint32_t amax = dpp_max16(absmax8(d[u]));
    mine = CH == 1 || (threadIdx.x & 15) == u ? amax : mine;
  }
  if (pow2) {
    encode_chunks<true, CH>(d, mine, row, col0, step, n, vec, codes, ldc, scales);
  } else {
    encode_chunks<false, CH>(d, mine, row, col0, step, n, vec, codes, ldc, scales);
  }
}

// -------------------------------------------------------------- forward ---
// One workgroup per row, CH chunks of eight columns a thread, the row kept in
// registers: every byte is moved once.
template <bool XF32, int STREAM, bool VEC, bool KEEP, int CH>
__global__ __launch_bounds__(CH == 4 ? kMaxNormThreads / 2 : kMaxNormThreads) void norm_row_kernel(NormArgs a) {
  static_assert(VEC || KEEP, "loads of unaligned rows are plain ones");
  constexpr bool RES = STREAM != kNoStream, HF32 = RES ? STREAM == kStreamF32 : XF32;
  __shared__ double part[kMaxNormThreads / 64];
  const int tid = threadIdx.x, step = (int)blockDim.x * 8;
  const bool out = a.y || a.codes;
  for (int row = blockIdx.x; row < a.rows; row += (int)gridDim.x) {
    Raw<HF32, 8> h[CH];
    Gain8 w[CH];
    {
      Raw<XF32, 8> x[CH];
      Raw<RES && HF32, 8> s[CH];
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const int col = c * step + tid * 8, left = a.n - col;
        x[c] = {};
        s[c] = {};
        if (left > 0) {
          x[c] = ld_row8<XF32, VEC, KEEP>(a.x, (int64_t)row * a.ldx, col, a.n);
          if constexpr (RES) s[c] = ld_row8<HF32, VEC, KEEP>(a.res, (int64_t)row * a.ldr, col, a.n);
        }
      }
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const int col = c * step + tid * 8, left = a.n - col;
        w[c] = {};
        if (out && left > 0) w[c] = ld_gain8<VEC>(a.weight, a.wf32, col, a.n);
      }
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        if constexpr (RES) {
          float v[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] = x[c].at(i) + s[c].at(i);
          h[c] = as_raw<HF32>(v);
        } else {
          h[c] = x[c];
        }
      }
    }
    double sum = 0.0;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const double v = (double)h[c].at(i);
        sum = __builtin_fma(v, v, sum);
      }
      forget(h[c]);
      const int col = c * step + tid * 8, left = a.n - col;
      if (RES && a.h && left > 0) st_raw(a.h, (int64_t)row * a.ldh + col, h[c], VEC ? 8 : left, VEC);
    }
    const float r = reciprocal_rms(block_sum(sum, part), a.inv_n, a.eps);
    if (tid == 0 && a.rstd) a.rstd[row] = r;
    if (out) {
      uint4 d[CH];
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const int col = c * step + tid * 8, left = a.n - col;
        float g[8], v[8];
        widen_gain8(w[c], a.wf32, g);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = normalised(h[c].at(i), r, g[i]);
        d[c] = pack_bf16x8(v);
        if (a.y && left > 0) st_bf16x8(a.y + (int64_t)row * a.ldy + col, d[c], VEC ? 8 : left, VEC);
      }
      if (a.codes) quantize_chunks<CH>(d, a.pow2, row, tid * 8, step, a.n, VEC, a.codes, a.ldc, a.scales);
    }
    if (row + (int)gridDim.x < a.rows) __syncthreads();  // (part is written again)
  }
}

// Rows of more columns than a workgroup's registers hold: the row is read
// twice, the second time from the stream just written (which may be the
// residual itself) where there is one.
template <bool XF32, int STREAM>
__global__ __launch_bounds__(kMaxNormThreads) void norm_long_kernel(NormArgs a) {
  constexpr bool RES = STREAM != kNoStream, HF32 = RES ? STREAM == kStreamF32 : XF32;
  __shared__ double part[kMaxNormThreads / 64];
  const int tid = threadIdx.x, step = (int)blockDim.x * 8;
  auto load = [&](int row, int col) {
    const auto x = ld_row8<XF32, false, true>(a.x, (int64_t)row * a.ldx, col, a.n);
    if constexpr (RES) {
      const auto s = ld_row8<HF32, false, true>(a.res, (int64_t)row * a.ldr, col, a.n);
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = x.at(i) + s.at(i);
      return as_raw<HF32>(v);
    } else {
      return x;
    }
  };
  for (int row = blockIdx.x; row < a.rows; row += (int)gridDim.x) {
    double sum = 0.0;
    for (int col = tid * 8; col < a.n; col += step) {
      const auto h = load(row, col);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const double v = (double)h.at(i);
        sum = __builtin_fma(v, v, sum);
      }
      if (RES && a.h) st_raw(a.h, (int64_t)row * a.ldh + col, h, a.n - col, false);
    }
    const float r = reciprocal_rms(block_sum(sum, part), a.inv_n, a.eps);
    if (tid == 0 && a.rstd) a.rstd[row] = r;
    if (a.y || a.codes) {
      for (int c0 = 0; c0 < a.n; c0 += step) {
        const int col = c0 + tid * 8, left = a.n - col;
        Raw<HF32, 8> h = {};
        float w[8] = {}, v[8];
        if (left > 0) {
          h = RES && a.h ? ld_row8<HF32, false, true>(a.h, (int64_t)row * a.ldh, col, a.n) : load(row, col);
          widen_gain8(ld_gain8<false>(a.weight, a.wf32, col, a.n), a.wf32, w);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = normalised(h.at(i), r, w[i]);
        const uint4 d[1] = {pack_bf16x8(v)};
        if (a.y && left > 0) st_bf16x8(a.y + (int64_t)row * a.ldy + col, d[0], left, false);
        if (a.codes) quantize_chunks<1>(d, a.pow2, row, col, 0, a.n, false, a.codes, a.ldc, a.scales);
      }
    }
    __syncthreads();  // (part is written again)
  }
}

// ------------------------------------------------------------- backward ---
// CH chunks of eight columns a thread; the row is kept in registers between
// the dot product and its use, and the gain and the thread's share of its
// gradient from row to row.  WAVE: every wave of the workgroup is on a row of
// its own, without a barrier; else a row is the workgroup's.  The workgroup's
// share of dw goes to `partial` at the end.
template <bool DF32, bool HF32, bool OF32, bool VEC, bool KEEP, int CH, bool WAVE>
__global__ __launch_bounds__(WAVE ? 256 : 1024) void norm_bwd_rows_kernel(NormBwdArgs a) {
  __shared__ double part[2][kMaxNormThreads / 64];
  __shared__ float share[WAVE ? CH * 512 : 1];
  const int slot = WAVE ? (int)threadIdx.x >> 6 : 0, tid = WAVE ? (int)threadIdx.x & 63 : (int)threadIdx.x;
  const int lanes = WAVE ? 64 : (int)blockDim.x, slots = WAVE ? (int)blockDim.x >> 6 : 1, step = lanes * 8;
  float w[CH][8], dw[CH][8];
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int col = c * step + tid * 8;
    Gain8 g = {};
    if (a.weight && col < a.n) g = ld_gain8<VEC>(a.weight, a.wf32, col, a.n);
    widen_gain8(g, a.wf32, w[c]);
#pragma unroll
    for (int i = 0; i < 8; ++i) dw[c][i] = 0.0f;
  }
  int turn = 0;
  for (int64_t row64 = (int64_t)blockIdx.x * slots + slot; row64 < a.rows; row64 += (int64_t)gridDim.x * slots) {
    const int row = (int)row64;
    const float r = a.rstd[row];
    Raw<DF32, 8> dy[CH];
    Raw<HF32, 8> h[CH];
    Raw<OF32, 8> res[CH];
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int col = c * step + tid * 8;
      dy[c] = {};
      h[c] = {};
      res[c] = {};
      if (col < a.n) {
        dy[c] = ld_row8<DF32, VEC, KEEP>(a.dy, (int64_t)row * a.lddy, col, a.n);
        h[c] = ld_row8<HF32, VEC, KEEP>(a.h, (int64_t)row * a.ldh, col, a.n);
        if (a.dres) res[c] = ld_row8<OF32, VEC, KEEP>(a.dres, (int64_t)row * a.lddr, col, a.n);
      }
    }
    double sum = 0.0;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float d = dy[c].at(i), v = h[c].at(i);
        dw[c][i] = __builtin_fmaf(d, v * r, dw[c][i]);
        sum = __builtin_fma((double)(d * w[c][i]), (double)v, sum);
      }
      // (the sum is formed here, not where it is used with every widened value alive until then)
      asm volatile("" : "+v"(sum));
      forget(dy[c]);
      forget(h[c]);
    }
    if (!a.dx && !a.codes) continue;
    sum = wave_sum(sum);
    if constexpr (!WAVE) {
      // two sets of partial sums in turn: a wave two rows ahead has passed the barrier in between
      if ((tid & 63) == 0) part[turn][tid >> 6] = sum;
      __syncthreads();
      sum = part[turn][0];
      for (int i = 1; i < lanes >> 6; ++i) sum += part[turn][i];
      turn ^= 1;
    }
    const float mean = (float)(sum * (double)r * a.inv_n);
    uint4 d[CH];
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int col = c * step + tid * 8, left = a.n - col;
      float g[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        g[i] = (dy[c].at(i) * w[c][i] - (h[c].at(i) * r) * mean) * r;
        if (a.dres) g[i] += res[c].at(i);
      }
      const auto o = as_raw<OF32>(g);
      if (a.dx && left > 0) st_raw(a.dx, (int64_t)row * a.lddx + col, o, VEC ? 8 : left, VEC);
      if constexpr (OF32) {
        d[c] = pack_bf16x8(g);
      } else {
        d[c] = make_uint4(o.w[0], o.w[1], o.w[2], o.w[3]);
      }
    }
    if (a.codes) quantize_chunks<CH>(d, a.pow2, row, tid * 8, step, a.n, VEC, a.codes, a.ldc, a.scales);
  }
  if (!a.dweight) return;
  if constexpr (WAVE) {
    // the slots' shares, one after another
    for (int s = 0; s < slots; ++s) {
      if (slot == s) {
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            float* p = share + (c * 8 + i) * 64 + tid;
            dw[c][i] = s ? *p + dw[c][i] : dw[c][i];
            if (s < slots - 1) *p = dw[c][i];
          }
      }
      __syncthreads();
    }
    if (slot < slots - 1) return;
  }
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int col = c * step + tid * 8, left = a.n - col;
    float* p = a.partial + (int64_t)blockIdx.x * a.ldp + col;
    if (left > 0) {
      // (rows of partial are padded to whole chunks)
      *reinterpret_cast<float4*>(p) = make_float4(dw[c][0], dw[c][1], dw[c][2], dw[c][3]);
      *reinterpret_cast<float4*>(p + 4) = make_float4(dw[c][4], dw[c][5], dw[c][6], dw[c][7]);
    }
  }
}

// Rows of more columns than a workgroup's registers hold: gone over twice, the
// gain's gradient by a kernel of its own.
template <bool DF32, bool HF32, bool OF32>
__global__ __launch_bounds__(kMaxNormThreads) void norm_bwd_long_kernel(NormBwdArgs a) {
  __shared__ double part[kMaxNormThreads / 64];
  const int step = (int)blockDim.x * 8, tid = threadIdx.x;
  for (int row = blockIdx.x; row < a.rows; row += (int)gridDim.x) {
    const float r = a.rstd[row];
    auto load = [&](int col, float* g, float* h) {
      float w[8];
      widen(ld_row8<DF32, false, true>(a.dy, (int64_t)row * a.lddy, col, a.n), g);
      widen(ld_row8<HF32, false, true>(a.h, (int64_t)row * a.ldh, col, a.n), h);
      widen_gain8(ld_gain8<false>(a.weight, a.wf32, col, a.n), a.wf32, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) g[i] *= w[i];
    };
    double sum = 0.0;
    for (int col = tid * 8; col < a.n; col += step) {
      float g[8], h[8];
      load(col, g, h);
#pragma unroll
      for (int i = 0; i < 8; ++i) sum = __builtin_fma((double)g[i], (double)h[i], sum);
    }
    const float mean = (float)(block_sum(sum, part) * (double)r * a.inv_n);
    for (int c0 = 0; c0 < a.n; c0 += step) {
      const int col = c0 + tid * 8, left = a.n - col;
      float g[8] = {}, h[8] = {}, s[8] = {};
      if (left > 0) {
        load(col, g, h);
        if (a.dres) widen(ld_row8<OF32, false, true>(a.dres, (int64_t)row * a.lddr, col, a.n), s);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        g[i] = (g[i] - (h[i] * r) * mean) * r;
        if (a.dres) g[i] += s[i];
      }
      if (a.dx && left > 0) st_raw(a.dx, (int64_t)row * a.lddx + col, as_raw<OF32>(g), left, false);
      const uint4 d[1] = {pack_bf16x8(g)};
      if (a.codes) quantize_chunks<1>(d, a.pow2, row, col, 0, a.n, false, a.codes, a.ldc, a.scales);
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
  a.partial[(int64_t)blockIdx.y * a.ldp + col] = sum;
}

// The blocks' shares of 64 columns: 64 sums of every 64th block, four columns a
// thread, then those in their order.
__global__ __launch_bounds__(1024) void norm_dw_sum_kernel(const float* partial, int blocks, int n, int64_t ldp, float* dw) {
  __shared__ __attribute__((aligned(16))) float part[64][64];
  const int tid = threadIdx.x, group = tid >> 4, c4 = (tid & 15) * 4, col = (int)blockIdx.x * 64 + c4;
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
  if (col < n) {
#pragma unroll 4
    for (int b = group; b < blocks; b += 64) {
      const float4 v = *reinterpret_cast<const float4*>(partial + (int64_t)b * ldp + col);
      s.x += v.x;
      s.y += v.y;
      s.z += v.z;
      s.w += v.w;
    }
  }
  *reinterpret_cast<float4*>(&part[group][c4]) = s;
  __syncthreads();
  const int c = tid & 63, q = tid >> 6;  // 16 waves, four of the sums each
  float v = (part[4 * q][c] + part[4 * q + 1][c]) + (part[4 * q + 2][c] + part[4 * q + 3][c]);
  __syncthreads();
  part[q][c] = v;
  __syncthreads();
  if (tid < 64 && (int)blockIdx.x * 64 + tid < n) {
    v = part[0][tid];
#pragma unroll
    for (int i = 1; i < 16; ++i) v += part[i][tid];
    dw[blockIdx.x * 64 + tid] = v;
  }
}

}  // namespace

static int norm_grid(int rows) { return rows < kMaxNormGrid ? rows : kMaxNormGrid; }

template <bool XF32, int STREAM, bool VEC, bool KEEP>
static void launch_norm_rows(const NormArgs& a, int threads, int chunks, hipStream_t stream) {
  auto kernel = chunks == 1   ? norm_row_kernel<XF32, STREAM, VEC, KEEP, 1>
                : chunks == 2 ? norm_row_kernel<XF32, STREAM, VEC, KEEP, 2>
                              : norm_row_kernel<XF32, STREAM, VEC, KEEP, 4>;
  hipLaunchKernelGGL(kernel, dim3(norm_grid(a.rows)), dim3(threads), 0, stream, a);
}

template <bool XF32, int STREAM>
static void launch_norm_typed(const NormArgs& a, hipStream_t stream) {
  const bool vec = a.n % 8 == 0 && a.ldx % 8 == 0 && (!a.res || a.ldr % 8 == 0) && (!a.h || a.ldh % 8 == 0) && (!a.y || a.ldy % 8 == 0) &&
                   (!a.codes || a.ldc % 8 == 0);
  const int chunks = norm_chunks(a.rows, a.n), threads = norm_threads(a.n, chunks);
  if (threads == 0) {
    hipLaunchKernelGGL((norm_long_kernel<XF32, STREAM>), dim3(norm_grid(a.rows)), dim3(kMaxNormThreads), 0, stream, a);
    return;
  }
  if constexpr (!XF32 && STREAM != kStreamF32) {
    if (vec && !input_stays_cached(a.rows, (int64_t)a.n * (STREAM == kNoStream ? 2 : 4))) {
      launch_norm_rows<XF32, STREAM, true, false>(a, threads, chunks, stream);
      return;
    }
  }
  if (vec) {
    launch_norm_rows<XF32, STREAM, true, true>(a, threads, chunks, stream);
  } else {
    launch_norm_rows<XF32, STREAM, false, true>(a, threads, chunks, stream);
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

template <bool DF32, bool HF32, bool OF32, bool VEC, bool KEEP>
static void launch_norm_bwd_rows(const NormBwdArgs& a, const NormBwdShape& s, hipStream_t stream) {
  auto kernel = !s.wave         ? norm_bwd_rows_kernel<DF32, HF32, OF32, VEC, KEEP, 2, false>
                : s.chunks == 1 ? norm_bwd_rows_kernel<DF32, HF32, OF32, VEC, KEEP, 1, true>
                                : norm_bwd_rows_kernel<DF32, HF32, OF32, VEC, KEEP, 2, true>;
  hipLaunchKernelGGL(kernel, dim3(s.blocks), dim3(s.threads), 0, stream, a);
}

template <bool DF32, bool HF32, bool OF32>
static void launch_norm_bwd_typed(const NormBwdArgs& a, hipStream_t stream) {
  const NormBwdShape s = norm_bwd_shape(a.rows, a.n);
  if (s.chunks == 0) {
    if (a.dx || a.codes)
      hipLaunchKernelGGL((norm_bwd_long_kernel<DF32, HF32, OF32>), dim3(norm_grid(a.rows)), dim3(kMaxNormThreads), 0, stream, a);
    if (a.dweight) {
      const int per = (a.rows + s.blocks - 1) / s.blocks;
      hipLaunchKernelGGL((norm_dw_kernel<DF32, HF32>), dim3((a.n + kNormThreads - 1) / kNormThreads, s.blocks), dim3(kNormThreads), 0, stream, a, per);
    }
    return;
  }
  const bool vec = a.n % 8 == 0 && a.lddy % 8 == 0 && a.ldh % 8 == 0 && (!a.dres || a.lddr % 8 == 0) && (!a.dx || a.lddx % 8 == 0) &&
                   (!a.codes || a.ldc % 8 == 0);
  if constexpr (!DF32 && !HF32 && !OF32) {
    if (vec && !input_stays_cached(a.rows, (int64_t)a.n * (a.dres ? 6 : 4))) {
      launch_norm_bwd_rows<DF32, HF32, OF32, true, false>(a, s, stream);
      return;
    }
  }
  if (vec) {
    launch_norm_bwd_rows<DF32, HF32, OF32, true, true>(a, s, stream);
  } else {
    launch_norm_bwd_rows<DF32, HF32, OF32, false, true>(a, s, stream);
  }
}

hipError_t launch_norm_backward(const NormBwdArgs& args, hipStream_t stream) {
  NormBwdArgs a = args;
  a.ldp = norm_partial_ld(a.n);
  if (a.rows > 0) {
    auto launch = a.df32 ? (a.hf32 ? (a.of32 ? launch_norm_bwd_typed<true, true, true> : launch_norm_bwd_typed<true, true, false>)
                                   : (a.of32 ? launch_norm_bwd_typed<true, false, true> : launch_norm_bwd_typed<true, false, false>))
                         : (a.hf32 ? (a.of32 ? launch_norm_bwd_typed<false, true, true> : launch_norm_bwd_typed<false, true, false>)
                                   : (a.of32 ? launch_norm_bwd_typed<false, false, true> : launch_norm_bwd_typed<false, false, false>));
    launch(a, stream);
  }
  if (a.dweight) {
    const int blocks = a.rows > 0 ? norm_bwd_shape(a.rows, a.n).blocks : 0;
    hipLaunchKernelGGL(norm_dw_sum_kernel, dim3((a.n + 63) / 64), dim3(1024), 0, stream, a.partial, blocks, a.n, a.ldp, a.dweight);
  }
  return hipGetLastError();
}

}  // namespace fp8q
