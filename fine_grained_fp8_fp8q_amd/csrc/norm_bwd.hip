// The gradient of the residual addition with RMS norm (norm.hip), gfx950.
//
// With g = dy w, t = h r and c = rn32(mean(g h) r), the sum in 64 bits:
//   dx = (g - t c) r + dres,   dw = sum over rows of dy t.
// One pass: a row is kept in registers between the dot product and its use.
#include "fp8q_internal.h"
#include "norm_common.h"

namespace fp8q {
namespace {

constexpr int kSlots = 4;  // waves of a workgroup, each on a row of its own
constexpr int kNormThreads = 256;
constexpr int kMaxNormThreads = 1024;

template <bool DF32, bool HF32, bool OF32, int CH>
struct NormBwdRow {
  Raw<DF32, 8> dy[CH];
  Raw<HF32, 8> h[CH];
  Raw<OF32, 8> res[CH];
  float r;
};

// CH chunks of eight columns a thread; the gain and the thread's share of its
// gradient stay in registers from row to row.  WAVE: every wave of the
// workgroup is on a row of its own, without a barrier; else a row is the
// workgroup's.  The next row's loads are on their way while a row is worked on:
// the registers hold two rows, which leaves two waves a SIMD, and their bytes
// are what is in flight.  The workgroup's share of dw goes to `partial` at the
// end.  HBM bounds it where rows are long and many (8192 x 7168 BF16 87 us with
// the sum of the shares, 5.4 TB/s at 3:1, 73 us at the rates of plain reads and
// fills; its codes too 108), the two launches where they are few (one row 6.9
// us), and the vector instructions where rows begin anywhere (their ends are
// shifted into place: 4096 x 7001 70 us, the bytes 36).
// Three chunks a lane with float32 values are held to the registers of two waves
// a SIMD: float32 dy and dx beside BF16 h on unaligned rows need four more
// (8192 x 1030 34.7 us with those spilled, 38.4 with one wave).
template <bool DF32, bool HF32, bool OF32, bool VEC, bool KEEP, int CH, bool WAVE>
__global__ __launch_bounds__(WAVE ? 256 : 512, WAVE && CH == 3 && (DF32 || HF32 || OF32) ? 2 : 1) void norm_bwd_rows_kernel(NormBwdArgs a) {
  // Rows of 129 to 192 chunks with float32 values go to a wave each or to
  // workgroups of two, by their number.  Both add a lane's chunks 128 apart, then
  // those 64 apart, which are the two waves', then the lanes: the same sum.
  constexpr bool kApart = (DF32 || HF32 || OF32) && CH == (WAVE ? 3 : 2);
  __shared__ double part[2][kApart && !WAVE ? 128 : kMaxNormThreads / 64];
  __shared__ __attribute__((aligned(16))) float4 share[WAVE ? kSlots * CH * 128 : 1];
  const int slot = WAVE ? (int)threadIdx.x >> 6 : 0, tid = WAVE ? (int)threadIdx.x & 63 : (int)threadIdx.x;
  const int lanes = WAVE ? 64 : (int)blockDim.x, slots = WAVE ? (int)blockDim.x >> 6 : 1, step = lanes * 8;
  auto load = [&](int64_t row) {
    const bool on = row < a.rows;
    const int64_t at = on ? row : 0;
    const Row<DF32, VEC, KEEP> dy(a.dy, at * a.lddy, a.n, on);
    const Row<HF32, VEC, KEEP> h(a.h, at * a.ldh, a.n, on);
    const Row<OF32, VEC, KEEP> res(a.dres, at * a.lddr, a.n, on && a.dres);
    NormBwdRow<DF32, HF32, OF32, CH> v;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int col = c * step + tid * 8;
      v.dy[c] = dy.load(col);
      v.h[c] = h.load(col);
      v.res[c] = {};
      if (VEC || a.dres) v.res[c] = res.load(col);
    }
    v.r = a.rstd[at];
    return v;
  };
  const int64_t rows_a_turn = (int64_t)gridDim.x * slots;
  int64_t row = (int64_t)blockIdx.x * slots + __builtin_amdgcn_readfirstlane(slot);
  auto v = load(row);
  float w[CH][8], dw[CH][8];
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int col = c * step + tid * 8;
    Gain8 g = {};
    if (a.weight) g = ld_gain8<VEC>(a.weight, a.wf32, col, a.n);
    widen_gain8<VEC>(g, a.wf32, col, a.n, w[c]);
#pragma unroll
    for (int i = 0; i < 8; ++i) dw[c][i] = 0.0f;
  }
  int turn = 0;
  for (; row < a.rows; row += rows_a_turn) {
    auto next = load(row + rows_a_turn);
    __builtin_amdgcn_sched_barrier(0);  // (the loads go out here)
    const float r = v.r;
    double sum = 0.0;
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      const int c = kApart && WAVE ? (3 - k) % 3 : k;  // (0, 2, 1: two sums at a time)
      const double before = sum;
      if (kApart) sum = 0.0;
      Row<DF32, VEC>(a.dy, 0, a.n).settle(c * step + tid * 8, v.dy[c]);
      Row<HF32, VEC>(a.h, 0, a.n).settle(c * step + tid * 8, v.h[c]);
      Row<OF32, VEC>(a.dres, 0, a.n).settle(c * step + tid * 8, v.res[c]);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float d = v.dy[c].at(i), h = v.h[c].at(i);
        dw[c][i] = __builtin_fmaf(d, h * r, dw[c][i]);
        sum = __builtin_fma((double)(d * w[c][i]), (double)h, sum);
      }
      if (kApart) sum = before + sum;
      // (the sum is formed here, not where it is used with every widened value alive until then)
      asm volatile("" : "+v"(sum));
      forget(v.dy[c]);
      forget(v.h[c]);
    }
    if (a.dx || a.codes) {
      if (kApart && !WAVE && lanes == 128) {
        part[turn][tid] = sum;
        __syncthreads();
        sum = wave_sum(sum + part[turn][tid ^ 64]);
        turn ^= 1;
      } else {
        sum = wave_sum(sum);
        if constexpr (!WAVE) {
          // two sets of partial sums in turn: a wave two rows ahead has passed the barrier in between
          if ((tid & 63) == 0) part[turn][tid >> 6] = sum;
          __syncthreads();
          sum = part[turn][0];
          for (int i = 1; i < lanes >> 6; ++i) sum += part[turn][i];
          turn ^= 1;
        }
      }
      const float mean = (float)(sum * (double)r * a.inv_n);
      const Row<OF32, VEC> dx(a.dx, row * a.lddx, a.n, a.dx != nullptr);
      uint4 d[CH];
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        float g[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          g[i] = (v.dy[c].at(i) * w[c][i] - (v.h[c].at(i) * r) * mean) * r;
          if (a.dres) g[i] += v.res[c].at(i);
        }
        const auto o = as_raw<OF32>(g);
        if (VEC || a.dx) dx.store(c * step + tid * 8, o);
        if constexpr (OF32) {
          d[c] = pack_bf16x8(g);
        } else {
          d[c] = make_uint4(o.w[0], o.w[1], o.w[2], o.w[3]);
        }
      }
      if (a.codes) quantize_chunks<VEC, CH>(d, a.pow2, row, tid * 8, step, a.n, a.codes, a.ldc, a.scales);
    }
    v = next;
  }
  if (!a.dweight) return;
  if constexpr (WAVE) {
    if (slots > 1) {
      // the slots' shares side by side, four columns a place, then summed in their order
#pragma unroll
      for (int c = 0; c < CH; ++c)
#pragma unroll
        for (int i = 0; i < 8; i += 4) share[slot * CH * 128 + (2 * c + i / 4) * 64 + tid] = make_float4(dw[c][i], dw[c][i + 1], dw[c][i + 2], dw[c][i + 3]);
      __syncthreads();
      for (int k = threadIdx.x; k < CH * 128; k += blockDim.x) {
        const int col = (k >> 7) * 512 + (k & 63) * 8;
        float4 v = share[k];
        for (int s = 1; s < slots; ++s) {
          const float4 u = share[s * CH * 128 + k];
          v.x += u.x;
          v.y += u.y;
          v.z += u.z;
          v.w += u.w;
        }
        if (col < a.n) *reinterpret_cast<float4*>(a.partial + (int64_t)blockIdx.x * a.ldp + col + (k >> 6 & 1) * 4) = v;
      }
      return;
    }
  }
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int col = c * step + tid * 8;
    float* p = a.partial + (int64_t)blockIdx.x * a.ldp + col;
    if (col < a.n) {
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
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const float r = a.rstd[row];
    auto load = [&](int col, float* g, float* h) {
      float w[8];
      widen(Row<DF32, false>(a.dy, row * a.lddy, a.n).settled(col), g);
      widen(Row<HF32, false>(a.h, row * a.ldh, a.n).settled(col), h);
      widen_gain8<false>(ld_gain8<false>(a.weight, a.wf32, col, a.n), a.wf32, col, a.n, w);
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
        if (a.dres) widen(Row<OF32, false>(a.dres, row * a.lddr, a.n).settled(col), s);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        g[i] = (g[i] - (h[i] * r) * mean) * r;
        if (a.dres) g[i] += s[i];
      }
      if (a.dx) Row<OF32, false>(a.dx, row * a.lddx, a.n).store(col, as_raw<OF32>(g));
      const uint4 d[1] = {pack_bf16x8(g)};
      if (a.codes) quantize_chunks<false, 1>(d, a.pow2, row, col, 0, a.n, a.codes, a.ldc, a.scales);
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
// thread, then those in their order.  (256 shares of 7168 columns 3.6 us: the
// launch and two loads that wait for one another.)
__global__ __launch_bounds__(1024) void norm_dw_sum_kernel(const float* partial, int blocks, int n, int64_t ldp, float* dw) {
  __shared__ __attribute__((aligned(16))) float part[64][64];
  const int tid = threadIdx.x, group = tid >> 4, c4 = (tid & 15) * 4, c = tid & 63, q = tid >> 6;
  for (int64_t col0 = (int64_t)blockIdx.x * 64; col0 < n; col0 += (int64_t)gridDim.x * 64) {
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    if (col0 + c4 < n) {
#pragma unroll 4
      for (int b = group; b < blocks; b += 64) {
        const float4 v = *reinterpret_cast<const float4*>(partial + b * ldp + col0 + c4);
        s.x += v.x;
        s.y += v.y;
        s.z += v.z;
        s.w += v.w;
      }
    }
    *reinterpret_cast<float4*>(&part[group][c4]) = s;
    __syncthreads();
    // 16 waves, four of the sums each
    float v = (part[4 * q][c] + part[4 * q + 1][c]) + (part[4 * q + 2][c] + part[4 * q + 3][c]);
    __syncthreads();
    part[q][c] = v;
    __syncthreads();
    if (tid < 64 && col0 + tid < n) {
      v = part[0][tid];
#pragma unroll
      for (int i = 1; i < 16; ++i) v += part[i][tid];
      dw[col0 + tid] = v;
    }
    if (col0 + (int64_t)gridDim.x * 64 < n) __syncthreads();  // (part is written again)
  }
}

}  // namespace

template <bool DF32, bool HF32, bool OF32, bool VEC, bool KEEP>
static void launch_norm_bwd_rows(const NormBwdArgs& a, const NormBwdShape& s, hipStream_t stream) {
  // (of a workgroup, a row and the next one of float32 values take the registers at two chunks)
  constexpr int kMost = DF32 || HF32 || OF32 ? 2 : 4;
  auto kernel = !s.wave         ? norm_bwd_rows_kernel<DF32, HF32, OF32, VEC, KEEP, kMost, false>
                : s.chunks == 1 ? norm_bwd_rows_kernel<DF32, HF32, OF32, VEC, KEEP, 1, true>
                : s.chunks == 2 ? norm_bwd_rows_kernel<DF32, HF32, OF32, VEC, KEEP, 2, true>
                : s.chunks == 3 ? norm_bwd_rows_kernel<DF32, HF32, OF32, VEC, KEEP, 3, true>
                                : norm_bwd_rows_kernel<DF32, HF32, OF32, VEC, KEEP, kMost, true>;
  hipLaunchKernelGGL(kernel, dim3(s.blocks), dim3(s.threads), 0, stream, a);
}

template <bool DF32, bool HF32, bool OF32>
static void launch_norm_bwd_typed(const NormBwdArgs& a, hipStream_t stream) {
  const NormBwdShape s = norm_bwd_shape(a.rows, a.n, DF32 || HF32 || OF32);
  if (s.chunks == 0) {
    if (a.dx || a.codes)
      hipLaunchKernelGGL((norm_bwd_long_kernel<DF32, HF32, OF32>), dim3(a.rows < kMaxNormGrid ? a.rows : kMaxNormGrid), dim3(kMaxNormThreads), 0, stream, a);
    if (a.dweight) {
      const int per = norm_dw_rows(a.rows, s.blocks);
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
    const int blocks = a.rows > 0 ? norm_bwd_shape(a.rows, a.n, a.df32 || a.hf32 || a.of32).blocks : 0;
    const int groups = (a.n + 63) / 64;
    hipLaunchKernelGGL(norm_dw_sum_kernel, dim3(groups < kMaxNormGrid ? groups : kMaxNormGrid), dim3(1024), 0, stream, a.partial, blocks, a.n, a.ldp, a.dweight);
  }
  return hipGetLastError();
}

}  // namespace fp8q
