// The router's choice of experts and its gradient, gfx950.
//
// Scores of a token's logits x: s_e = 1 / (1 + exp(-x_e)) or
// exp(x_e) / sum exp(x).  The choice goes by s_e + b_e (without a bias by x_e,
// which the scores rise with): the best groups first, by their best or their
// two best experts, then the topk best experts in them, ties to the lower
// index.  Scores are held in 64 bits: two experts whose scores differ by less
// than a float32 step are no rarity among 256 of them over a batch, and which
// of them is taken should not depend on how the sum or the exponential was
// rounded.
//
// An expert whose logit or bias is -inf or NaN is never chosen; where fewer
// than topk are left, the rest of the row is -1 with weight 0 (a row of the
// table without an expert, which the sort drops and the weighted sum skips).
#include "fp8q_internal.h"
#include "quant_common.h"

namespace fp8q {
namespace {

constexpr int kGateWaves = 4;
constexpr int kGateLane = 16;  // experts a lane may hold
constexpr double kNone = -__builtin_inf();

__device__ __forceinline__ float ld_logit(const void* p, bool f32, int64_t i) {
  return f32 ? static_cast<const float*>(p)[i] : __uint_as_float((uint32_t)static_cast<const uint16_t*>(p)[i] << 16);
}

// A logit as it is used: NaN is none (-inf), +inf the largest number.
__device__ __forceinline__ double as_logit(float x) { return x == x ? (double)fminf(x, 3.402823466e38f) : kNone; }

__device__ __forceinline__ double gate_sum(double v) {
#pragma unroll
  for (int d = 32; d; d >>= 1) v += __shfl_xor(v, d);
  return v;
}
__device__ __forceinline__ double gate_max(double v) {
#pragma unroll
  for (int d = 32; d; d >>= 1) v = fmax(v, __shfl_xor(v, d));
  return v;
}

// Score of a logit; softmax: top the row's largest, inv 1 / sum exp(x - top).
__device__ __forceinline__ double score_of(double x, bool sigmoid, double top, double inv) {
  if (sigmoid) return 1.0 / (1.0 + exp(-x));
  return x > kNone ? exp(x - top) * inv : 0.0;
}

// One wave per token.  The lanes are shared out evenly over the groups (64 /
// the power of two above them each), a lane holds consecutive experts of its
// group, so a lower lane's experts come before a higher one's.
template <int P>
__global__ __launch_bounds__(64 * kGateWaves) void gate_kernel(GateArgs a) {
  const int lane = threadIdx.x & 63;
  const int per_group = a.experts / a.groups;
  const int lpg = 64 / a.group_lanes;  // (group_lanes: the power of two)
  const int per = (per_group + lpg - 1) / lpg;
  const int group = lane / lpg, first = (lane % lpg) * per;
  const int base = group * per_group + first;
  const int mine = group < a.groups ? min(max(per_group - first, 0), per) : 0;  // experts of this lane
  for (int t = (int)blockIdx.x * kGateWaves + (int)(threadIdx.x >> 6); t < a.tokens; t += (int)gridDim.x * kGateWaves) {
    const int64_t row = (int64_t)t * a.ld;
    double x[P], key[P];
#pragma unroll
    for (int p = 0; p < P; ++p) x[p] = p < mine ? as_logit(ld_logit(a.logits, a.lf32, row + base + p)) : kNone;
    double top = kNone, inv = 0.0;
    if (!a.sigmoid) {
#pragma unroll
      for (int p = 0; p < P; ++p) top = fmax(top, x[p]);
      top = gate_max(top);
      double total = 0.0;
#pragma unroll
      for (int p = 0; p < P; ++p)
        if (x[p] > kNone) total += exp(x[p] - top);
      total = gate_sum(total);
      inv = total > 0.0 ? 1.0 / total : 0.0;
    }
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const double s = score_of(x[p], a.sigmoid, top, inv);
      if (a.scores && p < mine) a.scores[(int64_t)t * a.experts + base + p] = (float)s;
      key[p] = x[p];
      if (p < mine && a.bias && x[p] > kNone) {
        const double k = s + (double)a.bias[base + p];
        key[p] = k > kNone ? k : kNone;
      }
    }
    if (a.groups > 1) {
      // the group's best and second best; two best: of their scores
      double b1 = kNone, b2 = kNone;
#pragma unroll
      for (int p = 0; p < P; ++p) {
        double k = key[p];
        if (a.two_best && !a.bias && k > kNone) k = score_of(x[p], a.sigmoid, top, inv);
        b2 = fmax(b2, fmin(b1, k));
        b1 = fmax(b1, k);
      }
      for (int d = 1; d < lpg; d <<= 1) {
        const double o1 = __shfl_xor(b1, d), o2 = __shfl_xor(b2, d);
        b2 = fmax(fmax(b2, o2), fmin(b1, o1));
        b1 = fmax(b1, o1);
      }
      if (a.two_best && b2 > kNone) b1 += b2;
      int before = 0;
      for (int g = 0; g < a.groups; ++g) {
        const double o = __shfl(b1, g * lpg);
        before += o > b1 || (o == b1 && g < group);
      }
      if (before >= a.top_groups) {
#pragma unroll
        for (int p = 0; p < P; ++p) key[p] = kNone;
      }
    }
    // topk rounds; lane j keeps the j-th expert
    int chosen = -1;
    for (int j = 0; j < a.topk; ++j) {
      double best = kNone;
#pragma unroll
      for (int p = 0; p < P; ++p) best = fmax(best, key[p]);
      const double all = gate_max(best);
      const uint64_t have = __builtin_amdgcn_ballot_w64(best == all && all > kNone);
      if (have == 0) break;
      const int owner = __builtin_ctzll(have);
      int e = -1;
#pragma unroll
      for (int p = P - 1; p >= 0; --p)
        if (key[p] == all) e = p;
      if (lane == owner) {
#pragma unroll
        for (int p = 0; p < P; ++p)
          if (p == e) key[p] = kNone;
      }
      e = __shfl(base + e, owner);
      if (lane == j) chosen = e;
    }
    double w = 0.0;
    if (chosen >= 0) w = score_of(as_logit(ld_logit(a.logits, a.lf32, row + chosen)), a.sigmoid, top, inv);
    if (a.renormalize) {
      const double total = gate_sum(w);
      w = total > 0.0 ? w / total : 0.0;
    }
    if (lane < a.topk) {
      const int64_t at = (int64_t)t * a.topk + lane;
      if (a.i64) {
        static_cast<int64_t*>(a.chosen)[at] = chosen;
      } else {
        static_cast<int32_t*>(a.chosen)[at] = chosen;
      }
      a.weights[at] = (float)(a.scale * w);
      if (a.load && chosen >= 0) atomicAdd(a.load + chosen, 1);
    }
  }
}

// Gradient, one wave per token: with ds_e = d loss / d s_e,
//   renormalised  ds_e = scale (dw_e - sum_k dw_k s_k / S) / S, S = sum of the chosen scores,
//   else          ds_e = scale dw_e,
// plus dscores; dx = ds s (1 - s), or s (ds - sum over all experts of ds s).
__global__ __launch_bounds__(64 * kGateWaves) void gate_bwd_kernel(GateBwdArgs a) {
  const int lane = threadIdx.x & 63;
  for (int t = (int)blockIdx.x * kGateWaves + (int)(threadIdx.x >> 6); t < a.tokens; t += (int)gridDim.x * kGateWaves) {
    const int64_t row = (int64_t)t * a.ld;
    auto logit = [&](int e) { return as_logit(ld_logit(a.logits, a.lf32, row + e)); };
    double top = kNone, inv = 0.0;
    if (!a.sigmoid) {
      for (int e = lane; e < a.experts; e += 64) top = fmax(top, logit(e));
      top = gate_max(top);
      double total = 0.0;
      for (int e = lane; e < a.experts; e += 64) {
        const double x = logit(e);
        if (x > kNone) total += exp(x - top);
      }
      total = gate_sum(total);
      inv = total > 0.0 ? 1.0 / total : 0.0;
    }
    // lane j: the j-th choice
    int e = -1;
    double ds = 0.0;
    if (lane < a.topk) {
      const int64_t at = (int64_t)t * a.topk + lane;
      const int64_t c = a.i64 ? static_cast<const int64_t*>(a.chosen)[at] : static_cast<const int32_t*>(a.chosen)[at];
      if (c >= 0 && c < a.experts) {
        e = (int)c;
        ds = (double)a.dweights[at];
      }
    }
    if (a.renormalize) {
      const double s = e >= 0 ? score_of(logit(e), a.sigmoid, top, inv) : 0.0;
      const double total = gate_sum(s), dot = gate_sum(e >= 0 ? ds * s : 0.0);
      ds = total > 0.0 ? (ds - dot / total) / total : 0.0;
    }
    ds *= a.scale;
    auto grad = [&](int i) {
      double d = a.dscores ? (double)a.dscores[(int64_t)t * a.experts + i] : 0.0;
      for (int j = 0; j < a.topk; ++j) {
        const int ej = __shfl(e, j);
        const double dj = __shfl(ds, j);
        if (ej == i) d += dj;
      }
      return d;
    };
    double mean = 0.0;
    if (!a.sigmoid) {
      for (int e0 = 0; e0 < a.experts; e0 += 64) {
        const int i = min(e0 + lane, a.experts - 1);
        const double x = logit(i), d = grad(i) * score_of(x, false, top, inv);
        if (e0 + lane < a.experts && x > kNone) mean += d;
      }
      mean = gate_sum(mean);
    }
    for (int e0 = 0; e0 < a.experts; e0 += 64) {
      const int i = min(e0 + lane, a.experts - 1);
      const double x = logit(i), s = score_of(x, a.sigmoid, top, inv);
      double d = a.sigmoid ? grad(i) * s * (1.0 / (1.0 + exp(x))) : s * (grad(i) - mean);
      if (!(x > kNone)) d = 0.0;
      if (e0 + lane < a.experts) {
        const int64_t at = (int64_t)t * a.ldd + i;
        if (a.of32) {
          static_cast<float*>(a.dlogits)[at] = (float)d;
        } else {
          static_cast<uint16_t*>(a.dlogits)[at] = __builtin_bit_cast(uint16_t, (__bf16)(float)d);
        }
      }
    }
  }
}

int gate_grid(int tokens) {
  const int want = (tokens + kGateWaves - 1) / kGateWaves;
  return want < kMaxGateGrid ? want : kMaxGateGrid;
}

}  // namespace

hipError_t launch_gate(GateArgs a, hipStream_t stream) {
  a.group_lanes = 1;
  while (a.group_lanes < a.groups) a.group_lanes *= 2;
  const int lpg = 64 / a.group_lanes, per = (a.experts / a.groups + lpg - 1) / lpg;
  auto kernel = per <= 1 ? gate_kernel<1> : per <= 2 ? gate_kernel<2> : per <= 4 ? gate_kernel<4> : per <= 8 ? gate_kernel<8> : gate_kernel<kGateLane>;
  hipLaunchKernelGGL(kernel, dim3(gate_grid(a.tokens)), dim3(64 * kGateWaves), 0, stream, a);
  return hipGetLastError();
}

hipError_t launch_gate_backward(const GateBwdArgs& a, hipStream_t stream) {
  hipLaunchKernelGGL(gate_bwd_kernel, dim3(gate_grid(a.tokens)), dim3(64 * kGateWaves), 0, stream, a);
  return hipGetLastError();
}

}  // namespace fp8q
