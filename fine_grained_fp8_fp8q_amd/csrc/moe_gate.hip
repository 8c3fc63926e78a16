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
// The batch of 16384 tokens, eight of 256 experts in four of eight groups, takes
// 13.6 us (the bytes 2.8, the launch 2.6): 1210 vector instructions for the four
// tokens of a wave, all of whose 4096 start, load and choose at the same time.
// One token takes 4.5 us.
//
// An expert whose logit or bias is -inf or NaN is never chosen; where fewer
// than topk are left, the rest of the row is -1 with weight 0 (a row of the
// table without an expert, which the sort drops and the weighted sum skips).
#include "chunk8.h"
#include "fp8q_internal.h"

namespace fp8q {
namespace {

constexpr int kGateWaves = 4;
constexpr int kGateLane = 16;  // experts a lane may hold
constexpr int kGateLoadPairs = 8192;  // pairs that a workgroup counts
constexpr int kGateLoadApart = 4096;  // pairs from which they are counted by a kernel of their own
constexpr double kNone = -__builtin_inf();

__device__ __forceinline__ float ld_logit(const void* p, bool f32, int64_t i) {
  return f32 ? static_cast<const float*>(p)[i] : __uint_as_float((uint32_t)static_cast<const uint16_t*>(p)[i] << 16);
}

// A logit as it is used: NaN is none (-inf), +inf the largest number.
__device__ __forceinline__ double as_logit(float x) { return x == x ? (double)fminf(x, 3.402823466e38f) : kNone; }

// f over a token's L lanes (16: one DPP row, 32: two, or the whole wave), the
// same in each.  All 64 lanes must be active.
template <int L, class F>
__device__ __forceinline__ double gate_all(double v, F f) {
  v = f(v, dpp_double<0xB1>(v));
  v = f(v, dpp_double<0x4E>(v));
  v = f(v, dpp_double<0x141>(v));
  v = f(v, dpp_double<0x140>(v));
  if constexpr (L == 32) v = f(v, __shfl_xor(v, 16));
  if constexpr (L == 64) v = f(f(lane_double(v, 0), lane_double(v, 16)), f(lane_double(v, 32), lane_double(v, 48)));
  return v;
}
template <int L>
__device__ __forceinline__ double gate_sum(double v) {
  return gate_all<L>(v, [](double x, double y) { return x + y; });
}
template <int L>
__device__ __forceinline__ double gate_max(double v) {
  return gate_all<L>(v, [](double x, double y) { return fmax(x, y); });
}

// exp(x) in 64 bits: x = k ln 2 + r with |r| <= ln 2 / 2 (ln 2 in two parts, so
// that k times the first is exact), the exponential series up to r^13 / 13!
// (the next term is below 2^-57), times 2^k.  Within 2 ulps; 0 and infinity
// where the result leaves the range.
__device__ __forceinline__ double exp64(double x) {
  x = fmin(fmax(x, -1100.0), 1100.0);
  const double k = __builtin_rint(x * 0x1.71547652b82fep+0);
  double r = __builtin_fma(-k, 0x1.62e42fefap-1, x);
  r = __builtin_fma(-k, 0x1.cf79abc9e3b3ap-40, r);
  double p = 1.0 / 6227020800.0;
  p = __builtin_fma(p, r, 1.0 / 479001600.0);
  p = __builtin_fma(p, r, 1.0 / 39916800.0);
  p = __builtin_fma(p, r, 1.0 / 3628800.0);
  p = __builtin_fma(p, r, 1.0 / 362880.0);
  p = __builtin_fma(p, r, 1.0 / 40320.0);
  p = __builtin_fma(p, r, 1.0 / 5040.0);
  p = __builtin_fma(p, r, 1.0 / 720.0);
  p = __builtin_fma(p, r, 1.0 / 120.0);
  p = __builtin_fma(p, r, 1.0 / 24.0);
  p = __builtin_fma(p, r, 1.0 / 6.0);
  p = __builtin_fma(p, r, 0.5);
  p = __builtin_fma(p, r, 1.0);
  p = __builtin_fma(p, r, 1.0);
  return __builtin_ldexp(p, (int)k);
}

// Score of a logit; softmax: top the row's largest, inv 1 / sum exp(x - top).
// Below -700 a sigmoid is exp(x), 1 + exp(-x) leaves the range before its
// reciprocal does.
__device__ __forceinline__ double score_of(double x, bool sigmoid, double top, double inv) {
  if (sigmoid) {
    const bool far = x < -700.0;
    const double t = exp64(far ? x : -x);
    return far ? t : 1.0 / (1.0 + t);
  }
  return x > kNone ? exp64(x - top) * inv : 0.0;
}

// The same for a float32 result: the hardware's estimate of the reciprocal and
// two Newton steps, a third of the division's instructions (a score below
// e^-120 is 0 in float32 either way).
__device__ __forceinline__ float score32(double x, bool sigmoid, double top, double inv) {
  if (!sigmoid) return x > kNone ? (float)(exp64(x - top) * inv) : 0.0f;
  const double d = 1.0 + exp64(fmin(-x, 120.0));
  double y = __builtin_amdgcn_rcp(d);
  y = __builtin_fma(__builtin_fma(-d, y, 1.0), y, y);
  y = __builtin_fma(__builtin_fma(-d, y, 1.0), y, y);
  return (float)y;
}

// The lanes of a token, L of them, are shared out evenly over the groups (L /
// the power of two above them each); a lane holds up to P experts of its group,
// by fours.  Its fours are consecutive, so that a lower lane's experts come
// before a higher one's, or (SPREAD) one of every round over the group's lanes:
// loads of whole lines, and no lane with a list too short for neighbours that
// are all among the best (16384 x 256 with the eight best side by side: 48 us
// with consecutive fours, 13.9 so; 13.2 and 13.6 without such neighbours).
template <int L, int P, bool SPREAD>
struct GateLane {
  int lane, lpg, group, base, step, mine;  // lpg: lanes of a group; base: the lane's first expert; step: from four to four
  bool fours;                              // groups of whole fours
  // The lane has the expert base + at(p) if at(p) < mine.
  __device__ __forceinline__ int at(int p) const { return (p >> 2) * step + (p & 3); }
  __device__ __forceinline__ explicit GateLane(const GateArgs& a) {
    const GateSplit& s = L == 64 ? a.wide : L == 32 ? a.middle : a.narrow;
    lane = threadIdx.x & (L - 1);
    lpg = 1 << s.lane_bits;
    const int first = (lane & (lpg - 1)) * (SPREAD ? 4 : s.per);
    step = SPREAD ? 4 * lpg : 4;
    group = lane >> s.lane_bits;
    base = group * a.per_group + first;
    mine = group < a.groups ? SPREAD ? a.per_group - first : min(max(a.per_group - first, 0), s.per) : 0;
    fours = a.per_group % 4 == 0;
  }
  // The lane's values of a row; those it does not have are the row's last.
  __device__ __forceinline__ void load(const void* p, bool f32, int64_t row, int experts, float (&f)[P]) const {
    int base = this->base;
    asm volatile("" : "+v"(base));  // (or an offset for every value is kept from turn to turn)
    if (!fours) {
#pragma unroll
      for (int c = 0; c < P; ++c) f[c] = ld_logit(p, f32, row + min(base + at(c), experts - 1));
    } else if (f32) {
#pragma unroll
      for (int c = 0; c < P; c += 4) {
        const auto r = ld_raw<true, 4, true>(p, row + min(base + at(c), experts - 4), 4, false);
#pragma unroll
        for (int i = 0; i < 4; ++i) f[c + i] = r.at(i);
      }
    } else {
#pragma unroll
      for (int c = 0; c < P; c += 4) {
        const auto r = ld_raw<false, 4, true>(p, row + min(base + at(c), experts - 4), 4, false);
#pragma unroll
        for (int i = 0; i < 4; ++i) f[c + i] = r.at(i);
      }
    }
  }
};

// The largest of N values, as a tree.
template <int N, class T, class F>
__device__ __forceinline__ T gate_tree(const T* v, F f) {
  if constexpr (N == 1) {
    return v[0];
  } else {
    return f(gate_tree<N / 2>(v, f), gate_tree<N - N / 2>(v + N / 2, f));
  }
}
template <int N>
__device__ __forceinline__ double gate_tree_max(const double* v) {
  return gate_tree<N>(v, [](double x, double y) { return fmax(x, y); });
}

// What the lanes of a wave have written to LDS is there for one another.
__device__ __forceinline__ void gate_wave_fence() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// A token's scores may all be so small that 64 bits hold them in few bits, or
// not at all: relative to the largest one they still have their shares of the
// sum.  (So far below zero a sigmoid is exp(x), as a softmax's numerator is.)
constexpr double kFarScores = 0x1p-900;
__device__ __forceinline__ bool far_scores(double total, bool sigmoid) { return total < kFarScores && (!sigmoid || total > 0.0); }

// What lane j of a token's lanes does with its j-th expert (-1: none).
template <int L>
__device__ __forceinline__ void gate_write(const GateArgs& a, int64_t t, bool real, int lane, int chosen, double w) {
  if (a.renormalize) {
    double total = gate_sum<L>(w);
    if (__builtin_amdgcn_ballot_w64(chosen >= 0 && far_scores(total, a.sigmoid))) {
      const double x = chosen >= 0 ? as_logit(ld_logit(a.logits, a.lf32, t * a.ld + chosen)) : kNone;
      const double top = gate_max<L>(x);
      const double e = chosen >= 0 ? exp64(x - top) : 0.0;
      const double sum = gate_sum<L>(e);
      if (far_scores(total, a.sigmoid)) {
        w = e;
        total = sum;
      }
    }
    w = total > 0.0 ? w / total : 0.0;
  }
  if (real && lane < a.topk) {
    const int64_t at = t * a.topk + lane;
    if (a.i64) {
      static_cast<int64_t*>(a.chosen)[at] = chosen;
    } else {
      static_cast<int32_t*>(a.chosen)[at] = chosen;
    }
    a.weights[at] = (float)(a.scale * w);
    if (a.load && chosen >= 0) atomicAdd(a.load + chosen, 1);
  }
}

// One token by a whole wave, every step in 64 bits.
template <int P>
__device__ __forceinline__ void gate_exact(const GateArgs& a, int64_t t) {
  const GateLane<64, P, false> at(a);
  const int64_t row = t * a.ld;
  float f[P];
  at.load(a.logits, a.lf32, row, a.experts, f);
  double x[P], key[P];
#pragma unroll
  for (int p = 0; p < P; ++p) x[p] = p < at.mine ? as_logit(f[p]) : kNone;
  double top = kNone, inv = 0.0;
  if (!a.sigmoid) {
    top = gate_max<64>(gate_tree_max<P>(x));
    double total = 0.0;
#pragma unroll
    for (int p = 0; p < P; ++p)
      if (x[p] > kNone) total += exp64(x[p] - top);
    total = gate_sum<64>(total);
    inv = total > 0.0 ? 1.0 / total : 0.0;
  }
  // scores where something asks for them; the choice is by x without a bias
  if (a.bias || a.scores || a.groups > 1) {
#pragma unroll
    for (int p = 0; p < P; ++p) key[p] = score_of(x[p], a.sigmoid, top, inv);
    if (a.scores) {
#pragma unroll
      for (int p = 0; p < P; ++p)
        if (p < at.mine) a.scores[t * a.experts + at.base + p] = (float)key[p];
    }
    if (a.bias) {
      at.load(a.bias, true, 0, a.experts, f);
#pragma unroll
      for (int p = 0; p < P; ++p) key[p] = key[p] + (double)f[p];
    }
  }
  if (a.groups > 1) {
    // the group's best and second best
    const bool by_key = a.bias || a.two_best;
    double b1 = kNone, b2 = kNone;
#pragma unroll
    for (int p = 0; p < P; ++p) {
      double k = by_key ? key[p] : x[p];
      k = x[p] > kNone && k > kNone ? k : kNone;
      b2 = fmax(b2, fmin(b1, k));
      b1 = fmax(b1, k);
    }
    for (int d = 1; d < at.lpg; d <<= 1) {
      const double o1 = __shfl_xor(b1, d), o2 = __shfl_xor(b2, d);
      b2 = fmax(fmax(b2, o2), fmin(b1, o1));
      b1 = fmax(b1, o1);
    }
    if (a.two_best && b2 > kNone) b1 += b2;
    int before = 0;
    for (int g = 0; g < a.groups; ++g) {
      const double o = __shfl(b1, g * at.lpg);
      before += o > b1 || (o == b1 && g < at.group);
    }
    if (before >= a.top_groups) {
#pragma unroll
      for (int p = 0; p < P; ++p) x[p] = kNone;
    }
  }
#pragma unroll
  for (int p = 0; p < P; ++p) {
    const double k = a.bias ? key[p] : x[p];
    key[p] = x[p] > kNone && k > kNone ? k : kNone;  // (a bias of NaN too)
  }
  // topk rounds; lane j keeps the j-th expert
  int chosen = -1;
  for (int j = 0; j < a.topk; ++j) {
    const double best = gate_tree_max<P>(key), all = gate_max<64>(best);
    // the lowest lane that holds it
    const uint64_t have = __builtin_amdgcn_ballot_w64(best == all && all > kNone);
    if (have == 0) break;
    const int owner = __builtin_ctzll(have);
    int e = 0;
#pragma unroll
    for (int p = P - 1; p >= 0; --p)
      if (key[p] == all) e = p;
    if (at.lane == owner) {
#pragma unroll
      for (int p = 0; p < P; ++p)
        if (p == e) key[p] = kNone;
    }
    e = __builtin_amdgcn_readlane(at.base + e, owner);
    if (at.lane == j) chosen = e;
  }
  double w = 0.0;
  if (chosen >= 0) w = score_of(as_logit(ld_logit(a.logits, a.lf32, row + chosen)), a.sigmoid, top, inv);
  gate_write<64>(a, t, true, at.lane, chosen, w);
}
template <int P>
__global__ __launch_bounds__(64 * kGateWaves) void gate_exact_kernel(GateArgs a) {
  const int64_t stride = (int64_t)gridDim.x * kGateWaves;
  for (int64_t t = (int64_t)blockIdx.x * kGateWaves + (int)(threadIdx.x >> 6); t < a.tokens; t += stride) gate_exact<P>(a, t);
}

// The middle one of three (one instruction).
__device__ __forceinline__ uint32_t med3(uint32_t a, uint32_t b, uint32_t c) { return max(min(a, b), min(max(a, b), c)); }
template <int L>
__device__ __forceinline__ uint32_t gate_max_u32(uint32_t v) {
  v = dpp_max16(v);
  if constexpr (L == 32) v = max(v, (uint32_t)__shfl_xor((int)v, 16));
  if constexpr (L == 64) {
    v = max(max((uint32_t)__builtin_amdgcn_readlane((int)v, 0), (uint32_t)__builtin_amdgcn_readlane((int)v, 16)),
            max((uint32_t)__builtin_amdgcn_readlane((int)v, 32), (uint32_t)__builtin_amdgcn_readlane((int)v, 48)));
  }
  return v;
}
template <int L>
__device__ __forceinline__ uint32_t gate_min_u32(uint32_t v) {
  return ~gate_max_u32<L>(~v);
}
// Order of float32 values as unsigned ones, NaN aside.
__device__ __forceinline__ uint32_t ordered(float f) {
  const uint32_t u = __float_as_uint(f);
  return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t u) { return __uint_as_float(u ^ ((u >> 31) ? 0x80000000u : 0xFFFFFFFFu)); }

// The choice by float32 scores where these are enough to know the 64-bit
// order, which is nearly always: a third of the instructions, and short ones.
// L lanes a token, 64 / L tokens a wave.
//
// Every open expert gets a 32-bit key, the lowest the best: d = the row's
// highest float32 score less its own, whose bits order like the number, with
// the index in the place of its last nine bits, so that keys differ and equal
// scores go by index.  Close to the highest, where it matters, d is finest.  A
// lane keeps its T best keys in order (a minimum and T - 1 medians of three per
// expert); rounds take the best head of all lanes.  The float32 score is within
// err of the 64-bit one:
//   sigmoid, u = 2^-24: 0.4 u of the exponent's rounding (1.5 u |x|, times s
//     (1 - s), with |x| s (1 - s) < 0.23), 0.5 u of exp2 (an ulp, times s (1 -
//     s)), u of the sum, 2 u of the reciprocal (an ulp): below 6 u;
//   softmax: its numerator 1 u (2.5 u |d|, d = x - top, with |d| e^-|d| < 0.37)
//     and 2 u; the denominator 2.5 u times the mean |d|, at most ln 512, 2 u of
//     exp2, 15 u of a lane's sum, u of its rounding, 2 u of the reciprocal, and
//     u of the product, each times s <= 1: below 48 u;
//   the sum with the bias u of it, and d u of that: 2 u of the largest.
// so two experts whose d differ by more than 2 err and the nine bits are in
// order.  Without a bias d comes from the logits themselves and never reverses
// them: any two different keys are in order if the logits differ at all.  Nor
// do BF16 logits x with |x| >= d / 32 share a d unless they are equal: others
// lie 2^-8 |x| away or more, and the d of a key steps by 2^-14 d.
// Two more experts than asked for are taken.  Where neighbours among them are
// not clear of one another, they change places by their 64-bit scores; if the
// last one chosen is not clear of the last one taken, somebody left out might
// belong in, and the wave does the token in 64 bits.  So it does if groups are
// not clear of one another or a lane's list ran out.
enum { kByLogit = 0, kBySigmoid = 1, kBySoftmax = 2 };  // what is chosen by: x, or the score with a bias
struct Four {
  double a, b, c, d;
};
template <int L, int P, int BY>
__global__ __launch_bounds__(64 * kGateWaves) void gate_kernel(GateArgs a) {
  constexpr int kTokens = 64 / L;         // of a wave
  constexpr int T = P < 8 ? P : 8;        // experts in a lane's list
  constexpr int kExactP = P * L > 256 ? P * L / 64 : 4;  // fewer where all 64 lanes share a token
  constexpr float U = 0x1p-24f, kLow = -__builtin_inff(), kLog2e = 1.44269504f;
  constexpr uint32_t kNoKey = 0xFFFFFFFFu;
  const GateLane<L, P, true> at(a);
  const int lane = at.lane, sub = (threadIdx.x & 63) / L, taken = a.topk + 2;
  const int64_t stride = (int64_t)gridDim.x * kGateWaves * kTokens;
  // (whole waves go round together; a token past the last is worked on as the last)
  for (int64_t t0 = ((int64_t)blockIdx.x * kGateWaves + (int)(threadIdx.x >> 6)) * kTokens; t0 < a.tokens; t0 += stride) {
    const bool real = t0 + sub < a.tokens;
    const int64_t t = real ? t0 + sub : a.tokens - 1;
    const int64_t row = t * a.ld;
    float x[P], key[P], bias[P];
    at.load(a.logits, a.lf32, row, a.experts, x);
    if constexpr (BY != kByLogit) at.load(a.bias, true, 0, a.experts, bias);
    int mine = at.mine;
    asm volatile("" : "+v"(mine));  // (or a mask for every p is kept from turn to turn)
#pragma unroll
    for (int p = 0; p < P; ++p) x[p] = ((at.at(p) < mine) & (x[p] == x[p])) ? fminf(x[p], 3.402823466e38f) : kLow;
    float top = kLow, err = 0.0f;
    if (BY == kBySoftmax || !a.sigmoid) {
      top = gate_tree<P>(x, [](float u, float v) { return fmaxf(u, v); });
      top = unordered(gate_max_u32<L>(ordered(top)));
    }
    if constexpr (BY == kByLogit) {
#pragma unroll
      for (int p = 0; p < P; ++p) key[p] = x[p];
    } else if constexpr (BY == kBySigmoid) {
      err = 6.0f * U;
#pragma unroll
      for (int p = 0; p < P; ++p) {
        const float k = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-x[p] * kLog2e)) + bias[p];
        key[p] = ((x[p] > kLow) & (bias[p] > kLow)) ? k : kLow;
      }
    } else {
      err = 48.0f * U;
      float total = 0.0f;
#pragma unroll
      for (int p = 0; p < P; ++p) {
        const float e = __builtin_amdgcn_exp2f((x[p] - top) * kLog2e);  // (a NaN in a row of -inf)
        key[p] = x[p] > kLow ? e : 0.0f;
        total += key[p];
      }
      total = (float)gate_sum<L>((double)total);
      const float inv = total > 0.0f ? __builtin_amdgcn_rcpf(total) : 0.0f;
#pragma unroll
      for (int p = 0; p < P; ++p) {
        const float k = key[p] * inv + bias[p];
        key[p] = ((x[p] > kLow) & (bias[p] > kLow)) ? k : kLow;
      }
    }
    bool unsure = false;
    if (a.groups > 1) {
      // the group's best and second best
      float b1 = kLow, b2 = kLow;
#pragma unroll
      for (int p = 0; p < P; ++p) {
        b2 = fmaxf(b2, fminf(b1, key[p]));
        b1 = fmaxf(b1, key[p]);
      }
      for (int d = 1; d < at.lpg; d <<= 1) {
        const float o1 = __shfl_xor(b1, d), o2 = __shfl_xor(b2, d);
        b2 = fmaxf(fmaxf(b2, o2), fminf(b1, o1));
        b1 = fmaxf(b1, o1);
      }
      const float rank = a.two_best && b2 > kLow ? b1 + b2 : b1;
      int before = 0;
      for (int g = 0; g < a.groups; ++g) {
        const float o = __shfl(rank, g * at.lpg, L);
        before += o > rank || (o == rank && g < at.group);
      }
      const bool open = before < a.top_groups;
      if constexpr (BY != kByLogit) {
        // every closed group has to be clear of every open one (two scores are
        // added to two biases, and the sums)
        const float off = 2.0f * err + 4.0f * U * ((b1 > kLow ? fabsf(b1) : 0.0f) + (b2 > kLow ? fabsf(b2) : 0.0f));
        const bool real_group = at.group < a.groups;
        const float in = -unordered(gate_max_u32<L>(ordered(open && real_group ? off - rank : kLow)));
        const float out = unordered(gate_max_u32<L>(ordered(!open && real_group ? rank + off : kLow)));
        unsure = !(off < 1e38f) || (out > kLow && !(in > out));
      }
      if (!open) {
#pragma unroll
        for (int p = 0; p < P; ++p) key[p] = kLow;
      }
    }
    float high = gate_tree<P>(key, [](float u, float v) { return fmaxf(u, v); });
    high = unordered(gate_max_u32<L>(ordered(high)));
    if constexpr (BY != kByLogit) unsure = unsure || high > 1e38f;  // (a bias beyond scores)
    uint32_t m[T];
#pragma unroll
    for (int i = 0; i < T; ++i) m[i] = kNoKey;
    int first = at.base;
    asm volatile("" : "+v"(first));
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const uint32_t d = (__float_as_uint(high - key[p]) & ~511u) | (uint32_t)(first + at.at(p));
      const uint32_t k = key[p] > kLow ? d : kNoKey;
#pragma unroll
      for (int i = T - 1; i > 0; --i)
        if (i <= p) m[i] = i < p ? med3(m[i - 1], m[i], k) : max(m[i - 1], k);
      m[0] = min(m[0], k);
    }
    uint32_t cand = kNoKey;  // lane j: the j-th best key
    int popped = 0;
    for (int j = 0; j < taken; ++j) {
      const uint32_t all = gate_min_u32<L>(m[0]);
      const uint32_t won = ((m[0] == all) & (all != kNoKey)) ? ~0u : 0u;
      cand = lane == j ? all : cand;
      // the winner's list moves up (by masks: of selects the compiler makes an indexed array)
#pragma unroll
      for (int i = 0; i + 1 < T; ++i) m[i] = (m[i + 1] & won) | (m[i] & ~won);
      m[T - 1] |= won;
      popped -= (int)won;
    }
    if (P > T) unsure = unsure || popped >= T;
    int chosen = cand != kNoKey ? (int)(cand & 511u) : -1;
    float logit = 0.0f;
    if (chosen >= 0) logit = ld_logit(a.logits, a.lf32, row + chosen);
    // whether an expert of key `far` is certainly behind one of key `near`
    const float most = 2.0f * err + 4.0f * U * fabsf(high);  // (and of what lies below, with its d)
    auto behind = [&](uint32_t near, uint32_t far) {
      const float dn = __uint_as_float(near & ~511u), df = __uint_as_float(far & ~511u);
      if constexpr (BY == kByLogit) return df > dn;
      return df - dn > most + df * 0x1p-12f;
    };
    // neighbours: lane j and j + 1
    const uint32_t next = (uint32_t)__shfl_down((int)cand, 1, L), last = (uint32_t)__shfl((int)cand, taken - 1, L);
    const float logit_next = __shfl_down(logit, 1, L), logit_last = __shfl(logit, taken - 1, L);
    bool close = lane < a.topk && next != kNoKey && !behind(cand, next);
    if (BY == kByLogit) close = close && logit != logit_next;  // (equal logits go by index)
    const uint64_t any_close = __builtin_amdgcn_ballot_w64(close);
    double s_top = kNone, s_inv = 0.0;
    // (four experts at a time, from the cache: all side by side their steps would
    // fill the registers of every call)
    auto four = [&](int from, auto f) {  // those from base + from
      double v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = f(as_logit(ld_logit(a.logits, a.lf32, row + first + min(from + i, mine - 1))));
      return Four{v[0], v[1], v[2], v[3]};
    };
    Four e{};  // the first four's exponentials
    if (!a.sigmoid) {
      // the 64-bit denominator where it is asked for
      s_top = as_logit(top);
      s_inv = 1.0;
      if (!a.renormalize || a.scores || (BY == kBySoftmax && any_close)) {
        double total = 0.0;
        for (int from = 0; from < mine; from += at.step) {
          e = four(from, [&](double v) { return exp64(v - s_top); });
          total += e.a + (from + 1 < mine ? e.b : 0.0) + ((from + 2 < mine ? e.c : 0.0) + (from + 3 < mine ? e.d : 0.0));
        }
        total = gate_sum<L>(total);
        s_inv = total > 0.0 ? 1.0 / total : 0.0;
      }
    }
    if (a.scores && real) {
      float* out = a.scores + t * a.experts + first;
      for (int from = 0; from < mine; from += at.step) {
        if (P > 4 || a.sigmoid) e = four(from, [&](double v) { return (double)score32(v, a.sigmoid, s_top, s_inv); });
        const bool unscaled = P <= 4 && !a.sigmoid;
        const float v[4] = {(float)(unscaled ? e.a * s_inv : e.a), (float)(unscaled ? e.b * s_inv : e.b), (float)(unscaled ? e.c * s_inv : e.c),
                            (float)(unscaled ? e.d * s_inv : e.d)};
        st_float4(out + from, v, mine - from, false);
      }
    }
    double s = chosen >= 0 ? score_of(as_logit(logit), a.sigmoid, s_top, s_inv) : 0.0;
    if (any_close) {
      // the taken ones in their 64-bit order: neighbours change places until none are wrong
      double k = chosen < 0 ? kNone : BY == kByLogit ? as_logit(logit) : s + (double)a.bias[chosen];
      const int me = threadIdx.x & 63;
      while (true) {
        const double kn = __shfl_down(k, 1, L);
        const int en = __shfl_down(chosen, 1, L);
        const uint64_t wrong = __builtin_amdgcn_ballot_w64(lane + 1 < taken && (kn > k || (kn == k && en >= 0 && en < chosen)));
        if (!wrong) break;
        const uint64_t even = wrong & 0x5555555555555555ull, pick = even ? even : wrong;  // (the first of each pair)
        const int from = lane + (int)(pick >> me & 1) - (int)(pick << 1 >> me & 1);
        k = __shfl(k, from, L);
        s = __shfl(s, from, L);
        chosen = __shfl(chosen, from, L);
        cand = (uint32_t)__shfl((int)cand, from, L);
      }
    }
    // the chosen ones have to be clear of whatever was left out, all of it behind the last one taken
    bool open_end = lane < a.topk && cand != kNoKey && last != kNoKey && !behind(cand, last);
    if (BY == kByLogit && !a.lf32) open_end = open_end && !(fabsf(logit_last) >= __uint_as_float(last & ~511u) * 0x1p-5f);
    unsure = unsure || open_end;
    const uint64_t redo = __builtin_amdgcn_ballot_w64(unsure);
    auto again = [&](int i) { return (redo >> (i * L & 63) & (~0ull >> (64 - L))) != 0; };  // token i of the wave
    gate_write<L>(a, t, real && !again(sub), lane, lane < a.topk ? chosen : -1, lane < a.topk ? s : 0.0);
    if (redo) {
      for (int i = 0; i < kTokens && t0 + i < a.tokens; ++i)
        if (again(i)) gate_exact<kExactP>(a, t0 + i);
    }
  }
}

// ------------------------------------------------------------- gradient ---
// With the chosen scores s_k, S their sum and w_k = s_k / S, the gradient that
// the weights bring to a chosen logit is
//   renormalised  scale w_k (dw_k - sum_j dw_j w_j), of a sigmoid times (1 - s_k),
//   else          scale dw_k s_k (1 - s_k), or scale s_k (dw_k - sum_j dw_j s_j);
// dscores add ds s (1 - s), or s (ds - sum over all experts of ds s).  A 1 / S
// that could leave the range, where w_k does not, is not formed (far_scores).
// (The renormalised softmax needs the chosen logits alone.)  Every step is in
// 64 bits: what is left of a difference may be little.

// What lane j of a token's lanes knows of its j-th choice: the expert (-1:
// none), the gradient of its weight (0 without one) and its logit.
struct GateChoice {
  int e;
  double dw, x;
};
template <int L>
__device__ __forceinline__ GateChoice gate_choice(const GateBwdArgs& a, int64_t t, int lane) {
  GateChoice c{-1, 0.0, kNone};
  if (lane < a.topk) {
    const int64_t at = t * a.topk + lane;
    const int64_t e = a.i64 ? static_cast<const int64_t*>(a.chosen)[at] : static_cast<const int32_t*>(a.chosen)[at];
    if (e >= 0 && e < a.experts) {
      c.e = (int)e;
      c.dw = (double)a.dweights[at];
      c.x = as_logit(ld_logit(a.logits, a.lf32, t * a.ld + e));
    }
  }
  return c;
}

// v summed over the token's choices of the same expert, in their order; a
// choice is nearly always alone with its expert.
template <int L>
__device__ __forceinline__ double gate_same(double v, int e, int topk) {
  bool twice = false;
  for (int j = 1; j < topk; ++j) {
    const int other = __shfl_down(e, j, L);
    twice = twice || (e >= 0 && other == e && (int)(threadIdx.x & (L - 1)) + j < L);
  }
  if (__builtin_amdgcn_ballot_w64(twice) == 0) return v;
  double sum = 0.0;
  for (int j = 0; j < topk; ++j) {
    const int ej = __shfl(e, j, L);
    const double vj = __shfl(v, j, L);
    sum += ej == e ? vj : 0.0;
  }
  return sum;
}

// A sigmoid, 1 - s, and its slope s (1 - s) = t / (1 + t)^2, t = e^-|x|.  1 + t
// is in [1, 2]: its reciprocal needs no scaling, and two Newton steps after the
// approximate one (half the cost of a division).
struct Sigmoid {
  double s, rest, slope;
};
__device__ __forceinline__ Sigmoid sigmoid64(double x) {
  const double t = exp64(-fabs(x)), d = 1.0 + t;
  double r = __builtin_amdgcn_rcp(d);
  r = __builtin_fma(__builtin_fma(-d, r, 1.0), r, r);
  r = __builtin_fma(__builtin_fma(-d, r, 1.0), r, r);
  return {x < 0.0 ? t * r : r, x < 0.0 ? r : t * r, t * r * r};
}

// w_k (dw_k - sum_j dw_j w_j) of a token's choices, s their scores.
template <int L>
__device__ __forceinline__ double gate_share_gradient(const GateChoice& c, double s, bool sigmoid) {
  const bool live = c.x > kNone;
  if (!live) s = 0.0;
  double total = gate_sum<L>(s), dot = gate_sum<L>(live ? c.dw * s : 0.0);
  if (__builtin_amdgcn_ballot_w64(live && far_scores(total, sigmoid))) {
    const double top = gate_max<L>(c.x), e = live ? exp64(c.x - top) : 0.0;
    const double sum = gate_sum<L>(e), edot = gate_sum<L>(live ? c.dw * e : 0.0);
    if (far_scores(total, sigmoid)) {
      s = e;
      total = sum;
      dot = edot;
    }
  }
  const double inv = total > 0.0 ? 1.0 / total : 0.0;  // (2^900 at most, or of a sum of 1 or more)
  return s * inv * (c.dw - dot * inv);
}

// Where only the chosen experts have a gradient (a sigmoid, or the renormalised
// softmax, without dscores): the row is laid out in LDS, zeros but for them, and
// its logits are read at them alone.  L lanes a token.  16384 x 256 float32: 8.6
// us, of which 2.6 are the launch and 2.5 the 17 MB that are written; the rest is
// two loads that wait for one another and the 64-bit steps of one choice a lane.
template <int L>
__global__ __launch_bounds__(64 * kGateWaves) void gate_bwd_few_kernel(GateBwdArgs a) {
  extern __shared__ __attribute__((aligned(16))) float rows[];
  constexpr int kTokens = 64 / L;
  const int lane = threadIdx.x & (L - 1), sub = (threadIdx.x & 63) / L;
  const int pad = (a.experts + 7) / 8 * 8;
  float* r = rows + ((threadIdx.x >> 6) * kTokens + sub) * pad;
  const int64_t stride = (int64_t)gridDim.x * kGateWaves * kTokens;
  for (int64_t t0 = ((int64_t)blockIdx.x * kGateWaves + (int)(threadIdx.x >> 6)) * kTokens; t0 < a.tokens; t0 += stride) {
    const bool real = t0 + sub < a.tokens;
    const int64_t t = real ? t0 + sub : a.tokens - 1;
    const GateChoice c = gate_choice<L>(a, t, lane);
    for (int i = lane * 4; i < pad; i += L * 4) *reinterpret_cast<float4*>(r + i) = make_float4(0.f, 0.f, 0.f, 0.f);
    gate_wave_fence();
    double dx;
    if (a.sigmoid) {
      const Sigmoid y = sigmoid64(c.x);
      dx = a.scale * (a.renormalize ? gate_share_gradient<L>(c, y.s, true) * y.rest : c.dw * y.slope);
    } else {
      const double top = gate_max<L>(c.x);
      const double e = c.x > kNone ? exp64(c.x - top) : 0.0;
      const double total = gate_sum<L>(e), w = total > 0.0 ? e / total : 0.0;
      const double dot = gate_sum<L>(c.e >= 0 ? c.dw * w : 0.0);
      dx = a.scale * w * (c.dw - dot);
    }
    dx = gate_same<L>(c.x > kNone ? dx : 0.0, c.e, a.topk);
    if (c.e >= 0) r[c.e] = (float)dx;
    gate_wave_fence();
    if (!real) continue;
    if (a.of32) {
      for (int i = lane * 4; i < a.experts; i += L * 4) {
        const float4 v = *reinterpret_cast<const float4*>(r + i);
        const float f[4] = {v.x, v.y, v.z, v.w};
        st_float4(static_cast<float*>(a.dlogits) + t * a.ldd + i, f, a.experts - i, false);
      }
    } else {
      for (int i = lane * 8; i < a.experts; i += L * 8) {
        const float4 u = *reinterpret_cast<const float4*>(r + i), v = *reinterpret_cast<const float4*>(r + i + 4);
        const float f[8] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
        st_bf16x8(static_cast<uint16_t*>(a.dlogits) + t * a.ldd + i, pack_bf16x8(f), a.experts - i, false);
      }
    }
  }
}

// Every expert: a lane has P consecutive ones, the chosen ones' part comes to it
// through LDS, where the lanes' p-th values lie side by side.  Bound by the
// exponentials of every expert in 64 bits (16384 x 256: 20 us, the bytes 8).
template <int L, int P>
__global__ __launch_bounds__(64 * kGateWaves) void gate_bwd_all_kernel(GateBwdArgs a) {
  extern __shared__ __attribute__((aligned(16))) double ds_rows[];
  constexpr int kTokens = 64 / L;
  const int lane = threadIdx.x & (L - 1), sub = (threadIdx.x & 63) / L, base = lane * P;
  double* r = ds_rows + ((threadIdx.x >> 6) * kTokens + sub) * (L * P);
  const int64_t stride = (int64_t)gridDim.x * kGateWaves * kTokens;
  for (int64_t t0 = ((int64_t)blockIdx.x * kGateWaves + (int)(threadIdx.x >> 6)) * kTokens; t0 < a.tokens; t0 += stride) {
    const bool real = t0 + sub < a.tokens;
    const int64_t t = real ? t0 + sub : a.tokens - 1;
    const GateChoice c = gate_choice<L>(a, t, lane);
    float f[P], g[P];
#pragma unroll
    for (int p = 0; p < P; p += 4) {
      const int left = a.experts - base - p;
      if (a.lf32) {
        const auto v = ld_raw<true, 4, true>(a.logits, t * a.ld + base + p, left, false);
#pragma unroll
        for (int i = 0; i < 4; ++i) f[p + i] = v.at(i);
      } else {
        const auto v = ld_raw<false, 4, true>(a.logits, t * a.ld + base + p, left, false);
#pragma unroll
        for (int i = 0; i < 4; ++i) f[p + i] = v.at(i);
      }
      const auto v = ld_raw<true, 4, true>(a.dscores, t * a.experts + base + p, a.dscores ? left : 0, false);
#pragma unroll
      for (int i = 0; i < 4; ++i) g[p + i] = v.at(i);
    }
#pragma unroll
    for (int p = 0; p < P; ++p) r[p * L + lane] = 0.0;
    gate_wave_fence();
    double top = kNone, inv = 0.0;
    double s[P];  // scores, or slopes of the sigmoid
#pragma unroll
    for (int p = 0; p < P; ++p) s[p] = base + p < a.experts ? as_logit(f[p]) : kNone;
    if (a.sigmoid) {
#pragma unroll
      for (int p = 0; p < P; ++p) s[p] = s[p] > kNone ? sigmoid64(s[p]).slope : 0.0;
    } else {
      top = gate_max<L>(gate_tree_max<P>(s));
      double total = 0.0;
#pragma unroll
      for (int p = 0; p < P; ++p) {
        s[p] = s[p] > kNone ? exp64(s[p] - top) : 0.0;
        total += s[p];
      }
      total = gate_sum<L>(total);
      inv = total > 0.0 ? 1.0 / total : 0.0;
#pragma unroll
      for (int p = 0; p < P; ++p) s[p] *= inv;
    }
    // the chosen logits' part, a softmax's without its mean
    double dx;
    if (a.sigmoid) {
      const Sigmoid y = sigmoid64(c.x);
      dx = a.renormalize ? gate_share_gradient<L>(c, y.s, true) * y.rest : c.dw * y.slope;
    } else {
      const double mine = score_of(c.x, false, top, inv);
      dx = a.renormalize ? gate_share_gradient<L>(c, mine, false) : c.dw * mine;
    }
    dx = c.x > kNone ? a.scale * dx : 0.0;
    double mean = 0.0;
    if (!a.sigmoid) {
      if (!a.renormalize) mean = dx;
#pragma unroll
      for (int p = 0; p < P; ++p)
        if (s[p] > 0.0) mean += (double)g[p] * s[p];
      mean = gate_sum<L>(mean);
    }
    dx = gate_same<L>(dx, c.e, a.topk);
    if (c.e >= 0) r[c.e % P * L + c.e / P] = dx;
    gate_wave_fence();
    float d[P];
#pragma unroll
    for (int p = 0; p < P; ++p) d[p] = (float)(r[p * L + lane] + (s[p] > 0.0 ? ((double)g[p] - mean) * s[p] : 0.0));
    gate_wave_fence();
    if (!real) continue;
#pragma unroll
    for (int p = 0; p < P; p += 4) {
      const int left = a.experts - base - p;
      if (left <= 0) continue;
      if (a.of32) {
        st_float4(static_cast<float*>(a.dlogits) + t * a.ldd + base + p, d + p, left, false);
      } else {
        const uint32_t lo = __builtin_bit_cast(uint32_t, c8_v2bf{(__bf16)d[p], (__bf16)d[p + 1]});
        const uint32_t hi = __builtin_bit_cast(uint32_t, c8_v2bf{(__bf16)d[p + 2], (__bf16)d[p + 3]});
        uint16_t* o = static_cast<uint16_t*>(a.dlogits) + t * a.ldd + base + p;
        if (left >= 4) {
          *reinterpret_cast<Any8*>(o) = Any8{{lo, hi}};
        } else {
          o[0] = (uint16_t)lo;
          if (left > 1) o[1] = (uint16_t)(lo >> 16);
          if (left > 2) o[2] = (uint16_t)hi;
        }
      }
    }
  }
}

// The number of pairs of every expert, added to load: counts in LDS, one set a
// wave, then one atomic an expert.  The pairs' own atomics on load, which of all
// XCDs meet in memory, come through at about one a nanosecond: eight of 256
// experts 1.9 us at 256 tokens, 4.4 at 512, 23 at 4096, 88 at 16384; this takes
// 2.0, 2.2, 2.7 and 2.8 us.
template <bool I64>
__global__ __launch_bounds__(1024) void gate_load_kernel(const void* chosen, int64_t pairs, int experts, int* load) {
  __shared__ int count[16][kMaxGateExperts];
  using Int = std::conditional_t<I64, int64_t, int32_t>;
  const Int* e = static_cast<const Int*>(chosen);
  int* mine = count[threadIdx.x >> 6];
  for (int i = threadIdx.x & 63; i < experts; i += 64) mine[i] = 0;
  gate_wave_fence();
  const int64_t lo = (int64_t)blockIdx.x * kGateLoadPairs + threadIdx.x;
  Int at[kGateLoadPairs / 1024];  // (all on their way together)
#pragma unroll
  for (int i = 0; i < kGateLoadPairs / 1024; ++i) at[i] = lo + i * 1024 < pairs ? e[lo + i * 1024] : -1;
#pragma unroll
  for (int i = 0; i < kGateLoadPairs / 1024; ++i)
    if (at[i] >= 0) atomicAdd(mine + at[i], 1);
  __syncthreads();
  for (int i = threadIdx.x; i < experts; i += 1024) {
    int sum = 0;
#pragma unroll
    for (int w = 0; w < 16; ++w) sum += count[w][i];
    if (sum) atomicAdd(load + i, sum);
  }
}

int gate_grid(int64_t waves) {
  const int64_t want = (waves + kGateWaves - 1) / kGateWaves;
  return (int)(want < kMaxGateGrid ? want : kMaxGateGrid);
}

}  // namespace

template <int L, int BY>
static void launch_gate_by(const GateArgs& a, int per, hipStream_t stream) {
  // (of 32 lanes nearly always more than four each: experts or choices enough that 16 would not do)
  auto kernel = L == 32 ? gate_kernel<L, kGateLane, BY> : per <= 4 ? gate_kernel<L, L == 32 ? kGateLane : 4, BY>
                : per <= 8 ? gate_kernel<L, L == 32 ? kGateLane : 8, BY> : gate_kernel<L, kGateLane, BY>;
  const int64_t waves = ((int64_t)a.tokens * L + 63) / 64;
  hipLaunchKernelGGL(kernel, dim3(gate_grid(waves)), dim3(64 * kGateWaves), 0, stream, a);
}
template <int L>
static void launch_gate_lanes(const GateArgs& a, int per, hipStream_t stream) {
  if (!a.bias) {
    launch_gate_by<L, kByLogit>(a, per, stream);
  } else if (a.sigmoid) {
    launch_gate_by<L, kBySigmoid>(a, per, stream);
  } else {
    launch_gate_by<L, kBySoftmax>(a, per, stream);
  }
}

// Four tokens a wave take less time in all, one a wave less for each: of 256
// experts, 2048 tokens 7.4 against 6.8 us, 4099 8.8 against 9.5, 16384 13.2
// against 22.7; of 60, 1024 tokens 3.6 against 3.9, 16384 5.5 against 15.4.
// Where the scores of all experts are written, in 64-bit steps, few lanes have
// many of them to do: of 60, 1024 tokens 5.0 against 5.3, 4096 5.2 against 8.6;
// of 128, 2048 8.0 against 7.2, 4096 7.1 against 8.7 (a softmax 7.8 against
// 8.6); of 160, 4096 9.0 against 8.7, 8192 12.5 against 14.8 (12.6 against
// 14.1); of 256, 4096 10.3 against 9.0, 8192 13.8 against 15.5 (a softmax 15.8
// against 14.9), 16384 21.6 against 26.3 (23.1 against 25.5).
static int gate_narrow_from(const GateArgs& a) {
  if (!a.scores) return a.narrow.per <= 8 ? 1024 : 4096;
  return a.narrow.per <= 4 ? 1024 : a.narrow.per <= 8 ? 4096 : a.narrow.per <= 12 || a.sigmoid ? 8192 : 16384;
}
// Two tokens a wave, where four would leave a lane more experts than its
// registers hold: of 384 experts, 2048 tokens 7.1 against 6.6 with one, 4096 7.9
// against 8.2, 16384 18.0 against 23.1; of 512, sixteen of them, 24 against 31.
// So where 16 lanes are too few for the choices, 15 to 30 of them, unless every
// score is written as well; with a bias, whose unclear tokens cost more, only
// from 16384 tokens on: sixteen of 256 by logits, 2048 tokens 6.7 against 5.8,
// 4096 7.4 against 7.9, 16384 18.1 against 22.1; with a bias 4096 9.9 against
// 9.1, 16384 22.6 against 23.9 (a softmax 13.6 against 11.7 and 26.3 against 27.5).
static int gate_middle_from(const GateArgs& a) { return a.bias && a.narrow.fits ? 16384 : 4096; }

// How `lanes` lanes a token share out the experts (GateLane).
static GateSplit gate_split(const GateArgs& a, int lanes) {
  GateSplit s{};
  int groups = 1;
  while (groups < a.groups) groups *= 2;
  while ((groups << s.lane_bits) < lanes) ++s.lane_bits;
  s.per = (a.per_group + (1 << s.lane_bits) - 1) >> s.lane_bits;
  s.per = (s.per + 3) / 4 * 4;
  s.fits = groups <= lanes && s.per <= kGateLane;
  return s;
}

hipError_t launch_gate(GateArgs a, hipStream_t stream) {
  int* const load = a.load;
  const int64_t pairs = (int64_t)a.tokens * a.topk;
  const bool apart = load && pairs >= kGateLoadApart;
  if (apart) a.load = nullptr;
  a.per_group = a.experts / a.groups;
  a.wide = gate_split(a, 64);
  a.middle = gate_split(a, 32);
  a.narrow = gate_split(a, 16);
  if (a.topk + 2 > 64 || (a.groups > 1 && a.two_best && !a.bias)) {
    // (no lane for each expert taken, two more than asked for; groups by scores, experts by logits)
    auto kernel = a.wide.per <= 4 ? gate_exact_kernel<4> : a.wide.per <= 8 ? gate_exact_kernel<8> : gate_exact_kernel<kGateLane>;
    hipLaunchKernelGGL(kernel, dim3(gate_grid(a.tokens)), dim3(64 * kGateWaves), 0, stream, a);
  } else if (a.narrow.fits && a.topk + 2 <= 16 && a.tokens >= gate_narrow_from(a)) {
    launch_gate_lanes<16>(a, a.narrow.per, stream);
  } else if (a.middle.fits && a.topk + 2 <= 32 && (!a.narrow.fits || (a.topk + 2 > 16 && !a.scores)) && a.tokens >= gate_middle_from(a)) {
    launch_gate_lanes<32>(a, a.middle.per, stream);
  } else {
    launch_gate_lanes<64>(a, a.wide.per, stream);
  }
  if (apart) {
    hipLaunchKernelGGL(a.i64 ? gate_load_kernel<true> : gate_load_kernel<false>, dim3((pairs + kGateLoadPairs - 1) / kGateLoadPairs), dim3(1024), 0, stream,
                       a.chosen, pairs, a.experts, load);
  }
  return hipGetLastError();
}

// 16 lanes a token leave a quarter of the waves, 64 the shorter way through a
// row.  Gradients at the choice alone, eight of 256 (us, 16 lanes / 64): 3.2 /
// 2.9 at one token, 3.8 / 3.8 at 2048, 4.1 / 4.6 at 4096, 8.5 / 12.0 at 16384.
// At every expert (a sigmoid's with dscores): of 60, 3.6 / 3.6 at one token,
// 6.4 / 16.5 at 16384; of 128, 5.3 / 5.0 at 2048, 5.5 / 6.5 at 4096, 11.7 /
// 18.8 at 16384; of 256, 6.8 / 3.8 at one, 22.5 / 19.4 at 16384.
hipError_t launch_gate_backward(const GateBwdArgs& a, hipStream_t stream) {
  const bool all = a.dscores || (!a.sigmoid && !a.renormalize);
  const bool wide = a.topk > 16 || (all ? a.experts > (a.tokens >= 4096 ? 128 : 64) : a.tokens < 2048);
  const int lanes = wide ? 64 : 16, tokens = kGateWaves * 64 / lanes;
  const dim3 grid(gate_grid(((int64_t)a.tokens * lanes + 63) / 64)), block(64 * kGateWaves);
  if (all) {
    const bool four = a.experts <= 4 * lanes;
    const auto kernel = wide ? (four ? gate_bwd_all_kernel<64, 4> : gate_bwd_all_kernel<64, 8>) : (four ? gate_bwd_all_kernel<16, 4> : gate_bwd_all_kernel<16, 8>);
    hipLaunchKernelGGL(kernel, grid, block, (size_t)tokens * lanes * (four ? 4 : 8) * sizeof(double), stream, a);
  } else {
    hipLaunchKernelGGL(wide ? gate_bwd_few_kernel<64> : gate_bwd_few_kernel<16>, grid, block, (size_t)tokens * ((a.experts + 7) / 8 * 8) * sizeof(float), stream, a);
  }
  return hipGetLastError();
}

}  // namespace fp8q
