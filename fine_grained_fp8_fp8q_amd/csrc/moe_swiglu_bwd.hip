// Gradient of the MoE's SwiGLU (tmdrlife.com wr_id=13334 ¶3-¶4: its inputs
// are cached in FP8 and its output is recomputed from them in the backward
// pass), gfx950.
//
// With s = sigma(g) = 1 / (1 + e^-g), x = [g | u] and y = g s u:
//   dg = dy u (s + g s (1 - s)),   du = dy g s.
// s and 1 - s both come from t = e^-|g| in (0, 1]: r = 1 / (1 + t), and
// (s, 1 - s) is (r, t r) for g >= 0 and (t r, r) for g < 0, so neither tail
// cancels.  Everything is float32; x is the BF16 up-projection output or its
// FP8 cache (an E4M3 code times its 1x128 scale, one rounding, none for
// power-of-two scales).  One pass reads x and dy once and writes, as asked,
// dx in BF16, dx quantized per 1x128 tile (of the BF16 value, as the plain
// quantizer would), and y in BF16.
#include "chunk8.h"
#include "fp8q_internal.h"
#include "quant_common.h"
#include "swiglu_common.h"

namespace fp8q {
namespace {

typedef __bf16 sb_v2bf __attribute__((ext_vector_type(2)));
typedef float sb_v2f __attribute__((ext_vector_type(2)));

struct SwigluBwdArgs {
  const void* x;
  const float* xscales;
  int64_t ldx;
  const uint16_t* dy;
  int64_t lddy;
  uint16_t* dx;      // null: not written
  int64_t lddx;
  uint8_t* codes;    // (QUANT)
  int64_t ldc;
  float* scales;
  uint16_t* y;       // null: not written
  int64_t ldy;
  int inter, nb, ntiles;
};

// Eight elements of x: BF16 (16 bytes) or E4M3 codes (8 bytes, in .x and .y)
// with their tile's scale.
template <bool CACHE>
__device__ __forceinline__ void widen8(uint4 c, float scale, float* v) {
  if constexpr (CACHE) {
    const uint32_t w[2] = {c.x, c.y};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const sb_v2f lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[i], false);
      const sb_v2f hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[i], true);
      v[4 * i] = lo[0] * scale;
      v[4 * i + 1] = lo[1] * scale;
      v[4 * i + 2] = hi[0] * scale;
      v[4 * i + 3] = hi[1] * scale;
    }
  } else {
    const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = bf16_lo(w[i]);
      v[2 * i + 1] = bf16_hi(w[i]);
    }
  }
}

// As in the forward kernel, a 16-lane DPP row owns one tile of 128 columns
// of inter (lane sub: 8 gates and 8 ups), a wave four tiles a step of a
// grid-stride loop, with the next step's loads in flight through the
// arithmetic of this one.
template <bool CACHE, bool QUANT, bool POW2, bool VEC>
__global__ __launch_bounds__(256) void swiglu_bwd_kernel(SwigluBwdArgs a) {
  const int lane = threadIdx.x & 63;
  const int grp = lane >> 4, sub = lane & 15;
  const uint32_t wave = (blockIdx.x * 256u + threadIdx.x) >> 6;
  const uint32_t step = gridDim.x * 16u;

  struct Chunk {
    uint4 g, u, d;
    float sg, su;
    int row, col, left;  // left: columns of inter from col on (0: no tile)
  };
  auto fetch = [&](uint32_t base, Chunk& c) {
    const uint32_t t = base + (uint32_t)grp;
    const bool valid = t < (uint32_t)a.ntiles;
    c.row = valid ? (int)(t / (uint32_t)a.nb) : 0;
    const int cb = valid ? (int)(t - (uint32_t)c.row * (uint32_t)a.nb) : 0;
    c.col = cb * 128 + sub * 8;
    c.left = valid ? a.inter - c.col : 0;
    if (VEC) c.left = c.left > 0 ? 8 : 0;  // whole chunks only
    c.sg = c.su = 1.0f;
    if constexpr (CACHE) {
      const uint8_t* src = static_cast<const uint8_t*>(a.x) + (int64_t)c.row * a.ldx + c.col;
      const uint2 g = ld_codes8(src, c.left, VEC), u = ld_codes8(src + a.inter, c.left, VEC);
      c.g = make_uint4(g.x, g.y, 0, 0);
      c.u = make_uint4(u.x, u.y, 0, 0);
      if (c.left > 0) {
        const float* s = a.xscales + (int64_t)c.row * (2 * a.nb) + cb;
        c.sg = s[0];
        c.su = s[a.nb];
      }
    } else {
      const uint16_t* src = static_cast<const uint16_t*>(a.x) + (int64_t)c.row * a.ldx + c.col;
      c.g = ld_bf16x8(src, c.left, VEC);
      c.u = ld_bf16x8(src + a.inter, c.left, VEC);
    }
    c.d = ld_bf16x8(a.dy + (int64_t)c.row * a.lddy + c.col, c.left, VEC);
  };

  uint32_t base = wave * 4u;
  if (base >= (uint32_t)a.ntiles) return;  // (wave-uniform)
  Chunk cur;
  fetch(base, cur);
  for (; base < (uint32_t)a.ntiles; base += step) {
    Chunk nxt = cur;
    const uint32_t nbase = base + step;
    if (nbase < (uint32_t)a.ntiles) fetch(nbase, nxt);  // (wave-uniform)
    float g[8], u[8], d[8];
    widen8<CACHE>(cur.g, cur.sg, g);
    widen8<CACHE>(cur.u, cur.su, u);
    widen8<false>(cur.d, 1.0f, d);
    uint32_t wg[4], wu[4], wy[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float dg[2], du[2], yy[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int k = 2 * i + h;
        const float t = exp_nonpos(-__builtin_fabsf(g[k]));
        const float r = __builtin_amdgcn_rcpf(1.0f + t);
        const float tr = t * r;
        const float s = g[k] >= 0.0f ? r : tr;
        const float silu = g[k] * s;
        yy[h] = silu * u[k];
        du[h] = d[k] * silu;
        dg[h] = (d[k] * u[k]) * __builtin_fmaf(silu, g[k] >= 0.0f ? tr : r, s);
      }
      wg[i] = __builtin_bit_cast(uint32_t, sb_v2bf{(__bf16)dg[0], (__bf16)dg[1]});
      wu[i] = __builtin_bit_cast(uint32_t, sb_v2bf{(__bf16)du[0], (__bf16)du[1]});
      wy[i] = __builtin_bit_cast(uint32_t, sb_v2bf{(__bf16)yy[0], (__bf16)yy[1]});
    }
    const uint4 cg = make_uint4(wg[0], wg[1], wg[2], wg[3]);
    const uint4 cu = make_uint4(wu[0], wu[1], wu[2], wu[3]);
    if (a.dx) {
      uint16_t* dst = a.dx + (int64_t)cur.row * a.lddx + cur.col;
      st_bf16x8(dst, cg, cur.left, VEC);
      st_bf16x8(dst + a.inter, cu, cur.left, VEC);
    }
    if (a.y)
      st_bf16x8(a.y + (int64_t)cur.row * a.ldy + cur.col, make_uint4(wy[0], wy[1], wy[2], wy[3]), cur.left, VEC);
    if constexpr (QUANT) {
      // inter is a multiple of 128: the gate chunk is tile cb of dx's row,
      // the up chunk tile nb + cb (every lane of the wave takes part)
      uint8_t* dst = a.codes + (int64_t)cur.row * a.ldc + cur.col;
      float* sdst = a.scales + (int64_t)cur.row * (2 * a.nb) + (cur.col >> 7);
      auto quant = [&](uint4 v, uint8_t* to, float* sto) {
        const TileScale ts = tile_scale<POW2>(dpp_max16(absmax8(v)));
        const uint2 c = encode8<POW2>(v, ts);
        st_codes8(to, c, cur.left, VEC);
        if (sub == 0 && cur.left > 0) *sto = ts.s;
      };
      quant(cg, dst, sdst);
      quant(cu, dst + a.inter, sdst + a.nb);
    }
    cur = nxt;
  }
}

template <bool CACHE, bool VEC>
void launch(const SwigluBwdArgs& a, bool pow2, hipStream_t stream) {
  const int64_t waves = ((int64_t)a.ntiles + 3) / 4;
  auto kernel = !a.codes ? swiglu_bwd_kernel<CACHE, false, false, VEC>
                         : pow2 ? swiglu_bwd_kernel<CACHE, true, true, VEC> : swiglu_bwd_kernel<CACHE, true, false, VEC>;
  hipLaunchKernelGGL(kernel, dim3(stream_grid(waves)), dim3(256), 0, stream, a);
}

}  // namespace

hipError_t launch_swiglu_backward(const void* x, const float* xscales, int rows, int inter, int64_t ldx,
                                  const uint16_t* dy, int64_t lddy, uint16_t* dx, int64_t lddx, bool pow2,
                                  uint8_t* codes, int64_t ldc, float* scales, uint16_t* y, int64_t ldy,
                                  hipStream_t stream) {
  SwigluBwdArgs a{};
  a.x = x; a.xscales = xscales; a.ldx = ldx; a.dy = dy; a.lddy = lddy; a.dx = dx; a.lddx = lddx;
  a.codes = codes; a.ldc = ldc; a.scales = scales; a.y = y; a.ldy = ldy;
  a.inter = inter; a.nb = (inter + 127) / 128; a.ntiles = rows * a.nb;  // < 2^31 (checked by the entry point)
  // VEC: whole 8-element chunks on 16-byte (codes: 8-byte) boundaries
  const bool vec = inter % 8 == 0 && ldx % 8 == 0 && lddy % 8 == 0 && (!dx || lddx % 8 == 0) &&
                   (!codes || ldc % 8 == 0) && (!y || ldy % 8 == 0);
  if (xscales) {
    vec ? launch<true, true>(a, pow2, stream) : launch<true, false>(a, pow2, stream);
  } else {
    vec ? launch<false, true>(a, pow2, stream) : launch<false, false>(a, pow2, stream);
  }
  return hipGetLastError();
}

}  // namespace fp8q
