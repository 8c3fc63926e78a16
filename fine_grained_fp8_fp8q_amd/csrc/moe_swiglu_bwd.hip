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
// of inter (lane sub: 8 gates and 8 ups), a wave four tiles that follow one
// another.  One pass, four tiles a wave: 32768 x 2048 from the cache with y
// takes 107 us (6.3 TB/s); a grid of 2048 workgroups that loop with the next
// tiles' loads in flight takes 124.
template <bool CACHE, bool QUANT, bool POW2, bool VEC, bool KEEP>
__global__ __launch_bounds__(256) void swiglu_bwd_kernel(SwigluBwdArgs a) {
  static_assert(VEC || KEEP, "loads of unaligned rows are plain ones");
  const int lane = threadIdx.x & 63;
  const int sub = lane & 15;
  const uint32_t t = ((blockIdx.x * 256u + threadIdx.x) >> 6) * 4u + (uint32_t)(lane >> 4);
  const bool valid = t < (uint32_t)a.ntiles;
  const int row = valid ? (int)(t / (uint32_t)a.nb) : 0;
  const int cb = valid ? (int)(t - (uint32_t)row * (uint32_t)a.nb) : 0;
  const int col = cb * 128 + sub * 8;
  int left = valid ? a.inter - col : 0;  // columns of inter from col on (0: no tile)
  if (VEC) left = left > 0 ? 8 : 0;      // whole chunks only

  uint4 cg, cu;
  float sg = 1.0f, su = 1.0f;
  if constexpr (CACHE) {
    const uint8_t* src = static_cast<const uint8_t*>(a.x) + (int64_t)row * a.ldx + col;
    const uint2 gc = ld_codes8<KEEP>(src, left, VEC), uc = ld_codes8<KEEP>(src + a.inter, left, VEC);
    cg = make_uint4(gc.x, gc.y, 0, 0);
    cu = make_uint4(uc.x, uc.y, 0, 0);
    if (left > 0) {
      const float* s = a.xscales + (int64_t)row * (2 * a.nb) + cb;
      sg = s[0];
      su = s[a.nb];
    }
  } else {
    const uint16_t* src = static_cast<const uint16_t*>(a.x) + (int64_t)row * a.ldx + col;
    cg = ld_bf16x8<KEEP>(src, left, VEC);
    cu = ld_bf16x8<KEEP>(src + a.inter, left, VEC);
  }
  const uint4 cd = ld_bf16x8<KEEP>(a.dy + (int64_t)row * a.lddy + col, left, VEC);

  float g[8], u[8], d[8], dg[8], du[8], y[8];
  widen8<CACHE>(cg, sg, g);
  widen8<CACHE>(cu, su, u);
  widen8<false>(cd, 1.0f, d);
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const float e = exp_nonpos(-__builtin_fabsf(g[k]));
    const float r = __builtin_amdgcn_rcpf(1.0f + e);
    const float er = e * r;
    const float s = g[k] >= 0.0f ? r : er;
    const float silu = g[k] * s;
    y[k] = silu * u[k];
    du[k] = d[k] * silu;
    dg[k] = (d[k] * u[k]) * __builtin_fmaf(silu, g[k] >= 0.0f ? er : r, s);
  }
  const uint4 og = pack_bf16x8(dg), ou = pack_bf16x8(du);
  if (a.dx) {
    uint16_t* dst = a.dx + (int64_t)row * a.lddx + col;
    st_bf16x8(dst, og, left, VEC);
    st_bf16x8(dst + a.inter, ou, left, VEC);
  }
  if (a.y) st_bf16x8(a.y + (int64_t)row * a.ldy + col, pack_bf16x8(y), left, VEC);
  if constexpr (QUANT) {
    // inter is a multiple of 128: the gate chunk is tile cb of dx's row, the
    // up chunk tile nb + cb (every lane of the wave takes part)
    uint8_t* dst = a.codes + (int64_t)row * a.ldc + col;
    float* sdst = a.scales + (int64_t)row * (2 * a.nb) + cb;
    auto quant = [&](uint4 v, uint8_t* to, float* sto) {
      const TileScale ts = tile_scale<POW2>(dpp_max16(absmax8(v)));
      st_codes8(to, encode8<POW2>(v, ts), left, VEC);
      if (sub == 0 && left > 0) *sto = ts.s;
    };
    quant(og, dst, sdst);
    quant(ou, dst + a.inter, sdst + a.nb);
  }
}

template <bool CACHE, bool VEC, bool KEEP>
void launch(const SwigluBwdArgs& a, bool pow2, hipStream_t stream) {
  const int grid = (int)(((int64_t)a.ntiles + 15) / 16);  // < 2^24
  auto kernel = !a.codes ? swiglu_bwd_kernel<CACHE, false, false, VEC, KEEP>
                : pow2   ? swiglu_bwd_kernel<CACHE, true, true, VEC, KEEP>
                         : swiglu_bwd_kernel<CACHE, true, false, VEC, KEEP>;
  hipLaunchKernelGGL(kernel, dim3(grid), dim3(256), 0, stream, a);
}

// VEC: whole 8-element chunks on 16-byte (codes: 8-byte) boundaries
template <bool CACHE>
void launch_form(const SwigluBwdArgs& a, bool vec, bool keep, bool pow2, hipStream_t stream) {
  if (vec) {
    keep ? launch<CACHE, true, true>(a, pow2, stream) : launch<CACHE, true, false>(a, pow2, stream);
  } else {  // (unaligned loads are plain ones)
    launch<CACHE, false, true>(a, pow2, stream);
  }
}

}  // namespace

hipError_t launch_swiglu_backward(const void* x, const float* xscales, int rows, int inter, int64_t ldx,
                                  const uint16_t* dy, int64_t lddy, uint16_t* dx, int64_t lddx, bool pow2,
                                  uint8_t* codes, int64_t ldc, float* scales, uint16_t* y, int64_t ldy,
                                  hipStream_t stream) {
  SwigluBwdArgs a{};
  a.x = x; a.xscales = xscales; a.ldx = ldx; a.dy = dy; a.lddy = lddy; a.dx = dx; a.lddx = lddx;
  a.codes = codes; a.ldc = ldc; a.scales = scales; a.y = y; a.ldy = ldy;
  a.inter = inter; a.nb = (inter + 127) / 128; a.ntiles = rows * a.nb;  // < 2^28 (checked by the entry point)
  const bool vec = inter % 8 == 0 && ldx % 8 == 0 && lddy % 8 == 0 && (!dx || lddx % 8 == 0) &&
                   (!codes || ldc % 8 == 0) && (!y || ldy % 8 == 0);
  const bool keep = input_stays_cached(rows, (xscales ? 1 : 2) * ldx + 2 * lddy);
  if (xscales) {
    launch_form<true>(a, vec, keep, pow2, stream);
  } else {
    launch_form<false>(a, vec, keep, pow2, stream);
  }
  return hipGetLastError();
}

}  // namespace fp8q
