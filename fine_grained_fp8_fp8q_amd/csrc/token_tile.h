// 128x1 token-axis tiles: from a workgroup's values in registers to codes and
// scales, feature-major (gfx950).
#pragma once

#include "quant_common.h"

namespace fp8q {

// Workgroups are dealt to the 8 XCDs in turn (workgroup i to XCD i % 8).
// This maps them so that each XCD runs one contiguous range of logical
// blocks: the token blocks of a feature group follow one another on one XCD,
// and the 4-byte scales they write, adjacent in each feature's scale row,
// meet in that XCD's L2 as whole lines instead of reaching memory as
// partial-line writes from eight L2s.
__device__ __forceinline__ int xcd_block(int bid, int nblk) {
  const int xcd = bid & 7, idx = bid >> 3;
  const int per = nblk >> 3, rem = nblk & 7;
  return xcd * per + min(xcd, rem) + idx;
}

// The workgroup's 256 threads hold 128 tokens x 64 features of BF16 values.
// Thread (q = tid/8, c8 = tid%8) has tokens 4q..4q+3 of features 8c8..8c8+7,
// so for each feature it holds four consecutive tokens: one code word.  The
// per-feature max-abs runs over the 32 threads sharing c8; codes go through
// LDS ([feature][token], 144-byte rows) and leave feature-major, 128 tokens
// (one 128-byte line) per feature.  Within a row the token words are rotated
// by 8 words per group of 8 features: the 64 lanes that write one word each
// (8 feature groups x 8 token words) then hit 64 distinct banks, where the
// unrotated rows put every feature group on the same two bank offsets.
constexpr int kTokenRowBytes = 144;  // 16-byte aligned rows for the store reads
struct TokenTileLds {
  uint32_t red[4][64];
  // per-feature scale state, read back 8 features (32 bytes) at a time
  __attribute__((aligned(16))) float div[64];
  __attribute__((aligned(16))) float mul[64];
  __attribute__((aligned(16))) int nege[64];
  unsigned char slow[64];
  int anyslow;  // some feature of the block has a tiny amax
  __attribute__((aligned(16))) uint8_t tile[64 * kTokenRowBytes];
};

// v: the thread's four tokens, values past the tensor +0.  t0, f0: the
// block's first token (of `rows`) and feature (of `cols`), tb its token block
// of ntb.  full: the block lies inside the tensor and the rows of codes are on
// 16-byte boundaries.
template <bool POW2>
__device__ __forceinline__ void token_tile(const uint4 (&v)[4], TokenTileLds& sh, int t0, int f0, int tb, int ntb, int rows, int cols, bool full,
                                           uint8_t* __restrict__ codes, int64_t ldc, float* __restrict__ scales) {
  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int wave = tid >> 6;
  const int c8 = tid & 7;
  const int q = tid >> 3;  // 0..31
  // per-feature max-abs over this thread's 4 tokens, packed two features per word
  const uint32_t k = 0x7FFF7FFFu;
  uint32_t m[4];
  m[0] = pk_max_u16(pk_max_u16(v[0].x & k, v[1].x & k), pk_max_u16(v[2].x & k, v[3].x & k));
  m[1] = pk_max_u16(pk_max_u16(v[0].y & k, v[1].y & k), pk_max_u16(v[2].y & k, v[3].y & k));
  m[2] = pk_max_u16(pk_max_u16(v[0].z & k, v[1].z & k), pk_max_u16(v[2].z & k, v[3].z & k));
  m[3] = pk_max_u16(pk_max_u16(v[0].w & k, v[1].w & k), pk_max_u16(v[2].w & k, v[3].w & k));
  // across the 8 lanes of the wave with the same c8 (lane bits 3..5):
  // lane l ^ 8 is lane l rotated by 8 within its 16-lane DPP row
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    m[i] = pk_max_u16(m[i], (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m[i], 0x128, 0xF, 0xF, false));
    m[i] = pk_max_u16(m[i], (uint32_t)__shfl_xor((int)m[i], 16));
    m[i] = pk_max_u16(m[i], (uint32_t)__shfl_xor((int)m[i], 32));
  }
  if (tid == 0) sh.anyslow = 0;
  if (lane < 8) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      sh.red[wave][8 * c8 + 2 * i] = m[i] & 0xFFFFu;
      sh.red[wave][8 * c8 + 2 * i + 1] = m[i] >> 16;
    }
  }
  __syncthreads();
  if (tid < 64) {
    const uint32_t a = max(max(sh.red[0][tid], sh.red[1][tid]), max(sh.red[2][tid], sh.red[3][tid]));
    const TileScale ts = tile_scale<POW2>(a);
    sh.div[tid] = ts.div;
    sh.mul[tid] = ts.mul;
    sh.nege[tid] = ts.neg_e;
    sh.slow[tid] = ts.slow;
    if (ts.slow) sh.anyslow = 1;
    if (f0 + tid < cols) scales[(int64_t)(f0 + tid) * ntb + tb] = ts.s;
  }
  __syncthreads();

  // encode: feature 8*c8 + j, tokens 4q..4q+3 -> one word at sh.tile[f][4q].
  // The thread's 8 features' scale state comes in as whole 16-byte LDS
  // reads; the scaling of x by 2^64 for a tiny-amax feature is taken only
  // when the block has one (a workgroup-uniform branch), so the common case
  // is the bare Markstein quotient.
  auto word_of = [&](int p, int j) {
    return (j >> 1) == 0 ? v[p].x : (j >> 1) == 1 ? v[p].y : (j >> 1) == 2 ? v[p].z : v[p].w;
  };
  auto put = [&](int j, uint32_t w) {
    const int f = 8 * c8 + j;
    *reinterpret_cast<uint32_t*>(&sh.tile[f * kTokenRowBytes + 4 * ((q + 8 * c8) & 31)]) = w;
  };
  if constexpr (POW2) {
    const int4 n0 = *reinterpret_cast<const int4*>(&sh.nege[8 * c8]);
    const int4 n1 = *reinterpret_cast<const int4*>(&sh.nege[8 * c8 + 4]);
    const int ne[8] = {n0.x, n0.y, n0.z, n0.w, n1.x, n1.y, n1.z, n1.w};
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float e[4];
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        const uint32_t word = word_of(p, j);
        e[p] = __builtin_ldexpf((j & 1) ? bf16_hi(word) : bf16_lo(word), ne[j]);
      }
      put(j, pack4_e4m3(e[0], e[1], e[2], e[3]));
    }
  } else {
    const float4 d0 = *reinterpret_cast<const float4*>(&sh.div[8 * c8]);
    const float4 d1 = *reinterpret_cast<const float4*>(&sh.div[8 * c8 + 4]);
    const float4 r0 = *reinterpret_cast<const float4*>(&sh.mul[8 * c8]);
    const float4 r1 = *reinterpret_cast<const float4*>(&sh.mul[8 * c8 + 4]);
    const float dv[8] = {d0.x, d0.y, d0.z, d0.w, d1.x, d1.y, d1.z, d1.w};
    const float ml[8] = {r0.x, r0.y, r0.z, r0.w, r1.x, r1.y, r1.z, r1.w};
    if (sh.anyslow == 0) {  // (workgroup-uniform)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        float e[4];
#pragma unroll
        for (int p = 0; p < 4; ++p) {
          const uint32_t word = word_of(p, j);
          const float xv = (j & 1) ? bf16_hi(word) : bf16_lo(word);
          const float q0 = xv * ml[j];
          const float er = __builtin_fmaf(-q0, dv[j], xv);
          e[p] = __builtin_copysignf(__builtin_fmaf(er, ml[j], q0), xv);
        }
        put(j, pack4_e4m3(e[0], e[1], e[2], e[3]));
      }
    } else {
      // a tiny-amax feature scales its x by 2^64 (its divisor already is)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        TileScale ts;
        ts.div = dv[j];
        ts.mul = ml[j];
        ts.neg_e = 0;
        ts.slow = sh.slow[8 * c8 + j] != 0;
        ts.xscale = ts.slow ? 0x1p64f : 1.0f;
        float e[4];
#pragma unroll
        for (int p = 0; p < 4; ++p) {
          const uint32_t word = word_of(p, j);
          e[p] = quotient_free((j & 1) ? bf16_hi(word) : bf16_lo(word), ts);
        }
        put(j, pack4_e4m3(e[0], e[1], e[2], e[3]));
        // (one feature at a time: this rare path keeps the fast path's
        // register budget)
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  }
  __syncthreads();

  // store: 8 consecutive lanes write one feature row's 128 token bytes, so
  // each store instruction covers 8 whole 128-byte row segments (spreading a
  // row over lanes of different instructions measured 25% slower)
#pragma unroll
  for (int it = 0; it < 2; ++it) {
    const int f = (tid >> 3) + 32 * it;
    const int ch = tid & 7;
    const uint4 w = *reinterpret_cast<const uint4*>(&sh.tile[f * kTokenRowBytes + 16 * ((ch + 2 * (f >> 3)) & 7)]);
    uint8_t* dst = codes + (int64_t)(f0 + f) * ldc + t0 + 16 * ch;
    if (full) {
      st_stream16(dst, w);
    } else if (f0 + f < cols) {
      const int nvalid = rows - (t0 + 16 * ch);
      const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        if (i < nvalid) dst[i] = (uint8_t)((ww[i >> 2] >> (8 * (i & 3))) & 0xFF);
      }
    }
  }
}

}  // namespace fp8q
