// Chunks of eight consecutive elements of a row: loads and stores for any
// row stride (gfx950).  A chunk whose row starts off a 16-byte boundary is
// still moved by one instruction (global memory takes vector accesses of any
// alignment here), only a chunk that crosses the row's end goes element by
// element: an odd stride costs a split cache line now and then instead of
// eight accesses a chunk.
#pragma once

#include "quant_common.h"

namespace fp8q {

struct __attribute__((packed, aligned(2))) Any16 {
  uint32_t w[4];
};
struct __attribute__((packed, aligned(1))) Any8 {
  uint32_t w[2];
};

// Eight BF16 values; those past `left` (which may be <= 0) are +0.  KEEP: a
// plain load instead of a streaming one (an unaligned load always is plain).
template <bool KEEP = false>
__device__ __forceinline__ uint4 ld_bf16x8(const uint16_t* p, int left, bool aligned) {
  if (left < 8) return load8_masked(p, left);
  if (aligned) return KEEP ? *reinterpret_cast<const uint4*>(p) : ld_stream16(p);
  const Any16 v = *reinterpret_cast<const Any16*>(p);
  return make_uint4(v.w[0], v.w[1], v.w[2], v.w[3]);
}

__device__ __forceinline__ void st_bf16x8(uint16_t* p, uint4 c, int left, bool aligned) {
  if (left >= 8) {
    if (aligned) {
      st_stream16(p, c);
    } else {
      *reinterpret_cast<Any16*>(p) = Any16{{c.x, c.y, c.z, c.w}};
    }
    return;
  }
  const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
  for (int i = 0; i < 7; ++i)
    if (i < left) p[i] = (uint16_t)(w[i >> 1] >> (16 * (i & 1)));
}

// Eight codes.
template <bool KEEP = false>
__device__ __forceinline__ uint2 ld_codes8(const uint8_t* p, int left, bool aligned) {
  if (left >= 8) {
    if (aligned) {
      if (KEEP) return *reinterpret_cast<const uint2*>(p);
      const u32x2 v = __builtin_nontemporal_load(reinterpret_cast<const u32x2*>(p));
      return make_uint2(v[0], v[1]);
    }
    const Any8 v = *reinterpret_cast<const Any8*>(p);
    return make_uint2(v.w[0], v.w[1]);
  }
  uint32_t w[2] = {0, 0};
#pragma unroll
  for (int i = 0; i < 7; ++i)
    if (i < left) w[i >> 2] |= (uint32_t)p[i] << (8 * (i & 3));
  return make_uint2(w[0], w[1]);
}

__device__ __forceinline__ void st_codes8(uint8_t* p, uint2 c, int left, bool aligned) {
  if (left < 8) {
    store8_masked(p, c, left);
  } else if (aligned) {
    st_stream8(p, c);
  } else {
    *reinterpret_cast<Any8*>(p) = Any8{{c.x, c.y}};
  }
}

// W consecutive float32 or BF16 values as they come: kept in flight in this
// form (half the registers for BF16) and widened where they are used.
template <bool F32, int W>
struct Raw {
  static constexpr int N = F32 ? W : W / 2;
  uint32_t w[N];
  __device__ __forceinline__ float at(int i) const {
    if constexpr (F32) {
      return __uint_as_float(w[i]);
    } else {
      return i & 1 ? bf16_hi(w[i >> 1]) : bf16_lo(w[i >> 1]);
    }
  }
};

// Those past `left` are +0.  W = 8, or 4: the columns of a lane where the
// output is float32, so that the 64 lanes of a store write one run of 1 KiB
// (eight columns a lane make every store instruction skip 16 bytes after each
// 16: partial lines, which go to memory at half the rate).
template <bool F32, int W, bool KEEP = false>
__device__ __forceinline__ Raw<F32, W> ld_raw(const void* base, int64_t at, int left, bool aligned) {
  Raw<F32, W> r;
  if (left >= W) {
    const uint16_t* p = static_cast<const uint16_t*>(base) + at * (F32 ? 2 : 1);
    if constexpr (Raw<F32, W>::N == 2) {
      const uint2 c = ld_codes8<KEEP>(reinterpret_cast<const uint8_t*>(p), 8, aligned);
      r.w[0] = c.x;
      r.w[1] = c.y;
    } else {
#pragma unroll
      for (int i = 0; i < Raw<F32, W>::N; i += 4) {
        const uint4 c = ld_bf16x8<KEEP>(p + 2 * i, 8, aligned);
        r.w[i] = c.x;
        r.w[i + 1] = c.y;
        r.w[i + 2] = c.z;
        r.w[i + 3] = c.w;
      }
    }
    return r;
  }
#pragma unroll
  for (int i = 0; i < Raw<F32, W>::N; ++i) r.w[i] = 0;
#pragma unroll
  for (int i = 0; i < W - 1; ++i) {
    if (i < left) {
      if constexpr (F32) {
        r.w[i] = static_cast<const uint32_t*>(base)[at + i];
      } else {
        r.w[i >> 1] |= (uint32_t) static_cast<const uint16_t*>(base)[at + i] << (16 * (i & 1));
      }
    }
  }
  return r;
}

__device__ __forceinline__ void st_float4(float* p, const float* f, int left, bool aligned) {
  if (left >= 4) {
    const uint4 a = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
    st_bf16x8(reinterpret_cast<uint16_t*>(p), a, 8, aligned);
    return;
  }
#pragma unroll
  for (int i = 0; i < 3; ++i)
    if (i < left) p[i] = f[i];
}

// Eight float32 values -> BF16, nearest even by the hardware convert
// (infinities and NaN stay what they are).
typedef __bf16 c8_v2bf __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint4 pack_bf16x8(const float* f) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = __builtin_bit_cast(uint32_t, c8_v2bf{(__bf16)f[2 * i], (__bf16)f[2 * i + 1]});
  return make_uint4(w[0], w[1], w[2], w[3]);
}

}  // namespace fp8q
