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

// Eight BF16 values; those past `left` (which may be <= 0) are +0.
__device__ __forceinline__ uint4 ld_bf16x8(const uint16_t* p, int left, bool aligned) {
  if (left < 8) return load8_masked(p, left);
  if (aligned) return ld_stream16(p);
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
__device__ __forceinline__ uint2 ld_codes8(const uint8_t* p, int left, bool aligned) {
  if (left >= 8) {
    if (aligned) {
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

// Eight float32 or BF16 values of a row as float32.
struct F8 {
  float v[8];
};

template <bool F32>
__device__ __forceinline__ F8 ld_float8(const void* base, int64_t at, int left, bool aligned) {
  F8 r;
  if constexpr (F32) {
    const float* p = static_cast<const float*>(base) + at;
    if (left >= 8) {
      uint4 a, b;
      if (aligned) {
        a = ld_stream16(p);
        b = ld_stream16(p + 4);
      } else {
        a = ld_bf16x8(reinterpret_cast<const uint16_t*>(p), 8, false);
        b = ld_bf16x8(reinterpret_cast<const uint16_t*>(p + 4), 8, false);
      }
      const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
      for (int i = 0; i < 8; ++i) r.v[i] = __uint_as_float(w[i]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) r.v[i] = i < left ? p[i] : 0.0f;
    }
  } else {
    const uint4 a = ld_bf16x8(static_cast<const uint16_t*>(base) + at, left, aligned);
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      r.v[2 * i] = bf16_lo(w[i]);
      r.v[2 * i + 1] = bf16_hi(w[i]);
    }
  }
  return r;
}

__device__ __forceinline__ void st_float8(float* p, const F8& f, int left, bool aligned) {
  if (left >= 8) {
    const uint4 a = make_uint4(__float_as_uint(f.v[0]), __float_as_uint(f.v[1]), __float_as_uint(f.v[2]), __float_as_uint(f.v[3]));
    const uint4 b = make_uint4(__float_as_uint(f.v[4]), __float_as_uint(f.v[5]), __float_as_uint(f.v[6]), __float_as_uint(f.v[7]));
    st_bf16x8(reinterpret_cast<uint16_t*>(p), a, 8, aligned);
    st_bf16x8(reinterpret_cast<uint16_t*>(p + 4), b, 8, aligned);
    return;
  }
#pragma unroll
  for (int i = 0; i < 7; ++i)
    if (i < left) p[i] = f.v[i];
}

// Eight float32 values -> BF16, nearest even by the hardware convert
// (infinities and NaN stay what they are).
typedef __bf16 c8_v2bf __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint4 pack_bf16x8(const F8& f) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = __builtin_bit_cast(uint32_t, c8_v2bf{(__bf16)f.v[2 * i], (__bf16)f.v[2 * i + 1]});
  return make_uint4(w[0], w[1], w[2], w[3]);
}

}  // namespace fp8q
