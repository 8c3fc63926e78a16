// What the RMS norm's kernels share (gfx950): the products of a normalised
// row, rounded the same way everywhere, and sums over a wave.
//
// With r = 1 / sqrt(mean(h^2) + eps), the sum in 64 bits and r rounded once to
// float32, a row's output is y = bf16(fl(fl(h r) w)).  The sum's order depends on
// the row's width alone, not on the number of rows, by which its split over
// threads goes (split_sum, norm_bwd_shape): so r, and with it every bit of y, of
// its codes and of its scales, is that of the row alone.  (In another order a
// 64-bit sum differs by some 2^-50, which moves r by a step seldom, but not
// never; a float32 sum moves r now and then, and with it a tile's scale by a
// step of BF16.)  The 64-bit steps are two of some twenty instructions a value.
#pragma once

#include "chunk8.h"

namespace fp8q {

// The last s of eight values that a chunk at a row's end was loaded too early:
// a row's last chunk is read as its last eight columns and moved down once it
// is used, so that it costs no branch and no load after another.
__device__ __forceinline__ Raw<false, 8> moved_down(Raw<false, 8> r, int s) {
  if (s & 4) r = Raw<false, 8>{{r.w[2], r.w[3], 0, 0}};
  if (s & 2) r = Raw<false, 8>{{r.w[1], r.w[2], r.w[3], 0}};
  if (s & 1) {
    r = Raw<false, 8>{{__builtin_amdgcn_alignbit(r.w[1], r.w[0], 16), __builtin_amdgcn_alignbit(r.w[2], r.w[1], 16),
                       __builtin_amdgcn_alignbit(r.w[3], r.w[2], 16), r.w[3] >> 16}};
  }
  return r;
}
__device__ __forceinline__ Raw<true, 8> moved_down(Raw<true, 8> r, int s) {
  if (s & 4) r = Raw<true, 8>{{r.w[4], r.w[5], r.w[6], r.w[7], 0, 0, 0, 0}};
  if (s & 2) r = Raw<true, 8>{{r.w[2], r.w[3], r.w[4], r.w[5], r.w[6], r.w[7], 0, 0}};
  if (s & 1) r = Raw<true, 8>{{r.w[1], r.w[2], r.w[3], r.w[4], r.w[5], r.w[6], r.w[7], 0}};
  return r;
}

// The first `left` (1 .. 7) of eight values in three stores at most.
__device__ __forceinline__ void st_part(uint16_t* p, Raw<false, 8> r, int left) {
  if (left & 4) {
    *reinterpret_cast<Any8*>(p) = Any8{{r.w[0], r.w[1]}};
    r = Raw<false, 8>{{r.w[2], r.w[3], 0, 0}};
    p += 4;
  }
  if (left & 2) {
    p[0] = (uint16_t)r.w[0];
    p[1] = (uint16_t)(r.w[0] >> 16);
    r.w[0] = r.w[1];
    p += 2;
  }
  if (left & 1) p[0] = (uint16_t)r.w[0];
}
__device__ __forceinline__ void st_part(float* p, Raw<true, 8> r, int left) {
  uint32_t* q = reinterpret_cast<uint32_t*>(p);
  if (left & 4) {
    *reinterpret_cast<Any16*>(q) = Any16{{r.w[0], r.w[1], r.w[2], r.w[3]}};
    r = Raw<true, 8>{{r.w[4], r.w[5], r.w[6], 0, 0, 0, 0, 0}};
    q += 4;
  }
  if (left & 2) {
    q[0] = r.w[0];
    q[1] = r.w[1];
    r.w[0] = r.w[2];
    q += 2;
  }
  if (left & 1) q[0] = r.w[0];
}

// One row of a tensor.  Aligned rows (VEC: 16-byte boundaries, whole chunks)
// go through a buffer resource of the row's bytes: past its end loads give 0
// and stores do nothing, without a branch, and a chunk of every row has the
// same offset.  Others are loaded by unaligned vector loads (see moved_down) and
// settled before use.  A row that is not `on` has no bytes, or if not VEC is
// one that may be read; KEEP: plain loads instead of streaming ones.
template <bool F32, bool VEC, bool KEEP = true>
struct Row {
  static constexpr int kBytes = F32 ? 4 : 2;
  __amdgpu_buffer_rsrc_t buf;
  uint8_t* base;
  int n;
  __device__ __forceinline__ Row(const void* p, int64_t at, int columns, bool on = true) {
    base = static_cast<uint8_t*>(const_cast<void*>(p)) + at * kBytes;
    n = columns;
    if constexpr (VEC) buf = __builtin_amdgcn_make_buffer_rsrc(base, 0, on ? n * kBytes : 0, 0x00020000);
  }
  __device__ __forceinline__ Raw<F32, 8> load(int col) const {
    Raw<F32, 8> r;
    if constexpr (VEC) {
#pragma unroll
      for (int i = 0; i < Raw<F32, 8>::N; i += 4) {
        const u32x4 v = __builtin_amdgcn_raw_buffer_load_b128(buf, col * kBytes + 4 * i, 0, KEEP ? 0 : 2);
        r.w[i] = v[0];
        r.w[i + 1] = v[1];
        r.w[i + 2] = v[2];
        r.w[i + 3] = v[3];
      }
      return r;
    } else {
      if (n < 8) return ld_raw<F32, 8, true>(base, 0, col == 0 ? n : 0, false);
      return ld_raw<F32, 8, true>(base, min(col, n - 8), 8, false);
    }
  }
  __device__ __forceinline__ void settle(int col, Raw<F32, 8>& r) const {
    if constexpr (!VEC) {
      const int early = col - (n - 8);
      if (n >= 8 && early > 0) r = early < 8 ? moved_down(r, early) : Raw<F32, 8>{};
    }
  }
  __device__ __forceinline__ Raw<F32, 8> settled(int col) const {
    auto r = load(col);
    settle(col, r);
    return r;
  }
  __device__ __forceinline__ void store(int col, const Raw<F32, 8>& r) const {
    if constexpr (VEC) {
#pragma unroll
      for (int i = 0; i < Raw<F32, 8>::N; i += 4)
        __builtin_amdgcn_raw_buffer_store_b128(u32x4{r.w[i], r.w[i + 1], r.w[i + 2], r.w[i + 3]}, buf, col * kBytes + 4 * i, 0, 2);
    } else {
      using T = std::conditional_t<F32, float, uint16_t>;
      T* p = reinterpret_cast<T*>(base) + col;
      if (n - col >= 8) {
#pragma unroll
        for (int i = 0; i < Raw<F32, 8>::N; i += 4)
          *reinterpret_cast<Any16*>(reinterpret_cast<uint32_t*>(p) + i) = Any16{{r.w[i], r.w[i + 1], r.w[i + 2], r.w[i + 3]}};
      } else if (n > col) {
        st_part(p, r, n - col);
      }
    }
  }
};

// Eight columns of the gain, float32 (lo, hi) or BF16 (lo), as they come.  The
// type is a matter of uniform branches, which cost less than twice the kernels.
struct Gain8 {
  uint4 lo, hi;
};
template <bool VEC>
__device__ __forceinline__ Gain8 ld_gain8(const void* p, bool f32, int col, int n) {
  Gain8 g;
  g.hi = make_uint4(0, 0, 0, 0);
  if (f32) {
    const auto r = Row<true, VEC>(p, 0, n).load(col);
    g.lo = make_uint4(r.w[0], r.w[1], r.w[2], r.w[3]);
    g.hi = make_uint4(r.w[4], r.w[5], r.w[6], r.w[7]);
  } else {
    const auto r = Row<false, VEC>(p, 0, n).load(col);
    g.lo = make_uint4(r.w[0], r.w[1], r.w[2], r.w[3]);
  }
  return g;
}
template <bool VEC>
__device__ __forceinline__ void widen_gain8(const Gain8& g, bool f32, int col, int n, float* v) {
  if (f32) {
    Raw<true, 8> r{{g.lo.x, g.lo.y, g.lo.z, g.lo.w, g.hi.x, g.hi.y, g.hi.z, g.hi.w}};
    Row<true, VEC>(nullptr, 0, n).settle(col, r);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = r.at(i);
  } else {
    Raw<false, 8> r{{g.lo.x, g.lo.y, g.lo.z, g.lo.w}};
    Row<false, VEC>(nullptr, 0, n).settle(col, r);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = r.at(i);
  }
}

// y before its rounding to BF16.
__device__ __forceinline__ float normalised(float h, float r, float w) { return (h * r) * w; }

// Sum over the wave, the same in every lane: within rows of 16 lanes by DPP
// (as dpp_max16), then the four rows' sums.  All 64 lanes must be active.
__device__ __forceinline__ double wave_sum(double v) {
  v += dpp_double<0xB1>(v);
  v += dpp_double<0x4E>(v);
  v += dpp_double<0x141>(v);
  v += dpp_double<0x140>(v);
  return (lane_double(v, 0) + lane_double(v, 16)) + (lane_double(v, 32) + lane_double(v, 48));
}

// Sum over the workgroup, the same in every thread; `part` holds one value a
// wave.  All threads take part, and none may write `part` again before the
// next barrier.
__device__ __forceinline__ double block_sum(double v, double* part) {
  v = wave_sum(v);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
  __syncthreads();
  double t = part[0];
  for (int i = 1; i < (int)blockDim.x >> 6; ++i) t += part[i];
  return t;
}

// Where few rows go to twice the threads of many, each with half the chunks, a
// thread's place in the row: of 32 lanes the first 16 have a tile of the row's
// first half of threads, the others the one that many rows give the same
// threads.  So the two halves of such a thread's sum are 16 lanes apart.  Of 192
// threads (NormShape) the last wave's have no other half: 64 in their order.
template <int CH>
__device__ __forceinline__ bool three_waves() {
  return CH == 1 && blockDim.x == 192;
}
template <int CH>
__device__ __forceinline__ int split_thread() {
  const int tid = threadIdx.x;
  if (three_waves<CH>() && tid >= 128) return tid - 64;
  return (tid >> 5) * 16 + (tid & 15) + (tid & 16 ? three_waves<CH>() ? 128 : (int)blockDim.x >> 1 : 0);
}
// block_sum of what those threads would have of many rows, bit for bit: first
// the two halves, then a wave's two tiles, then two waves, which are one there.
template <int CH>
__device__ __forceinline__ double split_sum(double v, double* part) {
  const bool whole = three_waves<CH>() && threadIdx.x >= 128;
  if (!whole) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    // (of x and x: the even one of two times 16 lanes in both, and the odd one in both)
    const auto lo = __builtin_amdgcn_permlane16_swap((uint32_t)u, (uint32_t)u, false, false);
    const auto hi = __builtin_amdgcn_permlane16_swap((uint32_t)(u >> 32), (uint32_t)(u >> 32), false, false);
    v = __builtin_bit_cast(double, (uint64_t)hi[0] << 32 | lo[0]) + __builtin_bit_cast(double, (uint64_t)hi[1] << 32 | lo[1]);
  }
  v += dpp_double<0xB1>(v);
  v += dpp_double<0x4E>(v);
  v += dpp_double<0x141>(v);
  v += dpp_double<0x140>(v);
  const double s = whole ? (lane_double(v, 0) + lane_double(v, 16)) + (lane_double(v, 32) + lane_double(v, 48)) : lane_double(v, 0) + lane_double(v, 32);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = s;
  __syncthreads();
  double t = part[0] + part[1];
  if (three_waves<CH>()) return t + part[2];
  for (int i = 2; i < (int)blockDim.x >> 6; i += 2) t += part[i] + part[i + 1];
  return t;
}

// 1 / sqrt(sum / n + eps), rounded once: the hardware's estimate and two
// Newton steps in 64 bits, a tenth of the instructions of a division and a root
// (every wave of a row works it out).  The limits keep the steps finite; beyond
// them the result is 0 or infinite in float32 either way, and a NaN stays one.
__device__ __forceinline__ float reciprocal_rms(double sum, double inv_n, double eps) {
  double m = __builtin_fma(sum, inv_n, eps);
  m = m < 0x1p-1000 ? 0x1p-1000 : m > 0x1p1000 ? 0x1p1000 : m;
  double y = __builtin_amdgcn_rsq(m);
#pragma unroll
  for (int i = 0; i < 2; ++i) y = __builtin_fma(0.5 * y, __builtin_fma(-m * y, y, 1.0), y);
  return (float)y;
}

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
// Chunks of eight BF16 values, each quantized with the 16-lane DPP row that
// holds its 1x128 tile; every lane of the wave takes part.  The scales of a
// DPP row's CH tiles are worked out once, by lane u for tile u, as in the row
// quantizer.
template <bool POW2, bool VEC, int CH>
__device__ __forceinline__ void encode_chunks(const uint4 (&d)[CH], uint32_t mine, int64_t row, int col0, int step, int n, uint8_t* codes,
                                              int64_t ldc, float* scales) {
  static_assert(CH >= 1 && CH <= 4, "tiles u = 0 .. CH - 1 of a DPP row");
  const int sub = threadIdx.x & 15, nb = (n + 127) >> 7;
  const TileScale tm = tile_scale<POW2>(mine);
  {
    const int col = col0 - 8 * sub + sub * step;  // first column of tile `sub`
    if (sub < CH && col < n) scales[row * nb + (col >> 7)] = tm.s;
  }
  uint8_t* out = codes + row * ldc;
  __amdgpu_buffer_rsrc_t buf;
  if constexpr (VEC) buf = __builtin_amdgcn_make_buffer_rsrc(out, 0, n, 0x00020000);
  auto store = [&](int u, const TileScale& ts, auto enc) {
    const uint2 c = enc(d[u], ts);
    const int col = col0 + u * step, left = n - col;
    if constexpr (VEC) {
      __builtin_amdgcn_raw_buffer_store_b64(u32x2{c.x, c.y}, buf, col, 0, 2);
    } else if (left >= 8) {
      *reinterpret_cast<Any8*>(out + col) = Any8{{c.x, c.y}};
    } else if (left > 0) {
      store8_masked(out + col, c, left);
    }
  };
  auto all = [&](auto enc) {
    store(0, row_tile_scale<POW2, 0>(tm), enc);
    if constexpr (CH > 1) store(1, row_tile_scale<POW2, 1>(tm), enc);
    if constexpr (CH > 2) store(2, row_tile_scale<POW2, 2>(tm), enc);
    if constexpr (CH > 3) store(3, row_tile_scale<POW2, 3>(tm), enc);
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
template <bool VEC, int CH>
__device__ __forceinline__ void quantize_chunks(const uint4 (&d)[CH], bool pow2, int64_t row, int col0, int step, int n, uint8_t* codes,
                                                int64_t ldc, float* scales) {
  uint32_t mine = 0;  // lane u: tile u's max-abs
#pragma unroll
  for (int u = 0; u < CH; ++u) {
    const uint32_t amax = dpp_max16(absmax8(d[u]));
    mine = CH == 1 || (threadIdx.x & 15) == u ? amax : mine;
  }
  if (pow2) {
    encode_chunks<true, VEC, CH>(d, mine, row, col0, step, n, codes, ldc, scales);
  } else {
    encode_chunks<false, VEC, CH>(d, mine, row, col0, step, n, codes, ldc, scales);
  }
}

}  // namespace fp8q
