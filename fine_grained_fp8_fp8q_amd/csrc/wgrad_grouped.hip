// Weight gradients of every expert of one device (jp-study.kr doc 258368 ¶3:
// Wgrad runs in FP8), gfx950:
//   dW[g,n,c] = sum_{b in group g} sd[n,b] sx[c,b] sum_{t in b} dY[t,n] X[t,c]
// The arithmetic of one output is that of the plain weight gradient
// (gemm.hip) step for step: E4M3 bytes widened to BF16 in registers, four
// chained BF16 MFMAs over a 128-token block, one float32 fold with the
// block's two scales; the FP8-unit and power-of-two forms likewise.
//
// What differs is the shape of the work.  An expert sees a few hundred
// tokens, so a tile's K loop is a few blocks long and the float32 output is
// most of the bytes: 16 experts of 4096 x 7168 write 1.88 GB, against 46 MB
// of operands at 4096 rows.  Measured on MI355X at that size (2.4 blocks a
// tile on average, groups from 0 to 11):
//   - outputs that go out as each lane holds them, 64 bytes of a row at a
//     time through the caches: 664 us; 16 rows at a time through LDS, so that
//     a store instruction writes whole rows of the wave's tile, and
//     non-temporal, so that the outputs do not push the operands out of the
//     L2: 484 us;
//   - the tiles of a gradient row by row instead of column by column: 446 us
//     (writes alone, every group empty: 332 us against 385);
//   - groups interleaved (tile rows of all groups in turn, or panels of 2 to
//     16 rows, or the fullest group with the emptiest), a persistent grid with
//     the next tile's loads under the last block of this one, both blocks of a
//     short loop loaded at once: no faster (452-482, 451-459, 453-517, 433
//     against 433 us), not kept.  (All on 128 x 128 tiles with the folded
//     form: a persistent grid of 256 x 256 tiles was not tried.)
// What bounds it now: the writes take 332 us alone and the products 326 us
// alone; together the power and the memory they share give 433-459.
#include <type_traits>

#include "fp8q_internal.h"
#include "quant_common.h"

namespace fp8q {
namespace {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef v4f v4f_any __attribute__((aligned(4)));  // on any element's boundary
typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) void* lds_void_ptr;

constexpr int BK = 128;
constexpr int kRsrcFlags = 0x00020000;

// WM x WN waves of 16 FM x 16 JN outputs.  A stage holds one K block: TM rows
// of dY^T, then TN of X^T, 128 B each.
template <int WM, int WN, int FM, int JN>
struct Shape {
  static constexpr int kWM = WM, kFM = FM, kJN = JN, kTM = 16 * FM * WM, kTN = 16 * JN * WN;
  static constexpr int kThreads = 64 * WM * WN, kE = kTM + kTN;  // scale entries: one per stage row
  static constexpr int kStage = kE * BK;
  static constexpr int kScaleHalf = 4 * kE * 4;  // scales of four K blocks, [block][entry]
  static constexpr int kLds = 2 * kStage + 2 * kScaleHalf;
  static constexpr int kLoads = kTM / (8 * WM * WN);  // load instructions of a wave per K block and operand
  static constexpr int kScales = 4 * kE / kThreads;   // scales of four K blocks that a thread brings
  static_assert(kTM == kTN && kTM % 64 == 0 && kLoads * 8 * WM * WN == kTM && kLoads <= 4 && kScales * kThreads == 4 * kE,
                "whole waves for each operand");
};
using Large = Shape<4, 2, 4, 8>;   // 256 x 256: one workgroup per compute unit
using Medium = Shape<2, 2, 4, 4>;  // 128 x 128: two
using Small = Shape<2, 2, 2, 2>;   // 64 x 64: four

struct WgArgs {
  const uint8_t* a;   // dY^T codes [rows, k]
  const float* sa;    // [rows, k/128]
  const uint8_t* w;   // X^T codes [n, k]
  const float* sw;    // [n, k/128]
  const int32_t* offsets;
  float* c;
  int64_t ldc;
  int rows, n, k;
  int tiles_m, tiles_n;
  int region_m, region_n, xcds_n;  // tiles of an XCD's region, XCDs along n
};

// 16-byte chunk swizzle of a 128-byte LDS row (16 rows reading one logical
// chunk cover 16 chunk slots across a pair of rows).
__device__ __forceinline__ int swz(int row) { return (row & 7) ^ ((row >> 3) & 1); }

// Eight E4M3 codes -> eight BF16 values times a power of two s, exactly.
__device__ __forceinline__ v8bf widen(int lo, int hi, float s) {
  const v2bf a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((unsigned)lo, s, false);
  const v2bf b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((unsigned)lo, s, true);
  const v2bf c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((unsigned)hi, s, false);
  const v2bf d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((unsigned)hi, s, true);
  return v8bf{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// ---- K loop, two stages: block kb + 1 streams in while kb is multiplied.
// Before the barrier every wave has its loads of block kb in LDS, its LDS
// writes done, and has consumed its reads of the stage that is refilled.
// Scales of the next group of four blocks are fetched at the third block of
// a group and written at its fourth.  The stages and the scale buffer are
// __restrict__ parameters of the function that runs the whole loop: only
// that tells the compiler's tracking of loads in flight into LDS that reads
// of the current stage and of the scales need not wait for the refill.
template <class Issue, class Fetch, class Put, class Compute>
__device__ __forceinline__ void k_step(int kb, int nkb, const uint8_t* __restrict__ cur, uint8_t* __restrict__ refill,
                                       uint8_t* __restrict__ scl, Issue& issue, Fetch& fetch, Put& put,
                                       Compute& compute) {
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
  if (kb + 1 < nkb) {
    if ((kb & 3) == 3) {
      put((kb >> 2) + 1, scl);
    } else if ((kb & 3) == 2) {
      fetch((kb >> 2) + 1);
    }
    issue(kb + 1, refill);
  }
  compute(cur, scl, kb);
}

template <class Issue, class Fetch, class Put, class Compute>
__device__ __forceinline__ void k_loop(int nkb, uint8_t* __restrict__ s0, uint8_t* __restrict__ s1,
                                       uint8_t* __restrict__ scl, Issue& issue, Fetch& fetch, Put& put,
                                       Compute& compute) {
  fetch(0);
  issue(0, s0);
  put(0, scl);
  int kb = 0;
  for (; kb + 2 <= nkb; kb += 2) {
    k_step(kb, nkb, s0, s1, scl, issue, fetch, put, compute);
    k_step(kb + 1, nkb, s1, s0, scl, issue, fetch, put, compute);
  }
  if (kb < nkb) k_step(kb, nkb, s0, s1, scl, issue, fetch, put, compute);
}

// ACC as FP8Q_ACC_*: 0 float32 grade, 1 FP8 matrix core, 2 hardware scales,
// 3 float32 grade with power-of-two scales.
template <class S, int ACC>
__global__ __launch_bounds__(S::kThreads, 2) void wgrad_grouped_kernel(WgArgs g) {
  constexpr int TM = S::kTM, TN = S::kTN, E = S::kE, WM = S::kWM, FM = S::kFM, JN = S::kJN, LI = S::kLoads, SB = S::kScales;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[S::kLds];

  // Grid = groups x 8 XCDs x the tiles of an XCD's region of a gradient (row
  // by row, so that the workgroups that run together write neighbouring
  // pieces of the same rows); workgroup i runs on XCD i % 8.
  const int per = 8 * g.region_m * g.region_n;
  const int gi = blockIdx.x / per;
  const int in = blockIdx.x - gi * per;
  const int xcd = in & 7, idx = in >> 3;
  const int rm = idx / g.region_n;
  const int tm = xcd / g.xcds_n * g.region_m + rm;
  const int tn = xcd % g.xcds_n * g.region_n + idx - rm * g.region_n;
  if (tm >= g.tiles_m || tn >= g.tiles_n) return;  // (regions past the edge)
  const int m0 = tm * TM, n0 = tn * TN;
  const int mrows = min(TM, g.rows - m0), nrows = min(TN, g.n - n0);
  // offsets outside [0, k], decreasing or off the 128-token blocks are
  // clamped and rounded down: every access stays inside the operands
  const int kb0 = min(max(g.offsets[gi], 0), g.k) / BK;
  const int nkb = max(min(max(g.offsets[gi + 1], 0), g.k) / BK - kb0, 0);

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave & (WM - 1), wn = wave / WM;
  const int r16 = lane & 15, c0 = 2 * (lane >> 4);
  const int arow0 = wm * 16 * FM + r16, wrow0 = wn * 16 * JN + r16;
  const int asw = swz(arow0), wsw = swz(wrow0);  // the same for rows + 16 f

  // ---- loads.  One wave instruction moves 8 rows x 128 B of codes into LDS;
  // rows past the operand's last read as zero (the buffer's range check,
  // which counts dwords; 256 rows of fewer than 2^24 tokens stay below 2^32).
  const uint32_t rowb = (uint32_t)g.k, kofs0 = (uint32_t)kb0 * BK;
  const __amdgpu_buffer_rsrc_t a_rsrc = __builtin_amdgcn_make_buffer_rsrc(
      (void*)(g.a + (size_t)m0 * rowb + kofs0), 0, (int)((uint32_t)mrows * rowb - kofs0), kRsrcFlags);
  const __amdgpu_buffer_rsrc_t w_rsrc = __builtin_amdgcn_make_buffer_rsrc(
      (void*)(g.w + (size_t)n0 * rowb + kofs0), 0, (int)((uint32_t)nrows * rowb - kofs0), kRsrcFlags);
  uint32_t r_off[4];
#pragma unroll
  for (int i = 0; i < LI; ++i) {
    const int row = (wave * LI + i) * 8 + (lane >> 3);
    r_off[i] = (uint32_t)row * rowb + 16u * (uint32_t)((lane & 7) ^ swz(row));
  }
  auto issue = [&](int kb, uint8_t* st) {
    const uint32_t kofs = (uint32_t)kb * BK;
#pragma unroll
    for (int i = 0; i < LI; ++i) {
      __builtin_amdgcn_raw_ptr_buffer_load_lds(a_rsrc, (lds_void_ptr)(st + (wave * LI + i) * 1024), 16, r_off[i], kofs, 0, 0);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(w_rsrc, (lds_void_ptr)(st + TM * BK + (wave * LI + i) * 1024), 16, r_off[i], kofs, 0, 0);
    }
  };
  // Scales: of the four blocks of a group a thread brings SB for one stage
  // row (past the group's or the row's end they are other blocks' scales,
  // which no product uses, or zero) a whole group ahead, and puts them in LDS
  // [block][entry], into the half the group uses.
  const uint32_t sblk = (uint32_t)(g.k / BK) * 4u, sofs0 = (uint32_t)kb0 * 4u;
  const int ent = tid & (E - 1), sb0 = wave * 64 / E * SB;  // stage row, first of the thread's blocks
  const bool a_side = (wave * 64 & (E - 1)) < TM;           // (the same for a whole wave)
  const float* sp = a_side ? g.sa + (size_t)m0 * (sblk >> 2) : g.sw + (size_t)n0 * (sblk >> 2);
  const __amdgpu_buffer_rsrc_t s_rsrc = __builtin_amdgcn_make_buffer_rsrc(
      (void*)(sp + kb0), 0, (int)((uint32_t)(a_side ? mrows : nrows) * sblk - sofs0), kRsrcFlags);
  const uint32_t s_off = (uint32_t)(a_side ? ent : ent - TM) * sblk + 4u * (uint32_t)sb0;
  float sreg[SB];
  auto fetch_scales = [&](int grp) {
#pragma unroll
    for (int b = 0; b < SB; ++b)
      sreg[b] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(s_rsrc, s_off + 16u * (uint32_t)grp + 4u * b, 0, 0));
  };
  auto put_scales = [&](int grp, uint8_t* scl) {
    float* half = reinterpret_cast<float*>(scl + (grp & 1) * S::kScaleHalf);
#pragma unroll
    for (int b = 0; b < SB; ++b) half[(sb0 + b) * E + ent] = sreg[b];
  };

  v4f acc[FM][JN];
#pragma unroll
  for (int f = 0; f < FM; ++f)
#pragma unroll
    for (int j = 0; j < JN; ++j) acc[f][j] = v4f{0.f, 0.f, 0.f, 0.f};

  // ---- one K block of a wave: JN W fragments x FM A fragments.  The MFMA
  // computes the transposed tile, so a lane owns output row m = r16 of a
  // fragment and four consecutive columns.
  auto compute = [&](const uint8_t* st, const float* Sc) {
    const uint8_t* Ab = st + arow0 * BK;
    const uint8_t* Wb = st + TM * BK + wrow0 * BK;
    auto a_lo = [&](int f) { return *reinterpret_cast<const v4i*>(Ab + f * 2048 + 16 * (c0 ^ asw)); };
    auto a_hi = [&](int f) { return *reinterpret_cast<const v4i*>(Ab + f * 2048 + 16 * ((c0 + 1) ^ asw)); };
    auto w_lo = [&](int j) { return *reinterpret_cast<const v4i*>(Wb + j * 2048 + 16 * (c0 ^ wsw)); };
    auto w_hi = [&](int j) { return *reinterpret_cast<const v4i*>(Wb + j * 2048 + 16 * ((c0 + 1) ^ wsw)); };
    const float* Sw = Sc + TM + wn * 16 * JN;
    if constexpr (ACC == 0 || ACC == 3) {
      float sa[FM], sw[ACC == 3 ? JN : 1];
#pragma unroll
      for (int f = 0; f < FM; ++f) sa[f] = Sc[arow0 + f * 16];
      if constexpr (ACC == 3) {
#pragma unroll
        for (int j = 0; j < JN; ++j) sw[j] = Sw[j * 16 + r16];
      }
      auto part = [](const v4i& lo, const v4i& hi, int q, float s) {
        const v4i& r = q < 2 ? lo : hi;
        return widen(r[(q & 1) * 2], r[(q & 1) * 2 + 1], s);
      };
      auto sa_of = [&](int f) { return ACC == 3 ? sa[f] : 1.0f; };
      auto sw_of = [&](int j) { return ACC == 3 ? sw[ACC == 3 ? j : 0] : 1.0f; };
      v8bf af[FM][4], bf[4];
      v4i alo[FM], ahi[FM];
#pragma unroll
      for (int f = 0; f < FM; ++f) {
        alo[f] = a_lo(f);
        ahi[f] = a_hi(f);
      }
      v4i w0lo = w_lo(0), w0hi = w_hi(0), wlo = w_lo(1), whi = w_hi(1);
      v4f p[FM], swj = v4f{0.f, 0.f, 0.f, 0.f};
      auto fold = [&](int j, int f) {
#pragma unroll
        for (int v = 0; v < 4; ++v) acc[f][j][v] = __builtin_fmaf(p[f][v], sa[f] * swj[v], acc[f][j][v]);
      };
#pragma unroll
      for (int j = 0; j < JN; ++j) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          if (j == 0) {
            bf[q] = part(w0lo, w0hi, q, sw_of(0));
#pragma unroll
            for (int f = 0; f < FM; ++f) af[f][q] = part(alo[f], ahi[f], q, sa_of(f));
            __builtin_amdgcn_sched_barrier(0);
          }
#pragma unroll
          for (int f = 0; f < FM; ++f) {
            if constexpr (ACC == 3) {
              acc[f][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(bf[q], af[f][q], acc[f][j], 0, 0, 0);
            } else {
              if (q == 0 && j > 0) fold(j - 1, f);
              p[f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(bf[q], af[f][q], q == 0 ? v4f{0.f, 0.f, 0.f, 0.f} : p[f], 0, 0, 0);
            }
            __builtin_amdgcn_sched_barrier(0);
          }
          // the slot's products are issued: widen the next fragment's part
          // into it, and refill the bytes that leaves with the one after
          if (j < JN - 1) bf[q] = part(wlo, whi, q, sw_of(j < JN - 1 ? j + 1 : j));
          if (ACC == 0 && q == 0) swj = *reinterpret_cast<const v4f*>(Sw + j * 16 + 4 * (lane >> 4));
          if (q == 1 && j < JN - 2) wlo = w_lo(j + 2);
          if (q == 3 && j < JN - 2) whi = w_hi(j + 2);
          __builtin_amdgcn_sched_barrier(0);
        }
      }
      if constexpr (ACC == 0) {
#pragma unroll
        for (int f = 0; f < FM; ++f) fold(JN - 1, f);
      }
    } else {
      auto cat = [](v4i lo, v4i hi) { return v8i{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]}; };
      auto e8m0 = [](float x) { return (int)((__float_as_uint(x) >> 23) & 0xFFu); };
      v8i af[FM], wf[2];
      float sa[FM];
      int ae[FM], we[JN];
      wf[0] = cat(w_lo(0), w_hi(0));
#pragma unroll
      for (int f = 0; f < FM; ++f) {
        af[f] = cat(a_lo(f), a_hi(f));
        sa[f] = Sc[arow0 + f * 16];
        ae[f] = e8m0(sa[f]);
      }
#pragma unroll
      for (int j = 0; j < JN; ++j) we[j] = ACC == 2 ? e8m0(Sw[j * 16 + r16]) : 0;
#pragma unroll
      for (int j = 0; j < JN; ++j) {
        if (j < JN - 1) wf[(j + 1) & 1] = cat(w_lo(j + 1), w_hi(j + 1));
        if constexpr (ACC == 2) {
#pragma unroll
          for (int f = 0; f < FM; ++f)
            acc[f][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wf[j & 1], af[f], acc[f][j], 0, 0, 0, we[j], 0, ae[f]);
        } else {
          const v4f swj = *reinterpret_cast<const v4f*>(Sw + j * 16 + 4 * (lane >> 4));
          v4f p[FM];
#pragma unroll
          for (int f = 0; f < FM; ++f)
            p[f] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wf[j & 1], af[f], v4f{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 0, 0, 0);
#pragma unroll
          for (int f = 0; f < FM; ++f)
#pragma unroll
            for (int v = 0; v < 4; ++v) acc[f][j][v] = __builtin_fmaf(p[f][v], sa[f] * swj[v], acc[f][j][v]);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  };

  const int mw = mrows - wm * 16 * FM, nw = nrows - wn * 16 * JN;  // rows and columns of the wave that exist
  if (nkb > 0) {
    auto comp = [&](const uint8_t* st, const uint8_t* scl, int kb) {
      if (mw > 0 && nw > 0) compute(st, reinterpret_cast<const float*>(scl + ((kb >> 2) & 1) * S::kScaleHalf) + (kb & 3) * E);
    };
    k_loop(nkb, lds, lds + S::kStage, lds + 2 * S::kStage, issue, fetch_scales, put_scales, comp);
  }

  // ---- epilogue: 16 rows (one M fragment) at a time through the wave's own
  // part of the stages, so that a store instruction writes whole rows of
  // 64 JN bytes.  Rows on 64-byte boundaries go out non-temporal: through the
  // caches the outputs push the operands, which other tiles still read, out
  // of the L2 (16 x 2290 x 3184, 4096 rows: 129 us, cached 157).  Rows off
  // them start and end inside a line, which the L2 puts together (16 x 2290 x
  // 3189: 176 us, non-temporal 181, element by element 255; 45 rows: 130, 174
  // and 213).
  __syncthreads();
  if (mw <= 0 || nw <= 0) return;
  constexpr int CH = 4 * JN, RI = 64 / CH;  // 16-byte chunks of a row, rows of a store instruction
  uint8_t* tile = lds + wave * 16 * CH * 16;
  const uint32_t put = (uint32_t)r16 * (16 * CH), putx = 16u * (uint32_t)((lane >> 4) ^ (r16 & (CH - 1)));
  const int lr = lane / CH, ch = lane & (CH - 1);
  const uint64_t voff = ((uint64_t)lr * (uint64_t)g.ldc + 4u * (uint32_t)ch) * 4u;
  uint8_t* cw = reinterpret_cast<uint8_t*>(g.c + ((int64_t)gi * g.rows + m0 + wm * 16 * FM) * g.ldc + n0 + wn * 16 * JN);
  const bool full = mw >= 16 * FM && nw >= 16 * JN;
  auto write = [&](auto streaming) {
    auto store = [](float* dst, v4f v) {
      if constexpr (decltype(streaming)::value) {
        __builtin_nontemporal_store(v, reinterpret_cast<v4f*>(dst));
      } else {
        *reinterpret_cast<v4f_any*>(dst) = v;
      }
    };
#pragma unroll
    for (int f = 0; f < FM; ++f) {
#pragma unroll
      for (int j = 0; j < JN; ++j) *reinterpret_cast<v4f*>(tile + put + (putx ^ (uint32_t)(64 * j))) = acc[f][j];
#pragma unroll
      for (int i = 0; i < JN; ++i) {
        const int row = i * RI + lr;
        const v4f v = *reinterpret_cast<const v4f*>(tile + row * (16 * CH) + 16 * (ch ^ (row & (CH - 1))));
        float* dst = reinterpret_cast<float*>(cw + (int64_t)(f * 16 + i * RI) * g.ldc * 4 + voff);
        if (full) {
          store(dst, v);
        } else if (f * 16 + row < mw) {
          if (4 * ch + 3 < nw) {
            store(dst, v);
          } else {
#pragma unroll
            for (int u = 0; u < 4; ++u)
              if (4 * ch + u < nw) dst[u] = v[u];
          }
        }
      }
    }
  };
  // (the scheduling barriers keep the compiler from making one store of the two kinds)
  if (g.ldc % 16 == 0) {
    write(std::true_type{});
  } else {
    __builtin_amdgcn_sched_barrier(0);
    write(std::false_type{});
    __builtin_amdgcn_sched_barrier(0);
  }
}

template <class S>
void launch(WgArgs g, int groups, int acc, hipStream_t stream) {
  g.tiles_m = (g.rows + S::kTM - 1) / S::kTM;
  g.tiles_n = (g.n + S::kTN - 1) / S::kTN;
  // Each XCD reads the codes of its region's rows and columns through its own
  // L2: of the ways to lay eight regions over the tiles, the one with the
  // smallest border.  (7168 x 2048, 16 groups: 8192 rows 319 -> 282 us and
  // 32768 rows 846 -> 816 us against eight regions side by side, 256 x 256
  // tiles, power-of-two float32 form, and 998 MB read instead of 2523; within
  // 2% either way for 4096 x 7168, where the writes decide.)  Both divide into
  // even regions.  Balance is not looked at: where tiles do not divide, the
  // same XCDs have more than their share in every group (128 x 128 tiles of
  // 1152 x 640 and 1100 x 1100: the fullest 1.60 and 1.48 times the mean and
  // two without work; 2816 x 2048, 2880 x 2880: 1.09; 64 x 64 tiles of 320 x
  // 320: 1.92), not measured against another layout.
  int best = 0;
  for (int xn = 1; xn <= 8; xn *= 2) {
    const int xm = 8 / xn, rm = (g.tiles_m + xm - 1) / xm, rn = (g.tiles_n + xn - 1) / xn;
    if (!best || rm + rn < best) {
      best = rm + rn;
      g.region_m = rm;
      g.region_n = rn;
      g.xcds_n = xn;
    }
  }
  const dim3 grid(8 * g.region_m * g.region_n * groups), block(S::kThreads);
  switch (acc) {
    case 1: hipLaunchKernelGGL((wgrad_grouped_kernel<S, 1>), grid, block, 0, stream, g); break;
    case 2: hipLaunchKernelGGL((wgrad_grouped_kernel<S, 2>), grid, block, 0, stream, g); break;
    case 3: hipLaunchKernelGGL((wgrad_grouped_kernel<S, 3>), grid, block, 0, stream, g); break;
    default:
      if constexpr (S::kJN <= 4) hipLaunchKernelGGL((wgrad_grouped_kernel<S, 0>), grid, block, 0, stream, g);
  }
}

}  // namespace

hipError_t launch_grouped_wgrad(const uint8_t* dy_t, const float* dy_scales, const uint8_t* x_t,
                                const float* x_scales, const int32_t* offsets, int groups, int cap, int nout,
                                int kin, int acc, float* dw, int64_t lddw, hipStream_t stream) {
  WgArgs g{};
  g.a = dy_t; g.sa = dy_scales; g.w = x_t; g.sw = x_scales; g.offsets = offsets; g.c = dw; g.ldc = lddw;
  g.rows = nout; g.n = kin; g.k = cap;
  // Tiles of 64 x 64 where larger ones leave compute units without work: fewer
  // tiles of 128 x 128 than three quarters of the units, or, as groups are
  // uneven and the fullest is the last, fewer than half of them in a group and
  // five for every two in all.  Groups x outputs, rows in all, float32 form,
  // against 128 x 128: 1 x 512 x 512, 16384 rows 65 and 155 us; 4 x 512 x 512,
  // 4096 rows 12.9 and 26.3; 8 x 1024 x 1024, 16384 rows 51 and 74; 16 x 768 x
  // 768 (576 tiles), 16384 rows 39 and 59; past the rule 1 x 2048 x 2048, 16384
  // rows 172 and 161, 16 x 1024 x 1024 (1024 tiles), 4096 rows 24.3 and 21.1.
  // (Four K blocks in flight instead of two, or eight waves a tile: nothing
  // gained.)  One workgroup walks all blocks of its tile, 0.5 us each: with few
  // tiles that, and not a rate, is the time.
  //
  // Forms that accumulate in the matrix core need half the vector work per
  // product on 256 x 256 tiles (a W fragment is widened for 64 rows either
  // way, an A fragment for 128 columns instead of 64).  That pays once a tile
  // has enough blocks to hide that a compute unit holds one such tile and not
  // two, and there are tiles for all units: 4096 x 7168, 16 groups,
  // power-of-two float32 form, 2.4 / 4.5 / 8.6 blocks a group: 424 / 631 / 951
  // us against 410 / 690 / 1050 on 128 x 128; 7168 x 2048, 16.6 blocks: 811
  // against 917 (hardware scales: 551 against 711, FP8 partials 688 against
  // 744).  Groups are uneven: of several the fullest alone has to keep a
  // quarter of the units busy, and all of them two tiles for each (16 x 1024 x
  // 2048, 16384 rows: 111 against 78 us; 4 x 2048 x 2048, 4096 rows: 52 against
  // 42; 16 x 2048 x 2048, 8192 rows: 84 against 85; one group of 4096 x 4096,
  // 4096 rows: 102 against 115).  The folded form is VALU-bound on either (1112
  // against 1062 us at 8.6 blocks) and spills on the large one.
  const auto tiles = [&](int t) { return (int64_t)((nout + t - 1) / t) * ((kin + t - 1) / t) * groups; };
  const int cus = device_cus();
  const bool fills = groups == 1 ? tiles(256) >= cus : tiles(256) >= 2 * cus && 4 * tiles(256) >= (int64_t)cus * groups;
  const bool few = 4 * tiles(128) <= 3 * cus || (2 * tiles(128) <= 5 * cus && 2 * tiles(128) <= (int64_t)cus * groups);
  if (few) {
    launch<Small>(g, groups, acc, stream);
  } else if (acc == 0 || cap / BK < 4 * groups || !fills) {
    launch<Medium>(g, groups, acc, stream);
  } else {
    launch<Large>(g, groups, acc, stream);
  }
  return hipGetLastError();
}

}  // namespace fp8q
