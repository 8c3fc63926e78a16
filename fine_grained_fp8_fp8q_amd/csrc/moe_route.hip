// The way of tokens to the experts of one device and back (gfx950): the
// routing table the dispatch gather and the grouped GEMMs read, the weighted
// sum of a token's expert rows, and the gradient of that sum.
//
// * Sort: the (token, choice) pairs of the hosted experts, ordered by expert
//   and inside an expert by pair index (a stable counting sort), with every
//   expert's rows starting at a multiple of `align`.
// * Combine: out[t] = sum_j w[t,j] y[row_of[t,j]], float32, one rounding.
// * Combine backward: dy[row_of[t,j]] = bf16(w[t,j] dout[t]), optionally
//   quantized per 1x128 tile (jp-study.kr doc 258368 ¶1, tmdrlife.com
//   wr_id=13334 ¶4: the activation gradient before the down-projections is
//   one of the tensors that take FP8), and dw[t,j] = <dout[t], y[row]>.
#include <type_traits>

#include "chunk8.h"
#include "fp8q_internal.h"
#include "quant_common.h"

namespace fp8q {
namespace {

// ------------------------------------------------------------------ sort ---
// Bound by latency: 16384 x 8 pairs over 16 of 256 experts are 1.6 MB in and
// out, and the two launches take 7.5 us together (replayed from a graph; over
// all 256 experts 10.0 us, 800,000 pairs 17.7 us; one token's pairs, one
// launch, 4.0 us).  The second launch reads the whole table of counts in
// every workgroup, column by column into registers (one LDS atomic per entry
// instead: 18.5 us at 256 experts); unlike one pass with a running total
// handed on, nobody waits for another workgroup.  The first pass of a chunk
// counts with plain LDS atomics, only the second needs the order within a
// wave (ranks by ballots in both: 10.0 instead of 8.2 us for 4096 pairs in one
// workgroup).
constexpr int kSortThreads = 1024, kSortWaves = kSortThreads / 64;

struct SortArgs {
  const void* experts;  // [tokens, ld] int32 or int64
  int topk;
  int64_t ld;
  int64_t first;        // hosted experts: first .. first + groups - 1
  int groups, align;
  int pairs;            // tokens * topk
  int cap;              // rows of the sorted layout
  int chunk;            // pairs per workgroup, a multiple of kSortThreads (of 64 per wave)
  int* offsets;         // [groups + 1]
  int* token;           // [cap]
  int* row_of;          // [pairs]
  int* hist;            // [workgroups, groups] pairs of each workgroup's chunk per expert (more than one workgroup)
};

// Hosted expert of pair p, -1 for an expert of another device.
template <typename IDX>
__device__ __forceinline__ int local_expert(const SortArgs& a, int p) {
  const int t = (int)((unsigned)p / (unsigned)a.topk);
  const int64_t e = (int64_t)static_cast<const IDX*>(a.experts)[(int64_t)t * a.ld + (p - t * a.topk)] - a.first;
  return e >= 0 && e < a.groups ? (int)e : -1;
}

// Lanes of the wave that hold the same expert as this one (0 for e < 0):
// one ballot per bit of the expert index.
__device__ __forceinline__ uint64_t same_expert(int e, int bits) {
  uint64_t mask = __builtin_amdgcn_ballot_w64(e >= 0);
  for (int i = 0; i < bits; ++i) {
    const uint64_t set = __builtin_amdgcn_ballot_w64((e >> i) & 1);
    mask &= ((e >> i) & 1) ? set : ~set;
  }
  return e >= 0 ? mask : 0;
}

__device__ __forceinline__ int index_bits(int groups) { return groups > 1 ? 32 - __clz(groups - 1) : 0; }

// Pairs per expert of each workgroup's chunk.
template <typename IDX>
__global__ __launch_bounds__(kSortThreads) void sort_count_kernel(SortArgs a) {
  __shared__ int cnt[kMaxSortGroups];
  const int tid = threadIdx.x;
  for (int e = tid; e < a.groups; e += kSortThreads) cnt[e] = 0;
  __syncthreads();
  const int64_t p0 = (int64_t)blockIdx.x * a.chunk;
  for (int i = 0; i < a.chunk; i += kSortThreads) {
    const int64_t p = p0 + i + tid;
    const int e = p < a.pairs ? local_expert<IDX>(a, (int)p) : -1;
    if (e >= 0) atomicAdd(&cnt[e], 1);
  }
  __syncthreads();
  for (int e = tid; e < a.groups; e += kSortThreads) a.hist[(int64_t)blockIdx.x * a.groups + e] = cnt[e];
}

// Every workgroup forms the whole table of group starts for itself (from the
// per-chunk counts, or, alone, from its own) and places its chunk: wave w
// takes the w-th sixteenth of it in order, so a pair's row is the group's
// start + the pairs of that expert in earlier chunks, in earlier waves, in
// earlier steps of this wave (a running count in LDS) and in lower lanes.
// The experts of the first four steps stay in registers between the two
// passes (all of them below a million pairs).
template <typename IDX>
__global__ __launch_bounds__(kSortThreads) void sort_place_kernel(SortArgs a) {
  extern __shared__ int lds[];
  const int G = a.groups;
  int* cnt = lds;                      // [kSortWaves][G]: running counts
  int* total = cnt + kSortWaves * G;   // [G] pairs of the expert
  int* start = total + G;              // [G + 1] first row of the group
  int* scan = start + G + 1;           // [kSortWaves]
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int blk = blockIdx.x, blocks = gridDim.x;
  const int bits = index_bits(G);
  const int steps = a.chunk / kSortThreads;
  const int64_t p0 = (int64_t)blk * a.chunk + (int64_t)wave * 64 * steps + lane;
  auto expert_at = [&](int s) {
    const int64_t p = p0 + 64 * s;
    return p < a.pairs ? local_expert<IDX>(a, (int)p) : -1;
  };
  constexpr int kHeld = 4;
  int held[kHeld];
#pragma unroll
  for (int s = 0; s < kHeld; ++s) held[s] = s < steps ? expert_at(s) : -1;
  for (int i = tid; i < (kSortWaves + 2) * G + 1; i += kSortThreads) lds[i] = 0;
  __syncthreads();

  auto count = [&](int e) {
    if (e >= 0) atomicAdd(&cnt[wave * G + e], 1);
  };
#pragma unroll
  for (int s = 0; s < kHeld; ++s)
    if (s < steps) count(held[s]);
  for (int s = kHeld; s < steps; ++s) count(expert_at(s));
  // pairs of each expert in all chunks, and in the chunks before this one
  // (kept in start[] until the group starts are known)
  if (blocks > 1) {
    const int stride = 1 << bits;  // threads e, e + stride, ... add up the column of expert e
    const int e = tid & (stride - 1), parts = kSortThreads >> bits;
    if (e < G) {
      int all = 0, before = 0;
#pragma unroll 8
      for (int b = tid >> bits; b < blocks; b += parts) {
        const int h = a.hist[b * G + e];
        all += h;
        before += b < blk ? h : 0;
      }
      if (all) atomicAdd(&total[e], all);
      if (before) atomicAdd(&start[e], before);
    }
  }
  __syncthreads();
  // exclusive running counts: before this wave (and, for wave 0, before this chunk)
  int mine = 0, padded = 0;
  if (tid < G) {
    int run = start[tid];
#pragma unroll
    for (int w = 0; w < kSortWaves; ++w) {
      const int c = cnt[w * G + tid];
      cnt[w * G + tid] = run;
      run += c;
    }
    mine = blocks > 1 ? total[tid] : run;
    padded = (int)(((int64_t)mine + a.align - 1) / a.align * a.align);
  }
  // inclusive scan of the padded group sizes (G <= kSortThreads)
  int inc = padded;
  for (int d = 1; d < 64; d <<= 1) {
    const int v = __shfl_up(inc, d);
    if (lane >= d) inc += v;
  }
  if (lane == 63) scan[wave] = inc;
  __syncthreads();
  for (int w = 0; w < wave; ++w) inc += scan[w];
  if (tid < G) {
    total[tid] = mine;
    start[tid] = inc - padded;
    if (tid == G - 1) start[G] = inc;
  }
  __syncthreads();
  if (blk == 0)
    for (int g = tid; g <= G; g += kSortThreads) a.offsets[g] = min(start[g], a.cap);

  auto place = [&](int s, int e) {
    const uint64_t same = same_expert(e, bits);
    const int first = same ? __builtin_ctzll(same) : 0;
    int before = 0;
    if (same && lane == first) before = atomicAdd(&cnt[wave * G + e], __builtin_popcountll(same));
    before = __shfl(before, first);
    const int64_t p = p0 + 64 * s;
    if (p < a.pairs) {
      int row = -1;
      if (e >= 0) {
        row = start[e] + before + __builtin_popcountll(same & ((uint64_t(1) << lane) - 1));
        if (row < a.cap) {
          a.token[row] = (int)((unsigned)p / (unsigned)a.topk);
        } else {
          row = -1;
        }
      }
      a.row_of[p] = row;
    }
  };
#pragma unroll
  for (int s = 0; s < kHeld; ++s)
    if (s < steps) place(s, held[s]);
  for (int s = kHeld; s < steps; ++s) place(s, expert_at(s));
  // rows without a pair: the padding of every group (a group to a wave, 160
  // groups padded to 128 take 8.0 us instead of 23.2 with a group to the
  // workgroup; long paddings by all of it), and everything behind the last one
  auto clear = [&](int64_t r) { a.token[r] = -1; };
  if (a.align > 1) {
    const bool all = a.align > kSortThreads;
    const int lanes = all ? kSortThreads : 64, first = all ? blk : blk * kSortWaves + wave;
    for (int g = first; g < G; g += all ? blocks : blocks * kSortWaves)
      for_rows(start[g] + total[g], all ? tid : lane, lanes, min(start[g + 1], a.cap), clear);
  }
  for_rows(start[G], blk * kSortThreads + tid, blocks * kSortThreads, a.cap, clear);
}

// --------------------------------------------------------------- combine ---
// One workgroup per token and chunk of 8 x threads columns: the rows and
// weights of the token are wave-uniform, and the chunks of up to eight rows
// are in flight at once.  A thread has eight columns side by side for a BF16
// output, and four in each half of the chunk for a float32 one (stores of
// whole lines: 54 us instead of 64-69 for 8192 x 7168).  Bound by HBM: 4096
// tokens x 8 rows x 7168 (BF16) at 5.9 TB/s (90 us).
template <bool YF32, bool OF32, bool VEC, bool KEEP>
__global__ __launch_bounds__(256) void combine_kernel(const void* __restrict__ y, int cap, int n, int64_t ldy,
                                                      const int* __restrict__ row_of,
                                                      const float* __restrict__ weights, int topk, int chunks,
                                                      void* __restrict__ out, int64_t ldo) {
  static_assert(VEC || KEEP, "loads of unaligned rows are plain ones");
  constexpr int W = OF32 ? 4 : 8, H = OF32 ? 2 : 1;  // columns of a load, loads of a row
  const int t = blockIdx.x / chunks;
  const int col0 = (blockIdx.x - t * chunks) * (int)blockDim.x * 8 + (int)threadIdx.x * W;
  if (col0 >= n) return;
  const int* rows = row_of + (int64_t)t * topk;
  const float* w = weights ? weights + (int64_t)t * topk : nullptr;
  float acc[H][W] = {};
  for (int j0 = 0; j0 < topk; j0 += 8) {
    Raw<YF32, W> v[8][H];
    bool has[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int r = j0 + u < topk ? rows[j0 + u] : -1;
      has[u] = (unsigned)r < (unsigned)cap;
      if (!has[u]) continue;
#pragma unroll
      for (int h = 0; h < H; ++h) {
        const int col = col0 + h * W * (int)blockDim.x;
        if (VEC && h > 0 && col >= n) continue;
        v[u][h] = ld_raw<YF32, W, KEEP>(y, (int64_t)r * ldy + col, VEC ? W : n - col, VEC);
      }
    }
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      if (!has[u]) continue;
      const float wj = w ? w[j0 + u] : 1.0f;
#pragma unroll
      for (int h = 0; h < H; ++h)
#pragma unroll
        for (int i = 0; i < W; ++i) acc[h][i] = __builtin_fmaf(wj, v[u][h].at(i), acc[h][i]);
    }
  }
  if constexpr (OF32) {
#pragma unroll
    for (int h = 0; h < H; ++h) {
      const int col = col0 + h * W * (int)blockDim.x;
      if (VEC && h > 0 && col >= n) continue;
      st_float4(static_cast<float*>(out) + (int64_t)t * ldo + col, acc[h], VEC ? W : n - col, VEC);
    }
  } else {
    st_bf16x8(static_cast<uint16_t*>(out) + (int64_t)t * ldo + col0, pack_bf16x8(acc[0]), VEC ? W : n - col0, VEC);
  }
}

// ------------------------------------------------------ combine backward ---
struct CombineBwdArgs {
  const void* dout;
  int64_t lddo;
  const void* y;         // null: no weight gradient
  int64_t ldy;
  const int* row_of;
  const float* weights;  // null: 1
  const int* token;      // null: rows without a pair are left alone
  uint16_t* dy;          // null: no BF16 rows
  int64_t lddy;
  uint8_t* codes;        // null: no E4M3 rows
  int64_t ldc;
  float* scales;
  float* dweights;
  int pairs, topk, n, cap;
};

constexpr int kZeroRows = 4;  // rows looked over by one of the trailing workgroups

// Zeros for `bytes` bytes at p, by the whole workgroup: single bytes up to a
// 16-byte boundary and from the last one on, 16 at a time between them (rows
// of 1030 BF16 values start on 4-byte boundaries: 3900 of them take 1.7 us so,
// 5.7 with 16-byte stores across the boundaries, 16 rows a workgroup).
__device__ __forceinline__ void clear_row(uint8_t* p, int64_t bytes) {
  const int head = (int)((16 - (reinterpret_cast<uintptr_t>(p) & 15)) & 15);
  if (bytes < 64) {
    if ((int)threadIdx.x < bytes) p[threadIdx.x] = 0;
    return;
  }
  const int64_t body = (bytes - head) >> 4, end = head + 16 * body;
  if ((int)threadIdx.x < head) p[threadIdx.x] = 0;
  if ((int)threadIdx.x < (int)(bytes - end)) p[end + threadIdx.x] = 0;
  for (int64_t i = threadIdx.x; i < body; i += blockDim.x) st_stream16(p + head + 16 * i, make_uint4(0, 0, 0, 0));
}

// Workgroup p < pairs: pair p.  The pairs of a token follow one another on
// one XCD, so its gradient row comes from HBM once and from that XCD's L2
// for the other choices (4096 x 8 x 7168 to E4M3: 160 us with the pairs dealt
// to the XCDs in turn, 158 us with streaming loads of that row, 144 us, 5.4
// TB/s, as it is; two to eight choices a workgroup, or the next chunk's loads
// ahead, change nothing).  The workgroups behind the pairs clear the rows
// without a pair.
template <bool DF32, bool YF32, bool POW2, bool VEC, bool KEEP>
__global__ __launch_bounds__(256) void combine_bwd_kernel(CombineBwdArgs a) {
  static_assert(VEC || KEEP, "loads of unaligned rows are plain ones");
  __shared__ float part[4];
  const int tid = threadIdx.x;
  const int nb = (a.n + 127) >> 7;
  const int step = (int)blockDim.x * 8;
  if ((int)blockIdx.x >= a.pairs) {
    const int r0 = ((int)blockIdx.x - a.pairs) * kZeroRows, at = r0 + (tid & 63);
    uint64_t clear = __builtin_amdgcn_ballot_w64((tid & 63) < kZeroRows && at < a.cap && a.token[at < a.cap ? at : 0] < 0);
    for (; clear; clear &= clear - 1) {
      const int r = r0 + __builtin_ctzll(clear);
      if (a.dy) clear_row(reinterpret_cast<uint8_t*>(a.dy + (int64_t)r * a.lddy), 2 * (int64_t)a.n);
      if (a.codes) {
        clear_row(a.codes + (int64_t)r * a.ldc, a.n);
        for (int j = tid; j < nb; j += (int)blockDim.x) a.scales[(int64_t)r * nb + j] = 0.0f;
      }
    }
    return;
  }
  // contiguous pairs on one XCD (workgroup i runs on XCD i % 8)
  const int xcd = blockIdx.x & 7, idx = blockIdx.x >> 3;
  const int per = a.pairs >> 3, rem = a.pairs & 7;
  const int p = xcd * per + min(xcd, rem) + idx;
  const int row = a.row_of[p];
  const float w = a.weights ? a.weights[p] : 1.0f;
  if ((unsigned)row >= (unsigned)a.cap) {
    if (tid == 0 && a.dweights) a.dweights[p] = 0.0f;
    return;
  }
  const int t = (int)((unsigned)p / (unsigned)a.topk);
  float dot = 0.0f;
  for (int c0 = 0; c0 < a.n; c0 += step) {
    const int col = c0 + tid * 8, left = VEC ? 8 : a.n - col;
    const bool in = col < a.n;
    float g[8] = {};
    if (in) {
      const auto gr = ld_raw<DF32, 8, true>(a.dout, (int64_t)t * a.lddo + col, left, VEC);
      Raw<YF32, 8> v = {};
      if (a.y) v = ld_raw<YF32, 8, KEEP>(a.y, (int64_t)row * a.ldy + col, left, VEC);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        g[i] = gr.at(i);
        dot = __builtin_fmaf(g[i], v.at(i), dot);
        g[i] = w * g[i];
      }
    }
    const uint4 d = pack_bf16x8(g);
    if (a.dy && in) st_bf16x8(a.dy + (int64_t)row * a.lddy + col, d, left, VEC);
    if (a.codes) {
      // a 16-lane DPP row holds one 1x128 tile; every lane takes part
      const TileScale ts = tile_scale<POW2>(dpp_max16(absmax8(d)));
      const uint2 c = encode8<POW2>(d, ts);
      if (in) {
        st_codes8(a.codes + (int64_t)row * a.ldc + col, c, left, VEC);
        if ((tid & 15) == 0) a.scales[(int64_t)row * nb + (col >> 7)] = ts.s;
      }
    }
  }
  if (!a.dweights) return;
  for (int d = 32; d; d >>= 1) dot += __shfl_xor(dot, d);
  if ((tid & 63) == 0) part[tid >> 6] = dot;
  __syncthreads();
  if (tid == 0) {
    for (int i = 1; i < (int)blockDim.x >> 6; ++i) dot += part[i];
    a.dweights[p] = dot;
  }
}

}  // namespace

template <typename IDX>
static hipError_t launch_sort(SortArgs a, int blocks, hipStream_t stream) {
  if (blocks > 1) hipLaunchKernelGGL(sort_count_kernel<IDX>, dim3(blocks), dim3(kSortThreads), 0, stream, a);
  const size_t lds = ((size_t)(kSortWaves + 2) * a.groups + 1 + kSortWaves) * sizeof(int);
  hipLaunchKernelGGL(sort_place_kernel<IDX>, dim3(blocks), dim3(kSortThreads), lds, stream, a);
  return hipGetLastError();
}

hipError_t launch_moe_sort(const void* experts, bool i64, int pairs, int topk, int64_t ld, int64_t first, int groups,
                           int align, int cap, int* offsets, int* token, int* row_of, int* hist,
                           hipStream_t stream) {
  SortArgs a{};
  a.experts = experts; a.topk = topk; a.ld = ld; a.first = first; a.groups = groups; a.align = align;
  a.pairs = pairs; a.cap = cap; a.offsets = offsets; a.token = token; a.row_of = row_of; a.hist = hist;
  const int blocks = sort_blocks(pairs);
  const int64_t per = ((int64_t)pairs + blocks - 1) / blocks;
  a.chunk = (int)((per + kSortThreads - 1) / kSortThreads * kSortThreads);
  if (a.chunk == 0) a.chunk = kSortThreads;
  return i64 ? launch_sort<int64_t>(a, blocks, stream) : launch_sort<int32_t>(a, blocks, stream);
}

// VEC: every row starts on a 16-byte boundary and has whole chunks, so the
// kernels need no checks of a chunk's end (with them at every load the two
// sums above take 97 and 74 us).
template <class F>
static void with_flag(bool flag, F f) {
  if (flag) {
    f(std::true_type{});
  } else {
    f(std::false_type{});
  }
}

// f(VEC, KEEP): rows that are not VEC are loaded one way only.
template <class F>
static void with_load(bool vec, bool keep, F f) {
  if (vec) {
    with_flag(keep, [&](auto kept) { f(std::true_type{}, kept); });
  } else {
    f(std::false_type{}, std::true_type{});
  }
}

hipError_t launch_moe_combine(const void* y, bool y_f32, int cap, int n, int64_t ldy, const int* row_of,
                              const float* weights, int tokens, int topk, bool out_f32, void* out, int64_t ldo,
                              hipStream_t stream) {
  const int items = (n + 7) / 8, threads = row_threads(n);
  const int chunks = (items + threads - 1) / threads;
  const dim3 grid((unsigned)(tokens * chunks)), block(threads);
  const bool keep = input_stays_cached(cap, ldy * (y_f32 ? 4 : 2));
  with_load(n % 8 == 0 && ldy % 8 == 0 && ldo % 8 == 0, keep, [&](auto vec, auto kept) {
    constexpr bool V = decltype(vec)::value, K = decltype(kept)::value;
    auto kernel = y_f32 ? (out_f32 ? combine_kernel<true, true, V, K> : combine_kernel<true, false, V, K>)
                        : (out_f32 ? combine_kernel<false, true, V, K> : combine_kernel<false, false, V, K>);
    hipLaunchKernelGGL(kernel, grid, block, 0, stream, y, cap, n, ldy, row_of, weights, topk, chunks, out, ldo);
  });
  return hipGetLastError();
}

hipError_t launch_moe_combine_backward(const void* dout, bool dout_f32, int tokens, int n, int64_t lddo,
                                       const void* y, bool y_f32, int cap, int64_t ldy, const int* row_of,
                                       const float* weights, int topk, const int* token, uint16_t* dy,
                                       int64_t lddy, bool pow2, uint8_t* codes, int64_t ldc, float* scales,
                                       float* dweights, hipStream_t stream) {
  CombineBwdArgs a{};
  a.dout = dout; a.lddo = lddo; a.y = y; a.ldy = ldy; a.row_of = row_of; a.weights = weights; a.token = token;
  a.dy = dy; a.lddy = lddy; a.codes = codes; a.ldc = ldc; a.scales = scales; a.dweights = dweights;
  a.pairs = tokens * topk; a.topk = topk; a.n = n; a.cap = cap;
  const bool whole = n % 8 == 0 && lddo % 8 == 0 && (!y || ldy % 8 == 0) && (!dy || lddy % 8 == 0) && (!codes || ldc % 8 == 0);
  const int zero = token && (dy || codes) ? (cap + kZeroRows - 1) / kZeroRows : 0;
  const dim3 grid(a.pairs + zero), block(combine_backward_threads(a.pairs, n));
  with_load(whole, y && input_stays_cached(cap, ldy * (y_f32 ? 4 : 2)), [&](auto vec, auto kept) {
    with_flag(pow2, [&](auto p2) {
      constexpr bool V = decltype(vec)::value, K = decltype(kept)::value, P = decltype(p2)::value;
      auto kernel = dout_f32 ? (y_f32 ? combine_bwd_kernel<true, true, P, V, K> : combine_bwd_kernel<true, false, P, V, K>)
                             : (y_f32 ? combine_bwd_kernel<false, true, P, V, K> : combine_bwd_kernel<false, false, P, V, K>);
      hipLaunchKernelGGL(kernel, grid, block, 0, stream, a);
    });
  });
  return hipGetLastError();
}

}  // namespace fp8q
