// Internal declarations shared by the host entry points (fp8q_api.cpp) and
// the kernel translation units.  Not part of the public ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace fp8q {

// Grid sizes of the streaming kernels (host code; 64-bit arithmetic, so a
// tile count up to 2^31 - 1 cannot overflow here).
//  rows_grid: the 1x128 row quantizer, one pass per wave (16 tiles per
//    wave: 16 per 64-thread workgroup, 128 per 512-thread workgroup) up to
//    kMaxRowsGrid workgroups, then a grid-stride loop whose stride is
//    tiles_per_wg * kMaxRowsGrid tiles.
//  stream_grid: four waves per workgroup, up to kMaxStreamGrid workgroups.
constexpr int kMaxRowsGrid = 1 << 20;
constexpr int kMaxStreamGrid = 2048;
inline int rows_grid(int64_t ntiles, int tiles_per_wg = 64) {
  const int64_t want = (ntiles + tiles_per_wg - 1) / tiles_per_wg;
  return (int)(want < kMaxRowsGrid ? want : kMaxRowsGrid);
}
inline int stream_grid(int64_t waves_needed) {
  const int64_t wg = (waves_needed + 3) / 4;
  return (int)(wg < kMaxStreamGrid ? (wg > 0 ? wg : 1) : kMaxStreamGrid);
}

// Launchers validate nothing: fp8q_api.cpp has checked shapes, alignment and
// the device before calling them.  Every size here is > 0 and < 2^31.
hipError_t launch_quant_rows(const uint16_t* x, int rows, int cols, int64_t ldx, bool pow2,
                             uint8_t* codes, int64_t ldc, float* scales, hipStream_t stream);
hipError_t launch_quant_token_t(const uint16_t* x, int rows, int cols, int64_t ldx, bool pow2,
                                uint8_t* codes, int64_t ldc, float* scales, hipStream_t stream);
hipError_t launch_quant_blocks(const uint16_t* w, int n, int k, int64_t ldw, bool pow2,
                               uint8_t* codes, int64_t ldc, float* scales, hipStream_t stream);

// the activation x [m, k] in 1x128 tiles and the weight w [n, k] in 128x128
// blocks, one launch
hipError_t launch_quant_linear(const uint16_t* x, int m, int k, int64_t ldx, bool a_pow2, uint8_t* a_codes,
                               int64_t lda, float* a_scales, const uint16_t* w, int n, int64_t ldw, bool w_pow2,
                               uint8_t* w_codes, int64_t ldwc, float* w_scales, hipStream_t stream);

hipError_t launch_quant_blocks_t(const uint16_t* w, int n, int k, int64_t ldw, bool pow2,
                                 uint8_t* codes, int64_t ldc, float* scales, uint8_t* codes_t,
                                 int64_t ldt, float* scales_t, hipStream_t stream);

hipError_t launch_gemm(const uint8_t* a, const float* a_scales, const uint8_t* w,
                       const float* w_scales, int m, int n, int k, bool bf16_out, int acc,
                       void* c, int64_t ldc, hipStream_t stream);
// float32-grade dense GEMM over 32 x 32 output tiles with the K blocks split
// over four waves (gemm_small.hip); launch_gemm takes it for outputs of at
// most small_gemm_limit() elements
hipError_t launch_gemm_small(const uint8_t* a, const float* a_scales, const uint8_t* w, const float* w_scales,
                             int m, int n, int k, bool bf16_out, void* c, int64_t ldc, hipStream_t stream);
// outputs (M * N) up to which the dense float32-grade GEMM uses the small
// kernel: the value set by set_small_gemm_limit, or, while none is set (or
// after a negative one), 8192 per compute unit of the current device
int64_t small_gemm_limit();
int64_t set_small_gemm_limit(int64_t max_outputs);  // returns the previous setting (-1: the default)
int device_cus();
// C = A . W^T rounded to BF16, quantized per 1x128 tile along N
hipError_t launch_gemm_quantized(const uint8_t* a, const float* a_scales, const uint8_t* w,
                                 const float* w_scales, int m, int n, int k, int acc, bool pow2,
                                 uint8_t* codes, int64_t ldc, float* scales, hipStream_t stream);
hipError_t launch_grouped_gemm(const uint8_t* a, const float* a_scales, const int32_t* offsets,
                               int groups, int rows_cap, const uint8_t* w, const float* w_scales,
                               int n, int k, bool bf16_out, int acc, void* c, int64_t ldc,
                               hipStream_t stream);
hipError_t launch_wgrad(const uint8_t* dy_t, const float* dy_scales, const uint8_t* x_t,
                        const float* x_scales, int nout, int kin, int t, int acc, float* dw,
                        int64_t lddw, hipStream_t stream);

hipError_t launch_gather_rows(const uint8_t* codes, int rows, int cols, int64_t ldc, const float* scales,
                              const int32_t* index, int n_out, uint8_t* out, int64_t ldo, float* out_scales,
                              hipStream_t stream);
// ccodes == nullptr: no cache of the input (cache_pow2, ldcc, cscales unused)
hipError_t launch_swiglu_quant(const uint16_t* x, int rows, int inter, int64_t ldx, bool pow2, uint8_t* codes,
                               int64_t ldc, float* scales, bool cache_pow2, uint8_t* ccodes, int64_t ldcc,
                               float* cscales, hipStream_t stream);

// Routing table (moe_route.hip): one workgroup alone up to kSortAlonePairs
// pairs; above, as many workgroups of 1024 pairs or more as there are, at
// most kMaxSortBlocks, after a launch that counts each one's pairs per expert
// (hist: int32 [blocks, groups]).
constexpr int kMaxSortGroups = 512;
constexpr int kSortAlonePairs = 4096;
constexpr int kMaxSortBlocks = 256;
inline int sort_blocks(int pairs) {
  if (pairs <= kSortAlonePairs) return 1;
  const int64_t blocks = ((int64_t)pairs + 1023) / 1024;
  return (int)(blocks < kMaxSortBlocks ? blocks : kMaxSortBlocks);
}
// f(row) for the rows first + lane, first + lane + lanes, ... below end.  first
// and end reach 2^31 - 1, so a row past the end is not a 32-bit number.
template <class F>
__host__ __device__ inline void for_rows(int first, int lane, int lanes, int end, F f) {
  for (int64_t r = (int64_t)first + lane; r < end; r += lanes) f(r);
}
hipError_t launch_moe_sort(const void* experts, bool i64, int pairs, int topk, int64_t ld, int64_t first, int groups,
                           int align, int cap, int* offsets, int* token, int* row_of, int* hist, hipStream_t stream);
// Streaming (non-temporal) loads pass the 256 MB Infinity Cache by.  An input
// that the kernel before has just written is found there by plain loads as
// long as all of it fits beside the output; a larger one is streamed.
// Measured, plain against streaming loads, inputs in rotation: combine of 87
// MB of rows 27 against 34 us (float32 out 38 against 52), 112 MB 25 against
// 23, 448 MB 95 against 88; combine backward of 59 MB 17.6 against 21.2, 117
// MB 41 against 39; SwiGLU backward from 34 MB of cache and gradient 13.6
// against 16.4, 67 MB 25.6 against 29.4, 134 MB 58 against 57.  Rows off
// 16-byte boundaries are always read with plain loads (chunk8.h).
inline bool input_stays_cached(int64_t rows, int64_t row_bytes) {
  return row_bytes == 0 || rows <= ((int64_t)96 << 20) / row_bytes;
}

// Threads of a workgroup that goes over a row of n columns, eight a thread:
// of 64, 128, 192 and 256 the one that leaves the fewest idle, the largest of
// equals (7168 columns: 7 x 128; 1030: 192).
inline int row_threads(int n) {
  const int items = (n + 7) / 8;
  int threads = 256;
  for (int c = 192; c >= 64; c -= 64)
    if ((items + c - 1) / c * c < (items + threads - 1) / threads * threads) threads = c;
  return threads;
}
// Combine backward.  Few pairs wait for the loads of one step after another:
// as few steps as there are (8 pairs of 6259 columns: 4 steps of 256 threads
// 5.4 us, 13 of 64 10.1).  Many hide each other's: as few idle threads (32768
// pairs of 7168 columns: 7 x 128 144 us, 4 x 256 149).  Rows of no columns
// still have a weight gradient to write, and so one wave.
inline int combine_backward_threads(int pairs, int n) {
  if (pairs > 2048) return row_threads(n);
  if (n == 0) return 64;
  const int items = (n + 7) / 8, steps = (items + 255) / 256;
  return ((items + steps - 1) / steps + 63) / 64 * 64;
}

hipError_t launch_moe_combine(const void* y, bool y_f32, int cap, int n, int64_t ldy, const int* row_of,
                              const float* weights, int tokens, int topk, bool out_f32, void* out, int64_t ldo,
                              hipStream_t stream);
// y == nullptr: no weight gradient; dy / codes == nullptr: that form of the rows is not written
hipError_t launch_moe_combine_backward(const void* dout, bool dout_f32, int tokens, int n, int64_t lddo,
                                       const void* y, bool y_f32, int cap, int64_t ldy, const int* row_of,
                                       const float* weights, int topk, const int* token, uint16_t* dy, int64_t lddy,
                                       bool pow2, uint8_t* codes, int64_t ldc, float* scales, float* dweights,
                                       hipStream_t stream);
// xscales == nullptr: x is BF16; else x are E4M3 codes with 1x128 scales
hipError_t launch_swiglu_backward(const void* x, const float* xscales, int rows, int inter, int64_t ldx,
                                  const uint16_t* dy, int64_t lddy, uint16_t* dx, int64_t lddx, bool pow2,
                                  uint8_t* codes, int64_t ldc, float* scales, uint16_t* y, int64_t ldy,
                                  hipStream_t stream);
hipError_t launch_grouped_wgrad(const uint8_t* dy_t, const float* dy_scales, const uint8_t* x_t,
                                const float* x_scales, const int32_t* offsets, int groups, int cap, int nout,
                                int kin, int acc, float* dw, int64_t lddw, hipStream_t stream);

// RMS norm (norm.hip): res == nullptr: h = x (h, ldh unused).  h, y, codes,
// rstd == nullptr: not written.
struct NormArgs {
  const void* x;
  int64_t ldx;
  const void* res;
  int64_t ldr;
  void* h;
  int64_t ldh;
  const void* weight;
  uint16_t* y;
  int64_t ldy;
  uint8_t* codes;
  int64_t ldc;
  float* scales;
  float* rstd;
  double eps, inv_n;  // inv_n: 1 / n, or 0
  int rows, n;
  bool xf32, sf32, wf32, pow2;
};
// A row of up to kMaxNormRow columns stays in the registers of its workgroup:
// chunks of eight columns that a thread of the forward pass keeps, and the
// threads (0: the row is longer and is read twice).  Many rows want few waves
// each, with many loads on their way in every one; few rows, or short ones, the
// shortest way through a row.  Microseconds at 1 / 2 / 4 chunks, BF16 stream to
// E4M3: 16384 x 7168 213 / 148 / 139, 2048 x 7168 26.5 / 19.8 / 19.2, 512 x 7168
// 8.7 / 7.3 / 7.5, one row 3.9 / 3.7 / 4.0; 16384 x 4096 87 / 79 / 80; 16384 x
// 2048 44.8 / 42.8 / 43.1, one row 2.7 / 3.0 / 3.6; 65536 x 512 44 / 52 / 84.
constexpr int kMaxNormRow = 16384;
constexpr int kMaxNormGrid = 1 << 20;  // workgroups; more rows go round
inline int norm_chunks(int rows, int n) {
  const int items = (n + 7) / 8;
  if (items <= (rows < 4096 ? 256 : 128)) return 1;
  return items > 512 && rows >= 2048 ? 4 : 2;
}
inline int norm_threads(int n, int chunks) {
  if (n > kMaxNormRow) return 0;
  const int per = ((n + 7) / 8 + chunks - 1) / chunks;
  return per == 0 ? 64 : (per + 63) / 64 * 64;
}
// Where many rows of the same width have twice the chunks, few have twice their
// threads (split), so that the sum over a row is the same; those of 128 threads
// whose last 64 have one chunk all the same 192 (4000 rows of 1030 columns 11.2
// us, 12.7 with 256).
struct NormShape {
  int chunks, threads;
  bool split;
};
inline NormShape norm_shape(int rows, int n) {
  const int chunks = norm_chunks(rows, n), most = norm_chunks(kMaxNormGrid, n);
  NormShape s{chunks, norm_threads(n, most) * (most / chunks), chunks != most};
  if (s.split && chunks == 1 && (n + 7) / 8 <= 192) s.threads = 192;
  return s;
}
hipError_t launch_norm(const NormArgs& a, hipStream_t stream);
// dres == nullptr: no such term; dx, codes, dweight == nullptr: not written.
// partial: float [norm_bwd_blocks(rows, n), norm_partial_ld(n)], only used for
// dweight.
struct NormBwdArgs {
  const void* dy;
  int64_t lddy;
  const void* h;
  int64_t ldh;
  const float* rstd;
  const void* weight;
  const void* dres;
  int64_t lddr;
  void* dx;
  int64_t lddx;
  uint8_t* codes;
  int64_t ldc;
  float* scales;
  float* dweight;
  float* partial;
  int64_t ldp;  // (set by the launcher)
  double inv_n;  // 1 / n
  int rows, n;
  bool df32, hf32, wf32, of32, pow2;
};
// How the backward pass goes over its rows (rows, n > 0; f32: some tensor of
// them is float32): a wave a row while `chunks` of eight columns a lane hold
// it, a workgroup above (chunks 0: the row is longer than that of 512 threads).
// Three chunks of float32 values take the registers of two waves a SIMD: only
// where there are rows enough (8192 rows of 1030 35 us, 43 by workgroups of two
// chunks a thread; one row 7.3 and 6.5).  The sums are the same bit for bit.
// `blocks` workgroups (of longer rows: blocks of them), each with a share of
// the gain's gradient.  As few blocks as keep the memory busy, since every
// share is written and read again: 8192 rows of 7168 BF16 columns take 87 us
// with 256 blocks, 90 with 512 (as many as fit); 16384 of 2048 50 and 51; 8192
// of 4096 62 and 56; 32768 of 512 34 and 28; and 4096 of 7001, whose rows begin
// anywhere and take more instructions, 80 and 71.  Few rows are spread over
// workgroups of fewer waves (256 rows of 1030: 9.2 us, 10.6 in 64 of four).
struct NormBwdShape {
  int threads, chunks, blocks;
  bool wave;
};
constexpr int kNormBwdBlocks = 512;
inline NormBwdShape norm_bwd_shape(int rows, int n, bool f32) {
  const int items = (n + 7) / 8, most = f32 ? 2 : 4;
  NormBwdShape s{};
  s.wave = items <= 64 * (most < 3 && rows >= 2048 ? 3 : most);
  s.chunks = n > kMaxNormRow / (f32 ? 2 : 1) ? 0 : items <= 64 ? 1 : items <= 128 ? 2 : s.wave && items <= 192 ? 3 : most;
  s.threads = s.chunks ? ((items + most - 1) / most + 63) / 64 * 64 : 1024;
  const int blocks = (s.wave ? s.chunks < 4 : s.threads < 256 || n % 8) || !s.chunks ? kNormBwdBlocks : kNormBwdBlocks / 2;
  if (s.wave) s.threads = 64 * (rows > 3 * blocks ? 4 : (rows + blocks - 1) / blocks);
  const int64_t want = s.wave ? ((int64_t)rows * 64 + s.threads - 1) / s.threads : s.chunks ? rows : ((int64_t)rows + 31) / 32;
  s.blocks = (int)(want < blocks ? want : blocks);
  return s;
}
// rows of each of `blocks` blocks (rows reach 2^31 - 1: their sum with the blocks is not a 32-bit number)
inline int norm_dw_rows(int rows, int blocks) { return (int)(((int64_t)rows + blocks - 1) / blocks); }
// blocks of the workspace: those of the types that take more
inline int norm_bwd_blocks(int rows, int n) {
  const int b = norm_bwd_shape(rows, n, false).blocks, f = norm_bwd_shape(rows, n, true).blocks;
  return b > f ? b : f;
}
inline int64_t norm_partial_ld(int n) { return ((int64_t)n + 7) / 8 * 8; }
hipError_t launch_norm_backward(const NormBwdArgs& a, hipStream_t stream);
// index == nullptr: row t of the output is row t of h
struct NormTokenArgs {
  const void* h;
  int64_t ldh;
  const float* rstd;
  const void* weight;
  const int* index;
  uint8_t* codes;
  int64_t ldc;
  float* scales;
  int rows, src_rows, n;
  bool hf32, wf32, pow2;
};
hipError_t launch_norm_token(const NormTokenArgs& a, hipStream_t stream);

// The router's choice (moe_gate.hip).
constexpr int kMaxGateExperts = 512;
constexpr int kMaxGateChoices = 64;  // one lane each
constexpr int kMaxGateGroups = 64;
constexpr int kMaxGateGrid = 1 << 20;
struct GateSplit {
  int lane_bits, per;  // lanes of a group (their log2), experts of a lane
  bool fits;
};
struct GateArgs {
  const void* logits;
  int64_t ld;
  const float* bias;  // null: none
  void* chosen;
  float* weights;
  float* scores;  // null: not written
  int* load;      // null: not counted
  double scale;
  int tokens, experts, topk, groups, top_groups;
  int per_group;                   // (set by the launcher, as the splits
  GateSplit wide, middle, narrow;  // of 64, 32 and 16 lanes a token)
  bool lf32, i64, sigmoid, two_best, renormalize;
};
hipError_t launch_gate(GateArgs a, hipStream_t stream);
struct GateBwdArgs {
  const float* dweights;
  const void* chosen;
  const void* logits;
  int64_t ld;
  const float* dscores;  // null: none
  void* dlogits;
  int64_t ldd;
  double scale;
  int tokens, experts, topk;
  bool lf32, of32, i64, sigmoid, renormalize;
};
hipError_t launch_gate_backward(const GateBwdArgs& a, hipStream_t stream);

}  // namespace fp8q
