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

}  // namespace fp8q
