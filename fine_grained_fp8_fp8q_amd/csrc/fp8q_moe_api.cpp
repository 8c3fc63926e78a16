// C-ABI entry points of the expert layer around the GEMMs (routing table,
// weighted sum and its gradient, SwiGLU's gradient, per-expert weight
// gradient): argument validation, device check and dispatch.  As in
// fp8q_api.cpp every check runs before anything touches the GPU.
#include "fp8q.h"
#include "fp8q_checks.h"
#include "fp8q_internal.h"

using namespace fp8q::checks;

namespace {
bool dtype_ok(int d) { return d == FP8Q_OUT_F32 || d == FP8Q_OUT_BF16; }
bool mode_ok(int m) { return m == FP8Q_SCALE_FREE || m == FP8Q_SCALE_POW2; }
// columns of a row that a workgroup goes over in steps (the step past the end fits in 32 bits)
constexpr int64_t kMaxRow = int64_t(1) << 30;
}  // namespace

extern "C" {

int64_t fp8q_moe_sort_workspace(int64_t tokens, int64_t topk, int32_t G) {
  if (!dim_ok(tokens) || !dim_ok(topk) || G <= 0 || tokens == 0 || topk == 0) return 0;
  if (topk > kMaxDim / tokens) return 0;
  const int blocks = fp8q::sort_blocks((int)(tokens * topk));
  return blocks > 1 ? (int64_t)blocks * G * (int64_t)sizeof(int32_t) : 0;
}

fp8q_status fp8q_moe_sort(const void* experts, int index_dtype, int64_t tokens, int64_t topk, int64_t ld_experts,
                          int64_t first_expert, int32_t G, int32_t align, int64_t rows_cap, int32_t* offsets,
                          int32_t* token, int32_t* row_of, void* workspace, int64_t workspace_bytes,
                          hipStream_t stream) {
  if (!dim_ok(tokens) || !dim_ok(topk) || !dim_ok(ld_experts) || !dim_ok(first_expert) ||
      !dim_ok(rows_cap) || G < 0 || align < 1 || workspace_bytes < 0)
    return FP8Q_ERR_INVALID_ARG;
  if (index_dtype != FP8Q_INDEX_I32 && index_dtype != FP8Q_INDEX_I64) return FP8Q_ERR_INVALID_ARG;
  if (G == 0) return FP8Q_OK;
  if (G > fp8q::kMaxSortGroups || ld_experts < topk || rows_cap % align) return FP8Q_ERR_SHAPE;
  const int64_t pairs = tokens > 0 && topk > kMaxDim / tokens ? kMaxDim + 1 : tokens * topk;
  if (pairs > kMaxDim || pairs + int64_t(G) * align > kMaxDim) return FP8Q_ERR_SHAPE;
  if (!offsets || (rows_cap > 0 && !token) || (pairs > 0 && (!experts || !row_of))) return FP8Q_ERR_INVALID_ARG;
  const int64_t need = fp8q_moe_sort_workspace(tokens, topk, G);
  if (need > 0 && (!workspace || workspace_bytes < need)) return FP8Q_ERR_INVALID_ARG;
  if (!aligned16(experts) || !aligned16(offsets) || !aligned16(token) || !aligned16(row_of) ||
      (need > 0 && !aligned16(workspace)))
    return FP8Q_ERR_ALIGN;
  if (fp8q_status st = check_device()) return st;
  return launched(fp8q::launch_moe_sort(experts, index_dtype == FP8Q_INDEX_I64, (int)pairs,
                                        topk > 0 ? (int)topk : 1, ld_experts, first_expert, (int)G, (int)align,
                                        (int)rows_cap, offsets, token, row_of, static_cast<int*>(workspace),
                                        stream));
}

fp8q_status fp8q_moe_combine(const void* y, int y_dtype, int64_t rows_cap, int64_t N, int64_t ld_y,
                             const int32_t* row_of, const float* weights, int64_t tokens, int64_t topk,
                             int out_dtype, void* out, int64_t ld_out, hipStream_t stream) {
  if (!dim_ok(rows_cap) || !dim_ok(N) || !dim_ok(ld_y) || !dim_ok(tokens) || !dim_ok(topk) || !dim_ok(ld_out))
    return FP8Q_ERR_INVALID_ARG;
  if (!dtype_ok(y_dtype) || !dtype_ok(out_dtype)) return FP8Q_ERR_INVALID_ARG;
  if (tokens == 0 || N == 0) return FP8Q_OK;
  if (!out || (topk > 0 && !row_of) || (rows_cap > 0 && !y)) return FP8Q_ERR_INVALID_ARG;
  if (ld_out < N || (rows_cap > 0 && ld_y < N)) return FP8Q_ERR_SHAPE;
  // one workgroup per token and at least 512 columns
  if (N >= kMaxRow || topk > kMaxDim / tokens || (N + 511) / 512 * tokens >= kMaxGroups) return FP8Q_ERR_SHAPE;
  if (!aligned16(out) || !aligned16(row_of) || !aligned16(weights) || !aligned16(y)) return FP8Q_ERR_ALIGN;
  if (fp8q_status st = check_device()) return st;
  return launched(fp8q::launch_moe_combine(y, y_dtype == FP8Q_OUT_F32, (int)rows_cap, (int)N, ld_y, row_of, weights,
                                           (int)tokens, (int)topk, out_dtype == FP8Q_OUT_F32, out, ld_out, stream));
}

fp8q_status fp8q_moe_combine_backward(const void* dout, int dout_dtype, int64_t tokens, int64_t N, int64_t ld_dout,
                                      const void* y, int y_dtype, int64_t rows_cap, int64_t ld_y,
                                      const int32_t* row_of, const float* weights, int64_t topk,
                                      const int32_t* token, void* dy_bf16, int64_t ld_dy, int scale_mode,
                                      uint8_t* dy_codes, int64_t ld_codes, float* dy_scales, float* dweights,
                                      hipStream_t stream) {
  if (!dim_ok(tokens) || !dim_ok(N) || !dim_ok(ld_dout) || !dim_ok(rows_cap) || !dim_ok(ld_y) || !dim_ok(topk) ||
      !dim_ok(ld_dy) || !dim_ok(ld_codes))
    return FP8Q_ERR_INVALID_ARG;
  if (!dtype_ok(dout_dtype) || !dtype_ok(y_dtype) || !mode_ok(scale_mode)) return FP8Q_ERR_INVALID_ARG;
  const bool rows_out = (dy_bf16 || dy_codes) && rows_cap > 0 && N > 0;
  const int64_t pairs = tokens > 0 && topk > kMaxDim / tokens ? kMaxDim + 1 : tokens * topk;
  if (!(rows_out && (pairs > 0 || token)) && !(dweights && pairs > 0)) return FP8Q_OK;
  if (pairs > 0 && (!row_of || (N > 0 && !dout))) return FP8Q_ERR_INVALID_ARG;
  if (dweights && rows_cap > 0 && N > 0 && !y) return FP8Q_ERR_INVALID_ARG;
  if (dy_codes && !dy_scales) return FP8Q_ERR_INVALID_ARG;
  if ((pairs > 0 && ld_dout < N) || (dweights && rows_cap > 0 && ld_y < N) || (rows_out && dy_bf16 && ld_dy < N) ||
      (rows_out && dy_codes && ld_codes < N))
    return FP8Q_ERR_SHAPE;
  // one workgroup per pair, and one per four rows to look for rows without one
  if (N >= kMaxRow || pairs + rows_cap / 4 + 1 >= kMaxGroups) return FP8Q_ERR_SHAPE;
  if (!aligned16(dout) || !aligned16(y) || !aligned16(row_of) || !aligned16(weights) || !aligned16(token) ||
      !aligned16(dy_bf16) || !aligned16(dy_codes) || !aligned16(dy_scales) || !aligned16(dweights))
    return FP8Q_ERR_ALIGN;
  if (fp8q_status st = check_device()) return st;
  return launched(fp8q::launch_moe_combine_backward(
      dout, dout_dtype == FP8Q_OUT_F32, (int)tokens, (int)N, ld_dout, dweights ? y : nullptr, y_dtype == FP8Q_OUT_F32,
      (int)rows_cap, ld_y, row_of, weights, (int)topk, token, static_cast<uint16_t*>(dy_bf16), ld_dy,
      scale_mode == FP8Q_SCALE_POW2, dy_codes, ld_codes, dy_scales, dweights, stream));
}

fp8q_status fp8q_swiglu_backward(const void* x, const float* x_scales, int64_t rows, int64_t inter, int64_t ld_x,
                                 const void* dy_bf16, int64_t ld_dy, void* dx_bf16, int64_t ld_dx, int scale_mode,
                                 uint8_t* dx_codes, int64_t ld_codes, float* dx_scales, void* y_bf16, int64_t ld_y,
                                 hipStream_t stream) {
  if (!dim_ok(rows) || !dim_ok(inter) || !dim_ok(ld_x) || !dim_ok(ld_dy) || !dim_ok(ld_dx) || !dim_ok(ld_codes) ||
      !dim_ok(ld_y))
    return FP8Q_ERR_INVALID_ARG;
  if (!mode_ok(scale_mode)) return FP8Q_ERR_INVALID_ARG;
  if (rows == 0 || inter == 0) return FP8Q_OK;
  if (!x || !dy_bf16 || (!dx_bf16 && !dx_codes && !y_bf16) || (dx_codes && !dx_scales)) return FP8Q_ERR_INVALID_ARG;
  if (ld_x < 2 * inter || ld_dy < inter || (dx_bf16 && ld_dx < 2 * inter) || (dx_codes && ld_codes < 2 * inter) ||
      (y_bf16 && ld_y < inter))
    return FP8Q_ERR_SHAPE;
  if ((x_scales || dx_codes) && inter % 128) return FP8Q_ERR_SHAPE;
  if (rows * ((inter + 127) / 128) >= 16 * (kMaxGroups - 1)) return FP8Q_ERR_SHAPE;  // 16 tiles a workgroup
  if (!aligned16(x) || !aligned16(x_scales) || !aligned16(dy_bf16) || !aligned16(dx_bf16) || !aligned16(dx_codes) ||
      !aligned16(dx_scales) || !aligned16(y_bf16))
    return FP8Q_ERR_ALIGN;
  if (fp8q_status st = check_device()) return st;
  return launched(fp8q::launch_swiglu_backward(
      x, x_scales, (int)rows, (int)inter, ld_x, static_cast<const uint16_t*>(dy_bf16), ld_dy,
      static_cast<uint16_t*>(dx_bf16), ld_dx, scale_mode == FP8Q_SCALE_POW2, dx_codes, ld_codes, dx_scales,
      static_cast<uint16_t*>(y_bf16), ld_y, stream));
}

fp8q_status fp8q_grouped_wgrad_ex(const uint8_t* dy_t, const float* dy_scales, const uint8_t* x_t,
                                  const float* x_scales, const int32_t* offsets, int32_t G, int64_t rows_cap,
                                  int64_t Nout, int64_t Kin, int acc, float* dw, int64_t ld_dw,
                                  hipStream_t stream) {
  if (G < 0 || !dim_ok(rows_cap) || !dim_ok(Nout) || !dim_ok(Kin) || !dim_ok(ld_dw)) return FP8Q_ERR_INVALID_ARG;
  if (!acc_ok(acc)) return FP8Q_ERR_INVALID_ARG;
  if (G == 0 || Nout == 0 || Kin == 0) return FP8Q_OK;
  if (!offsets) return FP8Q_ERR_INVALID_ARG;
  if (fp8q_status st = check_gemm_common(rows_cap, FP8Q_OUT_F32, dw, ld_dw, Kin)) return st;
  // one workgroup of 256 threads per 128 x 128 outputs, and eight regions of
  // whole tiles: at most seven rows and columns of them more
  const int64_t tiles = ((Nout + 127) / 128 + 7) * ((Kin + 127) / 128 + 7);
  // (the offsets of a tile's 256 rows, past the operand's last included, fit in 32 bits)
  if (rows_cap >= int64_t(1) << 24) return FP8Q_ERR_SHAPE;
  if (Nout * rows_cap >= kMaxOperandBytes || Kin * rows_cap >= kMaxOperandBytes || tiles >= kMaxGroups ||
      tiles * G >= kMaxGroups)
    return FP8Q_ERR_SHAPE;
  if (rows_cap > 0) {
    if (!dy_t || !dy_scales || !x_t || !x_scales) return FP8Q_ERR_INVALID_ARG;
    if (!aligned16(dy_t) || !aligned16(x_t) || !aligned16(dy_scales) || !aligned16(x_scales)) return FP8Q_ERR_ALIGN;
  }
  if (!aligned16(offsets)) return FP8Q_ERR_ALIGN;
  if (fp8q_status st = check_device()) return st;
  return launched(fp8q::launch_grouped_wgrad(dy_t, dy_scales, x_t, x_scales, offsets, (int)G, (int)rows_cap,
                                             (int)Nout, (int)Kin, acc, dw, ld_dw, stream));
}

fp8q_status fp8q_grouped_wgrad(const uint8_t* dy_t, const float* dy_scales, const uint8_t* x_t,
                               const float* x_scales, const int32_t* offsets, int32_t G, int64_t rows_cap,
                               int64_t Nout, int64_t Kin, float* dw, int64_t ld_dw, hipStream_t stream) {
  return fp8q_grouped_wgrad_ex(dy_t, dy_scales, x_t, x_scales, offsets, G, rows_cap, Nout, Kin, FP8Q_ACC_FP32, dw,
                               ld_dw, stream);
}

}  // extern "C"
