// C-ABI entry points of the step between a block's linear layers (residual
// addition with RMS norm and quantization, its gradient, token-axis tiles of
// the normalised rows, the router's choice and its gradient): argument
// validation, device check and dispatch.  As in fp8q_api.cpp every check runs
// before anything touches the GPU.
#include "fp8q.h"
#include "fp8q_checks.h"
#include "fp8q_internal.h"

using namespace fp8q::checks;

namespace {
bool dtype_ok(int d) { return d == FP8Q_OUT_F32 || d == FP8Q_OUT_BF16; }
bool mode_ok(int m) { return m == FP8Q_SCALE_FREE || m == FP8Q_SCALE_POW2; }
// columns of a row that a workgroup goes over in steps (the step past the end fits in 32 bits)
constexpr int64_t kMaxRow = int64_t(1) << 30;
// (NaN and infinities leave NaN)
bool is_finite(double v) { return v - v == 0.0; }
}  // namespace

extern "C" {

fp8q_status fp8q_rmsnorm_quantize(const void* x, int x_dtype, int64_t rows, int64_t N, int64_t ld_x, const void* residual,
                                  int stream_dtype, int64_t ld_residual, void* h, int64_t ld_h, const void* weight,
                                  int weight_dtype, double eps, void* y_bf16, int64_t ld_y, int scale_mode, uint8_t* codes,
                                  int64_t ld_codes, float* scales, float* rstd, hipStream_t stream) {
  if (!dim_ok(rows) || !dim_ok(N) || !dim_ok(ld_x) || !dim_ok(ld_residual) || !dim_ok(ld_h) || !dim_ok(ld_y) || !dim_ok(ld_codes))
    return FP8Q_ERR_INVALID_ARG;
  if (!dtype_ok(x_dtype) || !dtype_ok(stream_dtype) || !dtype_ok(weight_dtype) || !mode_ok(scale_mode)) return FP8Q_ERR_INVALID_ARG;
  if (!is_finite(eps) || !(eps > 0.0)) return FP8Q_ERR_INVALID_ARG;
  if (rows == 0 || (N == 0 && !rstd)) return FP8Q_OK;
  if (!h && !y_bf16 && !codes && !rstd) return FP8Q_ERR_INVALID_ARG;
  if (N > 0) {
    if (!x || !weight || (h && !residual) || (codes && !scales)) return FP8Q_ERR_INVALID_ARG;
    if (N >= kMaxRow || ld_x < N || (residual && ld_residual < N) || (h && ld_h < N) || (y_bf16 && ld_y < N) || (codes && ld_codes < N))
      return FP8Q_ERR_SHAPE;
    // over its own input the stream is written element by element; at another
    // stride it would overwrite rows that are still to be read
    if (h && h == residual && ld_h != ld_residual && rows > 1) return FP8Q_ERR_SHAPE;
  }
  if (!aligned16(x) || !aligned16(residual) || !aligned16(h) || !aligned16(weight) || !aligned16(y_bf16) || !aligned16(codes) ||
      !aligned16(scales) || !aligned16(rstd))
    return FP8Q_ERR_ALIGN;
  if (fp8q_status st = check_device()) return st;
  fp8q::NormArgs a{};
  a.x = x; a.ldx = ld_x; a.res = residual; a.ldr = ld_residual; a.h = h; a.ldh = ld_h; a.weight = weight;
  a.y = static_cast<uint16_t*>(y_bf16); a.ldy = ld_y; a.codes = codes; a.ldc = ld_codes; a.scales = scales; a.rstd = rstd;
  a.eps = eps; a.inv_n = N > 0 ? 1.0 / (double)N : 0.0; a.rows = (int)rows; a.n = (int)N;
  a.xf32 = x_dtype == FP8Q_OUT_F32; a.sf32 = stream_dtype == FP8Q_OUT_F32; a.wf32 = weight_dtype == FP8Q_OUT_F32;
  a.pow2 = scale_mode == FP8Q_SCALE_POW2;
  return launched(fp8q::launch_norm(a, stream));
}

int64_t fp8q_rmsnorm_backward_workspace(int64_t rows, int64_t N) {
  if (!dim_ok(rows) || !dim_ok(N) || N >= kMaxRow || rows == 0 || N == 0) return 0;
  return fp8q::norm_bwd_blocks((int)rows, (int)N) * fp8q::norm_partial_ld((int)N) * (int64_t)sizeof(float);
}

fp8q_status fp8q_rmsnorm_backward(const void* dy, int dy_dtype, int64_t rows, int64_t N, int64_t ld_dy, const void* h, int h_dtype,
                                  int64_t ld_h, const float* rstd, const void* weight, int weight_dtype, const void* dresidual,
                                  int64_t ld_dresidual, void* dx, int dx_dtype, int64_t ld_dx, int scale_mode, uint8_t* dx_codes,
                                  int64_t ld_codes, float* dx_scales, float* dweight, void* workspace, int64_t workspace_bytes,
                                  hipStream_t stream) {
  if (!dim_ok(rows) || !dim_ok(N) || !dim_ok(ld_dy) || !dim_ok(ld_h) || !dim_ok(ld_dresidual) || !dim_ok(ld_dx) || !dim_ok(ld_codes) ||
      workspace_bytes < 0)
    return FP8Q_ERR_INVALID_ARG;
  if (!dtype_ok(dy_dtype) || !dtype_ok(h_dtype) || !dtype_ok(weight_dtype) || !dtype_ok(dx_dtype) || !mode_ok(scale_mode))
    return FP8Q_ERR_INVALID_ARG;
  if (N == 0 || (rows == 0 && !dweight)) return FP8Q_OK;
  if (!dx && !dx_codes && !dweight) return FP8Q_ERR_INVALID_ARG;
  if (rows > 0 && (!dy || !h || !rstd || ((dx || dx_codes) && !weight) || (dx_codes && !dx_scales))) return FP8Q_ERR_INVALID_ARG;
  if (N >= kMaxRow || (rows > 0 && (ld_dy < N || ld_h < N || (dresidual && ld_dresidual < N) || (dx && ld_dx < N) || (dx_codes && ld_codes < N))))
    return FP8Q_ERR_SHAPE;
  // (as the stream over its own input: at another stride dx would overwrite rows of dresidual that are still to be read)
  if (dx && dx == dresidual && ld_dx != ld_dresidual && rows > 1) return FP8Q_ERR_SHAPE;
  const int64_t need = dweight ? fp8q_rmsnorm_backward_workspace(rows, N) : 0;
  if (need > 0 && (!workspace || workspace_bytes < need)) return FP8Q_ERR_INVALID_ARG;
  if (!aligned16(dy) || !aligned16(h) || !aligned16(rstd) || !aligned16(weight) || !aligned16(dresidual) || !aligned16(dx) ||
      !aligned16(dx_codes) || !aligned16(dx_scales) || !aligned16(dweight) || (need > 0 && !aligned16(workspace)))
    return FP8Q_ERR_ALIGN;
  if (fp8q_status st = check_device()) return st;
  fp8q::NormBwdArgs a{};
  a.dy = dy; a.lddy = ld_dy; a.h = h; a.ldh = ld_h; a.rstd = rstd; a.weight = weight; a.dres = dresidual; a.lddr = ld_dresidual;
  a.dx = dx; a.lddx = ld_dx; a.codes = dx_codes; a.ldc = ld_codes; a.scales = dx_scales; a.dweight = dweight;
  a.partial = static_cast<float*>(workspace); a.inv_n = 1.0 / (double)N; a.rows = (int)rows; a.n = (int)N;
  a.df32 = dy_dtype == FP8Q_OUT_F32; a.hf32 = h_dtype == FP8Q_OUT_F32; a.wf32 = weight_dtype == FP8Q_OUT_F32;
  a.of32 = dx_dtype == FP8Q_OUT_F32; a.pow2 = scale_mode == FP8Q_SCALE_POW2;
  return launched(fp8q::launch_norm_backward(a, stream));
}

fp8q_status fp8q_rmsnorm_quantize_t(const void* h, int h_dtype, int64_t h_rows, int64_t N, int64_t ld_h, const float* rstd,
                                    const void* weight, int weight_dtype, const int32_t* index, int64_t rows, int scale_mode,
                                    uint8_t* codes_t, int64_t ld_codes_t, float* scales_t, hipStream_t stream) {
  if (!dim_ok(h_rows) || !dim_ok(N) || !dim_ok(ld_h) || !dim_ok(rows) || !dim_ok(ld_codes_t)) return FP8Q_ERR_INVALID_ARG;
  if (!dtype_ok(h_dtype) || !dtype_ok(weight_dtype) || !mode_ok(scale_mode)) return FP8Q_ERR_INVALID_ARG;
  if (rows == 0 || N == 0) return FP8Q_OK;
  if ((h_rows > 0 && (!h || !rstd)) || !weight || !codes_t || !scales_t) return FP8Q_ERR_INVALID_ARG;
  if (!index && rows != h_rows) return FP8Q_ERR_SHAPE;
  if ((h_rows > 0 && ld_h < N) || ld_codes_t < rows) return FP8Q_ERR_SHAPE;
  if (((rows + 127) / 128) * ((N + 63) / 64) >= kMaxGroups) return FP8Q_ERR_SHAPE;
  if (!aligned16(h) || !aligned16(rstd) || !aligned16(weight) || !aligned16(index) || !aligned16(codes_t) || !aligned16(scales_t))
    return FP8Q_ERR_ALIGN;
  if (fp8q_status st = check_device()) return st;
  fp8q::NormTokenArgs a{};
  a.h = h; a.ldh = ld_h; a.rstd = rstd; a.weight = weight; a.index = index; a.codes = codes_t; a.ldc = ld_codes_t; a.scales = scales_t;
  a.rows = (int)rows; a.src_rows = (int)h_rows; a.n = (int)N;
  a.hf32 = h_dtype == FP8Q_OUT_F32; a.wf32 = weight_dtype == FP8Q_OUT_F32; a.pow2 = scale_mode == FP8Q_SCALE_POW2;
  return launched(fp8q::launch_norm_token(a, stream));
}

static fp8q_status check_gate(int logits_dtype, int64_t tokens, int64_t E, int64_t ld, int score, int64_t topk, double scale, int index_dtype) {
  if (!dim_ok(tokens) || !dim_ok(E) || !dim_ok(ld) || !dim_ok(topk)) return FP8Q_ERR_INVALID_ARG;
  if (!dtype_ok(logits_dtype) || (score != FP8Q_SCORE_SOFTMAX && score != FP8Q_SCORE_SIGMOID) || !is_finite(scale)) return FP8Q_ERR_INVALID_ARG;
  if (index_dtype != FP8Q_INDEX_I32 && index_dtype != FP8Q_INDEX_I64) return FP8Q_ERR_INVALID_ARG;
  if (E > fp8q::kMaxGateExperts || topk > fp8q::kMaxGateChoices || topk > E || (tokens > 1 && ld < E)) return FP8Q_ERR_SHAPE;
  return FP8Q_OK;
}

fp8q_status fp8q_moe_route(const void* logits, int logits_dtype, int64_t tokens, int64_t E, int64_t ld_logits, const float* bias,
                           int score, int32_t groups, int32_t top_groups, int group_score, int64_t topk, int renormalize, double scale,
                           int index_dtype, void* experts, float* weights, float* scores, int32_t* load, hipStream_t stream) {
  if (fp8q_status st = check_gate(logits_dtype, tokens, E, ld_logits, score, topk, scale, index_dtype)) return st;
  if (group_score != FP8Q_GROUP_MAX && group_score != FP8Q_GROUP_TOP_TWO) return FP8Q_ERR_INVALID_ARG;
  if (groups < 1 || top_groups < 1) return FP8Q_ERR_INVALID_ARG;
  if (groups > fp8q::kMaxGateGroups || top_groups > groups || E % groups || topk > E / groups * top_groups) return FP8Q_ERR_SHAPE;
  if (tokens == 0 || E == 0 || (topk == 0 && !scores)) return FP8Q_OK;
  if (!logits || (topk > 0 && (!experts || !weights))) return FP8Q_ERR_INVALID_ARG;
  if (!aligned16(logits) || !aligned16(bias) || !aligned16(experts) || !aligned16(weights) || !aligned16(scores) || !aligned16(load))
    return FP8Q_ERR_ALIGN;
  if (fp8q_status st = check_device()) return st;
  fp8q::GateArgs a{};
  a.logits = logits; a.ld = ld_logits; a.bias = bias; a.chosen = experts; a.weights = weights; a.scores = scores; a.load = load;
  a.scale = scale; a.tokens = (int)tokens; a.experts = (int)E; a.topk = (int)topk; a.groups = groups; a.top_groups = top_groups;
  a.lf32 = logits_dtype == FP8Q_OUT_F32; a.i64 = index_dtype == FP8Q_INDEX_I64; a.sigmoid = score == FP8Q_SCORE_SIGMOID;
  a.two_best = group_score == FP8Q_GROUP_TOP_TWO; a.renormalize = renormalize != 0;
  return launched(fp8q::launch_gate(a, stream));
}

fp8q_status fp8q_moe_route_backward(const float* dweights, const void* experts, int index_dtype, int64_t tokens, int64_t topk,
                                    const void* logits, int logits_dtype, int64_t E, int64_t ld_logits, int score, int renormalize,
                                    double scale, const float* dscores, void* dlogits, int dlogits_dtype, int64_t ld_dlogits,
                                    hipStream_t stream) {
  if (fp8q_status st = check_gate(logits_dtype, tokens, E, ld_logits, score, topk, scale, index_dtype)) return st;
  if (!dim_ok(ld_dlogits) || !dtype_ok(dlogits_dtype)) return FP8Q_ERR_INVALID_ARG;
  if (tokens == 0 || E == 0) return FP8Q_OK;
  if (!logits || !dlogits || (topk > 0 && (!experts || !dweights))) return FP8Q_ERR_INVALID_ARG;
  if (tokens > 1 && ld_dlogits < E) return FP8Q_ERR_SHAPE;
  if (!aligned16(dweights) || !aligned16(experts) || !aligned16(logits) || !aligned16(dscores) || !aligned16(dlogits)) return FP8Q_ERR_ALIGN;
  if (fp8q_status st = check_device()) return st;
  fp8q::GateBwdArgs a{};
  a.dweights = dweights; a.chosen = experts; a.logits = logits; a.ld = ld_logits; a.dscores = dscores; a.dlogits = dlogits; a.ldd = ld_dlogits;
  a.scale = scale; a.tokens = (int)tokens; a.experts = (int)E; a.topk = (int)topk;
  a.lf32 = logits_dtype == FP8Q_OUT_F32; a.of32 = dlogits_dtype == FP8Q_OUT_F32; a.i64 = index_dtype == FP8Q_INDEX_I64;
  a.sigmoid = score == FP8Q_SCORE_SIGMOID; a.renormalize = renormalize != 0;
  return launched(fp8q::launch_gate_backward(a, stream));
}

}  // extern "C"
