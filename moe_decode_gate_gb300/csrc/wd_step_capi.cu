// wd_step_capi.cu - the C-ABI of include/wd_step.h: argument checks on the host, and the launches.
#include <float.h>
#include <math.h>

#include "wd_step.cuh"

namespace {

bool aligned(const void* p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }
bool known(wd_dtype t) { return t == WD_BF16 || t == WD_FP16 || t == WD_FP32; }
uintptr_t size_of(wd_dtype t) { return t == WD_FP32 ? 4 : 2; }

}  // namespace

using wd::cuda_status;

extern "C" {

wd_status wd_rms_norm(const void* x, wd_dtype dtype, int64_t x_stride_token, int64_t x_stride_head, int64_t tokens,
                      int heads, int H, const void* weight, wd_dtype weight_dtype, const void* residual,
                      int64_t residual_stride_token, int64_t residual_stride_head, void* residual_out, float eps,
                      void* y, uint8_t* codes, uint8_t* scales, wd_stream_t stream) {
  if (!known(dtype) || (weight_dtype != dtype && weight_dtype != WD_FP32)) return WD_ERR_INVALID_ARG;
  if (tokens < 0 || heads < 1 || H < 1 || (!y && !codes) || !codes != !scales || (residual_out && !residual))
    return WD_ERR_INVALID_ARG;
  if (!(eps >= 1e-37f) || !(eps <= FLT_MAX)) return WD_ERR_INVALID_ARG;
  if (H > WD_NORM_MAX_H || tokens > INT32_MAX / heads || (codes && H % 32)) return WD_ERR_UNSUPPORTED_SHAPE;
  if (tokens == 0) return WD_OK;
  const uintptr_t n = size_of(dtype);
  if (!x || !aligned(x, n) || !aligned(weight, size_of(weight_dtype)) || !aligned(residual, n) ||
      !aligned(residual_out, n) || !aligned(y, n))
    return WD_ERR_INVALID_ARG;
  wd::NormArgs a{};
  a.x = x;
  a.x_token = x_stride_token;
  a.x_head = x_stride_head;
  a.residual = residual;
  a.residual_token = residual ? residual_stride_token : 0;
  a.residual_head = residual ? residual_stride_head : 0;
  a.weight = weight;
  a.weight_fp32 = weight_dtype == WD_FP32;
  a.residual_out = residual_out;
  a.y = y;
  a.codes = codes;
  a.scales = scales;
  a.rows = (int)(tokens * heads);
  a.heads = heads;
  a.H = H;
  a.eps = eps;
  return cuda_status(launch_rms_norm(a, dtype, reinterpret_cast<cudaStream_t>(stream)));
}

wd_status wd_route(const void* logits, wd_dtype dtype, int64_t stride_token, int64_t tokens, int E, int K,
                   wd_scores scores, const float* bias, int groups, int top_groups, int group_best, int renormalise,
                   float scale, int32_t* ids, float* weights, wd_stream_t stream) {
  if (!known(dtype) || (scores != WD_SOFTMAX && scores != WD_SIGMOID) || tokens < 0 || E < 1 || K < 1 || groups < 1 ||
      top_groups < 1 || top_groups > groups || group_best < 1 || group_best > 2 || !isfinite(scale))
    return WD_ERR_INVALID_ARG;
  if (E % groups || !wd::route_supported(E, groups) || K > WD_ROUTE_MAX_K || K > top_groups * (E / groups) ||
      tokens > (1 << 30))
    return WD_ERR_UNSUPPORTED_SHAPE;
  if (tokens == 0) return WD_OK;
  if (!logits || !ids || !weights || !aligned(logits, size_of(dtype)) || !aligned(bias, 4) || !aligned(ids, 4) ||
      !aligned(weights, 4))
    return WD_ERR_INVALID_ARG;
  wd::RouteArgs a{};
  a.logits = logits;
  a.stride = stride_token;
  a.bias = bias;
  a.ids = ids;
  a.weights = weights;
  a.tokens = (int)tokens;
  a.E = E;
  a.K = K;
  a.groups = top_groups == groups ? 1 : groups;  // all of them: no choice
  a.top_groups = top_groups == groups ? 1 : top_groups;
  a.group_best = E == groups ? 1 : group_best;  // of one expert: its key, which without a bias its logit orders
  a.sigmoid = scores == WD_SIGMOID;
  a.renormalise = renormalise != 0;
  a.scale = scale;
  return cuda_status(launch_route(a, dtype, reinterpret_cast<cudaStream_t>(stream)));
}

wd_status wd_adjust_logits(const void* logits, wd_dtype dtype, int64_t stride, int B, int V, const wd_history* history,
                           const float* repetition, const float* presence, const float* frequency,
                           const int32_t* bias_start, const int32_t* bias_ids, const float* bias_values, int biases,
                           const float* temperature, const int32_t* mask, int64_t mask_stride, void* out,
                           wd_dtype out_dtype, int64_t out_stride, wd_stream_t stream) {
  if (!known(dtype) || (out_dtype != dtype && out_dtype != WD_FP32) || B < 0 || V < 1 || biases < 0)
    return WD_ERR_INVALID_ARG;
  if (V > WD_LOGITS_MAX_V || B > 65535) return WD_ERR_UNSUPPORTED_SHAPE;
  if (B == 0) return WD_OK;
  if (!logits || !out || !aligned(logits, size_of(dtype)) || !aligned(out, size_of(out_dtype)) ||
      !aligned(repetition, 4) || !aligned(presence, 4) || !aligned(frequency, 4) || !aligned(temperature, 4) ||
      !aligned(mask, 4) || !aligned(bias_start, 4) || !aligned(bias_ids, 4) || !aligned(bias_values, 4))
    return WD_ERR_INVALID_ARG;
  if (bias_start ? !bias_ids || !bias_values : bias_ids || bias_values) return WD_ERR_INVALID_ARG;
  if (B > 1 && out_stride < V) return WD_ERR_INVALID_ARG;  // rows that overlap
  if (out == logits && (out_dtype != dtype || (B > 1 && out_stride != stride))) return WD_ERR_INVALID_ARG;
  wd::LogitsArgs a{};
  if (history && history->tokens) {
    if (!history->lengths || !aligned(history->tokens, 4) || !aligned(history->lengths, 4) ||
        !aligned(history->prompt_lengths, 4) || !aligned(history->seqs, 4) || history->slots < 1 ||
        history->columns < 0)
      return WD_ERR_INVALID_ARG;
    if (history->columns > WD_LOGITS_MAX_HISTORY) return WD_ERR_UNSUPPORTED_SHAPE;
    if (repetition || presence || frequency) a.history = *history;
  } else if (repetition || presence || frequency) {
    return WD_ERR_INVALID_ARG;
  }
  a.logits = logits;
  a.out = out;
  a.stride = stride;
  a.out_stride = out_stride;
  a.mask_stride = mask_stride;
  a.repetition = repetition;
  a.presence = presence;
  a.frequency = frequency;
  a.temperature = temperature;
  a.bias_start = biases ? bias_start : nullptr;
  a.bias_ids = bias_ids;
  a.bias_values = bias_values;
  a.mask = mask;
  a.B = B;
  a.V = V;
  a.biases = biases;
  return cuda_status(launch_adjust_logits(a, dtype, out_dtype, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
