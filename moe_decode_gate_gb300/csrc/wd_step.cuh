// wd_step.cuh - the launch interface between the kernels of include/wd_step.h
// and its C-ABI (wd_step_capi.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/wd_step.h"
#include "wd_launch.h"

namespace wd {

struct NormArgs {
  const void* x;
  long long x_token, x_head;  // strides in elements
  const void* residual;       // null: none
  long long residual_token, residual_head;
  const void* weight;  // null: ones
  bool weight_fp32, weight_aligned;  // (the second is launch_rms_norm's own)
  void *residual_out, *y;  // null: not wanted
  uint8_t *codes, *scales;
  int rows, heads, H;
  float eps;
};
cudaError_t launch_rms_norm(const NormArgs& a, wd_dtype dtype, cudaStream_t s);

struct RouteArgs {
  const void* logits;
  long long stride;
  const float* bias;
  int32_t* ids;
  float* weights;
  int tokens, E, K;
  int groups, top_groups, group_best;
  bool sigmoid, renormalise;
  float scale;
};
bool route_supported(int E, int groups);
cudaError_t launch_route(const RouteArgs& a, wd_dtype dtype, cudaStream_t s);

struct LogitsArgs {
  const void* logits;
  void* out;
  long long stride, out_stride, mask_stride;
  wd_history history;  // tokens null: no history
  const float *repetition, *presence, *frequency, *temperature;
  const int32_t *bias_start, *bias_ids;
  const float* bias_values;
  const int32_t* mask;
  int B, V, biases;
};
cudaError_t launch_adjust_logits(const LogitsArgs& a, wd_dtype dtype, wd_dtype out_dtype, cudaStream_t s);

}  // namespace wd
