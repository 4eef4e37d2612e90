// Internal launch interface of the block operators: the norm, scored routing,
// MXFP8 row gather and dense product around the routed experts.  Plain types
// only.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"

namespace moe {

struct NormArgs {
  const void* x;
  int x_fmt;
  int64_t ldx;
  const void* res;   // nullable
  int res_fmt;
  int64_t ldr;
  const void* gain;  // nullable: ones
  int gain_fmt;
  float eps;
  int T, H;
  void* sum;         // nullable; res_fmt
  int64_t lds;
  void* out;         // nullable
  int out_fmt;
  uint8_t* q;        // nullable, with q_scale
  uint8_t* q_scale;
};
cudaError_t launch_add_rmsnorm(const NormArgs& a, cudaStream_t s);

struct RouteArgs {
  const float* logits;
  int64_t ldl;
  const float* bias;  // nullable
  int T, E, k;
  int score;          // MOE_SCORE_*
  int n_group, topk_group, group_top;
  int renorm;
  float scale;
  int32_t* ids;
  float* w;
  uint32_t* dev_err;
};
cudaError_t launch_route_scored(const RouteArgs& a, cudaStream_t s);

cudaError_t launch_gather_mxfp8(const uint8_t* xq, const uint8_t* xs, const int32_t* inv, int T, int k, int H,
                                uint8_t* xp, uint8_t* xps, cudaStream_t s);

struct LinearArgs {
  const uint16_t* x;
  int64_t ldx;
  const uint16_t* w;
  int64_t ldw;
  const float* bias;  // nullable
  int act;            // MOE_ACT_*
  const void* res;    // nullable
  int res_fmt;
  int64_t ldr;
  int T, N, K;
  void* out;
  int out_fmt;
  int64_t ldo;
  uint32_t* dev_err;
  long long wait;     // bounded-wait limit in SM clock cycles
};
cudaError_t launch_linear(const LinearArgs& a, cudaStream_t s);
// on the tensor cores (linear_tc.cu): K, strides and addresses that TMA takes
bool linear_tc_supported(const LinearArgs& a);
cudaError_t launch_linear_tc(const LinearArgs& a, cudaStream_t s);
// T <= kFewTokens, same conditions (linear_few.cu)
constexpr int kFewTokens = 16;
cudaError_t launch_linear_few(const LinearArgs& a, cudaStream_t s);

}  // namespace moe
