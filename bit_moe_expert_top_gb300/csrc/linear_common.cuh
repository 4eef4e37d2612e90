// Epilogue arithmetic of moe_linear, shared by its kernels.
#pragma once
#include <stdint.h>

#include "block_ops.cuh"
#include "common.cuh"

namespace moe {

MOE_D float gelu_f32(float v) { return 0.5f * v * (1.0f + erff(v * 0.70710678118654752f)); }
MOE_D float swiglu_f32(float g, float u) { return silu_f32(g) * u; }

MOE_D float linear_act(float v, int act) {
  return act == MOE_ACT_SILU ? silu_f32(v) : (act == MOE_ACT_GELU ? gelu_f32(v) : v);
}

// out[t][n] = v + res[t][n], one rounding.
MOE_D void linear_store(const LinearArgs& a, int64_t t, int64_t n, float v) {
  if (a.res)
    v += a.res_fmt == MOE_FMT_F32 ? static_cast<const float*>(a.res)[t * a.ldr + n]
                                  : bf16_bits_to_f32(static_cast<const uint16_t*>(a.res)[t * a.ldr + n]);
  if (a.out_fmt == MOE_FMT_F32)
    static_cast<float*>(a.out)[t * a.ldo + n] = v;
  else
    static_cast<uint16_t*>(a.out)[t * a.ldo + n] = f32_to_bf16_rne(v);
}

}  // namespace moe
