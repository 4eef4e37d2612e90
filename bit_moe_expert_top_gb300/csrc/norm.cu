// Residual addition + root-mean-square norm, with an optional MXFP8 output.
#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"
#include "internal.cuh"

namespace moe {

namespace {

MOE_D float load_elem(const void* p, int fmt, int64_t i) {
  return fmt == MOE_FMT_F32 ? static_cast<const float*>(p)[i] : bf16_bits_to_f32(static_cast<const uint16_t*>(p)[i]);
}
MOE_D void store_elem(void* p, int fmt, int64_t i, float v) {
  if (fmt == MOE_FMT_F32)
    static_cast<float*>(p)[i] = v;
  else
    static_cast<uint16_t*>(p)[i] = f32_to_bf16_rne(v);
}

// One CTA per row, one element per thread and round: a warp's 32 elements
// are one MXFP8 block.  The row is read twice (sum of squares, then the
// outputs; the second time from cache).
__global__ void __launch_bounds__(256) add_rmsnorm_kernel(const NormArgs a) {
  __shared__ float part[8];
  pdl_wait();
  pdl_trigger();
  const int64_t t = blockIdx.x;
  const int tid = threadIdx.x, lane = tid & 31;
  float ss = 0.f;
  for (int i = tid; i < a.H; i += 256) {
    float y = load_elem(a.x, a.x_fmt, t * a.ldx + i);
    if (a.res) y += load_elem(a.res, a.res_fmt, t * a.ldr + i);
    ss = fmaf(y, y, ss);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
  if (lane == 0) part[tid >> 5] = ss;
  __syncthreads();
  ss = 0.f;
#pragma unroll
  for (int w = 0; w < 8; ++w) ss += part[w];
  const float inv = 1.0f / sqrtf(ss / static_cast<float>(a.H) + a.eps);
  for (int i0 = 0; i0 < a.H; i0 += 256) {
    const int i = i0 + tid;
    const bool ok = i < a.H;
    float n = 0.f;
    if (ok) {
      float y = load_elem(a.x, a.x_fmt, t * a.ldx + i);
      if (a.res) y += load_elem(a.res, a.res_fmt, t * a.ldr + i);
      if (a.sum) store_elem(a.sum, a.res_fmt, t * a.lds + i, y);
      n = y * inv;
      if (a.gain) n *= load_elem(a.gain, a.gain_fmt, i);
      if (a.out) store_elem(a.out, a.out_fmt, t * a.H + i, n);
    }
    if (a.q) {  // H % 32 == 0: a warp's block is whole or absent
      const float b = bf16_bits_to_f32(f32_to_bf16_rne(n));
      float amax = fabsf(b);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
      const int X = mx_scale_exp(amax);
      const uint16_t c = f32x2_to_e4m3x2(b * exp2i(-X), 0.f);
      if (ok) {
        a.q[t * a.H + i] = static_cast<uint8_t>(c);
        if (lane == 0) a.q_scale[t * (a.H / 32) + i / 32] = static_cast<uint8_t>(X + 127);
      }
    }
  }
}

}  // namespace

cudaError_t launch_add_rmsnorm(const NormArgs& a, cudaStream_t s) {
  return launch_pdl(add_rmsnorm_kernel, dim3(a.T), dim3(256), 0, s, a);
}

}  // namespace moe
