// Gather of MXFP8 token rows to the permuted rows of their experts.
#include <cuda_runtime.h>
#include <stdint.h>

#include "block_ops.cuh"
#include "common.cuh"
#include "internal.cuh"

namespace moe {

// One CTA per token: every 16-byte piece of the row is read once and written
// to the k permuted rows of the token.
__global__ void __launch_bounds__(128) gather_mxfp8_kernel(const uint8_t* __restrict__ xq,
                                                           const uint8_t* __restrict__ xs,
                                                           const int32_t* __restrict__ inv, int k, int H,
                                                           uint8_t* __restrict__ xp, uint8_t* __restrict__ xps) {
  pdl_wait();
  pdl_trigger();
  const size_t t = blockIdx.x;
  const int32_t* iv = inv + t * k;
  for (int i = threadIdx.x; i < H / 16; i += 128) {
    const uint4 v = reinterpret_cast<const uint4*>(xq + t * H)[i];
    for (int j = 0; j < k; ++j) {
      const int p = iv[j];
      if (p >= 0) reinterpret_cast<uint4*>(xp + static_cast<size_t>(p) * H)[i] = v;
    }
  }
  const int nb = H / 32;
  for (int i = threadIdx.x; i < nb; i += 128) {
    const uint8_t v = xs[t * nb + i];
    for (int j = 0; j < k; ++j) {
      const int p = iv[j];
      if (p >= 0) xps[static_cast<size_t>(p) * nb + i] = v;
    }
  }
}

cudaError_t launch_gather_mxfp8(const uint8_t* xq, const uint8_t* xs, const int32_t* inv, int T, int k, int H,
                                uint8_t* xp, uint8_t* xps, cudaStream_t s) {
  return launch_pdl(gather_mxfp8_kernel, dim3(T), dim3(128), 0, s, xq, xs, inv, k, H, xp, xps);
}

}  // namespace moe
