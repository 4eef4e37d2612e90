// Gather of MXFP8 token rows to the permuted rows of their experts.
#include <cuda_runtime.h>
#include <stdint.h>

#include "block_ops.cuh"
#include "common.cuh"
#include "internal.cuh"

namespace moe {

constexpr int kGatherThreads = 128;

// blockDim.x threads per token (short rows share a CTA): every 16-byte piece
// of the row is read once, up to four loads in flight per thread, and written
// to the k permuted rows of the token.  Bound by DRAM, nearly all of it
// writes: 167 us for 16384 tokens x 7168, k = 8 (6530 GB/s, 0.96 of the copy
// rate; 171 us with one piece at a time), 14.2 us for 16384 x 512 (17.0 with a
// CTA per token).
__global__ void __launch_bounds__(kGatherThreads) gather_mxfp8_kernel(const uint8_t* __restrict__ xq,
                                                                      const uint8_t* __restrict__ xs,
                                                                      const int32_t* __restrict__ inv, int T, int k,
                                                                      int H, uint8_t* __restrict__ xp,
                                                                      uint8_t* __restrict__ xps) {
  constexpr int U = 4;
  pdl_wait();
  pdl_trigger();
  const size_t t = static_cast<size_t>(blockIdx.x) * blockDim.y + threadIdx.y;
  if (t >= static_cast<size_t>(T)) return;
  const int32_t* iv = inv + t * k;
  const int n = H / 16, nb = H / 32, step = blockDim.x;
  const uint4* src = reinterpret_cast<const uint4*>(xq + t * H);
  for (int i0 = threadIdx.x; i0 < n; i0 += U * step) {
    uint4 v[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (i0 + u * step < n) v[u] = src[i0 + u * step];
    for (int j = 0; j < k; ++j) {
      const int p = iv[j];
      if (p < 0) continue;
      uint4* dst = reinterpret_cast<uint4*>(xp + static_cast<size_t>(p) * H);
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (i0 + u * step < n) dst[i0 + u * step] = v[u];
    }
  }
  for (int i = threadIdx.x; i < nb; i += step) {
    const uint8_t v = xs[t * nb + i];
    for (int j = 0; j < k; ++j) {
      const int p = iv[j];
      if (p >= 0) xps[static_cast<size_t>(p) * nb + i] = v;
    }
  }
}

cudaError_t launch_gather_mxfp8(const uint8_t* xq, const uint8_t* xs, const int32_t* inv, int T, int k, int H,
                                uint8_t* xp, uint8_t* xps, cudaStream_t s) {
  const int n = H / 16;
  const int half = (n + 63) / 64 * 32;  // two pieces a thread or more
  const int per = half < kGatherThreads ? half : kGatherThreads;
  const int rows = kGatherThreads / per;
  return launch_pdl(gather_mxfp8_kernel, dim3((T - 1) / rows + 1), dim3(per, rows), 0, s, xq, xs, inv, T, k, H, xp, xps);
}

}  // namespace moe
