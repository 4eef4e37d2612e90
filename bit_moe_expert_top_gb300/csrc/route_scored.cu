// Top-k routing on softmax or sigmoid scores with a balance bias and expert
// groups.
#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"
#include "internal.cuh"
#include "route_common.cuh"

namespace moe {

namespace {

// Two largest of a set, equal values counted as often as they occur.
struct Top2 {
  float a, b;
};
MOE_D Top2 top2_join(Top2 p, Top2 q) {
  return p.a >= q.a ? Top2{p.a, fmaxf(p.b, q.a)} : Top2{q.a, fmaxf(q.b, p.a)};
}

// One warp per token; scores s and selection scores c of its experts in
// shared memory.  Every selection is k rounds of a warp-wide maximum over
// 64-bit keys (route_key: value, then lowest index).
__global__ void __launch_bounds__(128) route_scored_kernel(const RouteArgs a) {
  extern __shared__ float sm[];
  pdl_wait();
  pdl_trigger();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int t = blockIdx.x * 4 + warp;
  if (t >= a.T) return;
  float* s = sm + warp * 2 * a.E;
  float* c = s + a.E;
  const float* row = a.logits + t * a.ldl;
  bool nan = false;

  float mx = -INFINITY;
  for (int e = lane; e < a.E; e += 32) {
    const float l = row[e];
    s[e] = l;
    if (l == l) mx = fmaxf(mx, l);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  float sum = 0.f;
  for (int e = lane; e < a.E; e += 32) {
    const float l = s[e];
    float v;
    if (a.score == MOE_SCORE_SIGMOID)
      v = 1.0f / (1.0f + expf(-l));
    else
      v = l == mx ? 1.0f : expf(l - mx);
    if (!(l > -INFINITY)) v = 0.f;  // masked, or NaN
    c[e] = v;
    sum += v;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  for (int e = lane; e < a.E; e += 32) {
    const float l = s[e];
    float v = c[e];
    if (a.score == MOE_SCORE_SOFTMAX && sum > 0.f) v = v / sum;
    float cc = v + (a.bias ? a.bias[e] : 0.f);
    if (l == -INFINITY) cc = -INFINITY;
    if (l != l) cc = l;
    nan |= (cc != cc);
    s[e] = v;
    c[e] = cc;
  }
  __syncwarp();
  if (__any_sync(0xffffffffu, nan) && lane == 0) set_err(a.dev_err, MOE_DEVERR_NAN_LOGIT);

  // groups: lane g holds group g's key
  const int per = a.E / a.n_group;
  uint32_t kept = 0xffffffffu;
  if (a.n_group > 1) {
    uint64_t gkey = 0;
    for (int g = 0; g < a.n_group; ++g) {
      Top2 m{-INFINITY, -INFINITY};
      for (int i = lane; i < per; i += 32) {
        const float v = c[g * per + i];
        if (v == v) m = top2_join(m, Top2{v, -INFINITY});
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1)
        m = top2_join(m, Top2{__shfl_xor_sync(0xffffffffu, m.a, o), __shfl_xor_sync(0xffffffffu, m.b, o)});
      if (lane == g) gkey = route_key(a.group_top == 2 ? m.a + m.b : m.a, g);
    }
    kept = 0;
    for (int j = 0; j < a.topk_group; ++j) {
      uint64_t m = gkey;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        const uint64_t other = __shfl_xor_sync(0xffffffffu, m, o);
        m = other > m ? other : m;
      }
      const int g = static_cast<int>(0xffffffffu - static_cast<uint32_t>(m));
      kept |= 1u << g;
      if (lane == g) gkey = 0;
    }
  }

  uint64_t mine = 0;  // lane j keeps slot j
  uint64_t last = ~0ull;
  for (int j = 0; j < a.k; ++j) {
    uint64_t m = 0;  // largest key below the last one taken
    for (int e = lane; e < a.E; e += 32) {
      if (!((kept >> (e / per)) & 1)) continue;
      const uint64_t key = route_key(c[e], e);
      if (key < last && key > m) m = key;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const uint64_t other = __shfl_xor_sync(0xffffffffu, m, o);
      m = other > m ? other : m;
    }
    if (lane == j) mine = m;
    last = m;
  }
  const int id = static_cast<int>(0xffffffffu - static_cast<uint32_t>(mine));
  float w = lane < a.k ? s[id] : 0.f;
  if (a.renorm) {
    float tot = 0.f;
    for (int j = 0; j < a.k; ++j) tot += __shfl_sync(0xffffffffu, w, j);
    w = tot > 0.f ? w / tot : 0.f;
  }
  if (lane < a.k) {
    a.ids[static_cast<size_t>(t) * a.k + lane] = id;
    a.w[static_cast<size_t>(t) * a.k + lane] = w * a.scale;
  }
}

}  // namespace

cudaError_t launch_route_scored(const RouteArgs& a, cudaStream_t s) {
  return launch_pdl(route_scored_kernel, dim3((a.T + 3) / 4), dim3(128), static_cast<size_t>(8) * a.E * sizeof(float), s,
                    a);
}

}  // namespace moe
