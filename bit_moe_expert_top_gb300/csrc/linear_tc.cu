// Dense matrix product with bias, activation and residual in its epilogue, on
// the tensor cores (tcgen05, bf16 operands, fp32 accumulators in TMEM).
//
// A tile is 128 weight rows per CTA (TMEM lane = weight row = output feature)
// times NT tokens (TMEM column = token): D = W_tile . X_tile^T, so a warp of
// the epilogue holds 32 consecutive outputs of one token in every register
// and reads and writes them as one coalesced piece.  CG = 2: a pair of CTAs
// forms one 256-row MMA (cta_group::2), each holding its own 128 weight rows
// and half of the tile's tokens.
//
// SwiGLU: the tile's 128 rows are four groups of 16 gate rows followed by the
// matching 16 up rows (one 4-dimensional TMA box), so gate and up of one
// output sit 16 lanes apart in one warp and meet by a shuffle.
//
//   warp 0      TMA: per stage 64 elements of K of the weight and token tiles,
//               128-byte swizzle
//   warp 1      MMA issue (CG = 2: in the pair's first CTA) and TMEM allocation
//   warps 2-9   epilogue, two warps per TMEM lane quarter, each on its half of
//               the tile's columns
//
// The accumulator is double-buffered in TMEM.  For fp32 outputs the MMA
// accumulates at most P.chunk stages (512 elements of K) into one buffer;
// the epilogue warps add the buffers into a running sum, also in TMEM, with
// rounding to nearest: the tensor core truncates when it accumulates, which
// at K = 4096 alone would put the result 4e-6 off.
//
// split > 1 (CG = 1): the CTAs of a cluster take consecutive parts of K for
// one tile, leave their partial sums in shared memory, and each adds up its
// share of the columns over the cluster in rank order (no atomics).
//
// Every mbarrier wait is bounded (MOE_DEVERR_TIMEOUT).
#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"
#include "internal.cuh"
#include "linear_common.cuh"
#include "tc_common.cuh"

namespace moe {

namespace {

constexpr int kThreads = 320;
constexpr int kBK = 64;          // K elements per stage: one 128-byte swizzled row
constexpr int kATile = 128 * kBK * 2;
constexpr int kChunk = 8;        // stages per accumulation of an fp32 output (512 of K)
constexpr int kCtl = 1024;       // barriers and flags
constexpr int kSmemMax = 232448;

template <int CG, int NT>
constexpr int stage_bytes() { return kATile + NT / CG * kBK * 2; }
template <int CG, int NT>
constexpr int num_stages() {
  constexpr int n = (kSmemMax - kCtl - 1024) / stage_bytes<CG, NT>();
  return n < 12 ? n : 12;
}
template <int CG, int NT>
constexpr int smem_bytes() { return kCtl + 1024 + num_stages<CG, NT>() * stage_bytes<CG, NT>(); }

struct TcParams {
  LinearArgs a;
  int mblocks, tblocks, tiles;  // row blocks (128 * CG rows), token blocks, their product
  int kblocks, chunk;           // stages of K, stages per accumulation
  int split;                    // CTAs of a cluster along K (CG = 1)
  int mfast;                    // neighbouring tiles share their tokens (1) or their weight rows (0)
};

// ------------------------------------------------------------------ PTX of CTA pairs and clusters
MOE_D uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
MOE_D void cluster_sync_all() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
MOE_D uint32_t map_rank(uint32_t saddr, uint32_t rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(saddr), "r"(rank));
  return r;
}
MOE_D float ld_cluster_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}
MOE_D void mbar_arrive_remote(uint32_t addr) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(addr) : "memory");
}
// As mbar_wait, with the acquire at cluster scope (arrivals of the peer CTA).
MOE_D bool mbar_wait_cluster(uint64_t* bar, uint32_t parity, long long limit) {
  const long long t0 = clock64();
  for (;;) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    if (ok) return true;
    if (clock64() - t0 > limit) return false;
  }
}

template <int CG>
MOE_D void tma_2d(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
  if (CG == 2)
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], "
        "[%4];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(bar)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
            dst),
        "l"(map), "r"(x), "r"(y), "r"(bar)
        : "memory");
}
template <int CG>
MOE_D void tma_4d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, int w, uint32_t bar) {
  if (CG == 2)
    asm volatile(
        "cp.async.bulk.tensor.4d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, "
        "%4, %5}], [%6];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
        "[%6];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
        : "memory");
}

template <int CG>
MOE_D void mma_ss(uint32_t d, uint64_t ad, uint64_t bd, uint32_t idesc, uint32_t accum) {
  if (CG == 2)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(ad), "l"(bd), "r"(idesc), "r"(accum)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(ad), "l"(bd), "r"(idesc), "r"(accum)
        : "memory");
}
// Arrives on the barrier (CG = 2: on that of both CTAs) when the MMAs issued so far are done.
template <int CG>
MOE_D void mma_commit(uint64_t* bar) {
  if (CG == 2)
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smem_u32(bar)),
        "h"(static_cast<uint16_t>(3))
        : "memory");
  else
    umma_commit_to(bar);
}
template <int CG>
MOE_D void tm_alloc_cg(uint32_t* dst, uint32_t ncols) {
  if (CG == 2)
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(dst)), "r"(ncols)
                 : "memory");
  else
    tm_alloc(dst, ncols);
}
template <int CG>
MOE_D void tm_free_cg(uint32_t taddr, uint32_t ncols) {
  if (CG == 2)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
  else
    tm_dealloc(taddr, ncols);
}
template <int CG>
MOE_D void tm_relinquish_cg() {
  if (CG == 2)
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  else
    tm_relinquish();
}

// CW consecutive TMEM columns of this thread's lane.
MOE_D void tm_ld8(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
}
MOE_D void tm_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
MOE_D void tm_st8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
MOE_D void tm_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
          taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
MOE_D void tm_ld(uint32_t t, uint32_t (&r)[8]) { tm_ld8(t, r); }
MOE_D void tm_ld(uint32_t t, uint32_t (&r)[16]) { tm_ld16(t, r); }
MOE_D void tm_ld(uint32_t t, uint32_t (&r)[32]) { tm_ld32(t, r); }
MOE_D void tm_st(uint32_t t, const uint32_t (&r)[8]) { tm_st8(t, r); }
MOE_D void tm_st(uint32_t t, const uint32_t (&r)[16]) { tm_st16(t, r); }
MOE_D void tm_st(uint32_t t, const uint32_t (&r)[32]) { tm_st32(t, r); }

// ------------------------------------------------------------------ epilogue
// M outputs of this lane, at rows (tokens) t0, t0 + step, ...: the residual is
// added and the sums are stored.  cnt > 0 of them are inside T.  The loads
// are issued together (rows past the end read the last one again): with a
// branch per load each waited for its own and the epilogue set the pace (838
// us instead of 342 us at T 16384, N 7168, K 2048 with a bf16 residual).
template <int M>
MOE_D void emit_rows(const LinearArgs& a, float (&v)[M], int64_t t0, int step, int cnt, int64_t n) {
  if (a.res) {
    const int64_t ld = a.ldr * step;
    if (a.res_fmt == MOE_FMT_F32) {
      const float* p = static_cast<const float*>(a.res) + t0 * a.ldr + n;
      float r[M];
#pragma unroll
      for (int c = 0; c < M; ++c) r[c] = p[(c < cnt ? c : cnt - 1) * ld];
#pragma unroll
      for (int c = 0; c < M; ++c) v[c] += r[c];
    } else {
      const uint16_t* p = static_cast<const uint16_t*>(a.res) + t0 * a.ldr + n;
      uint16_t r[M];
#pragma unroll
      for (int c = 0; c < M; ++c) r[c] = p[(c < cnt ? c : cnt - 1) * ld];
#pragma unroll
      for (int c = 0; c < M; ++c) v[c] += bf16_bits_to_f32(r[c]);
    }
  }
  const int64_t ld = a.ldo * step;
  if (a.out_fmt == MOE_FMT_F32) {
    float* p = static_cast<float*>(a.out) + t0 * a.ldo + n;
#pragma unroll
    for (int c = 0; c < M; ++c)
      if (c < cnt) p[c * ld] = v[c];
  } else {
    uint16_t* p = static_cast<uint16_t*>(a.out) + t0 * a.ldo + n;
#pragma unroll
    for (int c = 0; c < M; ++c)
      if (c < cnt) p[c * ld] = f32_to_bf16_rne(v[c]);
  }
}

// This lane's outputs of CW columns (tokens t0 ..): bias, activation,
// residual, store.  n: the lane's output feature (nok: inside N).
template <int CW>
MOE_D void emit(const LinearArgs& a, float (&v)[CW], int64_t t0, int64_t n, bool nok, int lane) {
  if (t0 >= a.T) return;  // warp-uniform
  const int nc = a.T - t0 < CW ? static_cast<int>(a.T - t0) : CW;
  if (a.act == MOE_ACT_SWIGLU) {
    // lanes 0-15: gate rows, lanes 16-31: the up rows of the same outputs.
    // Of columns (c, c + 1) the low half finishes c, the high half c + 1.
    const int hi = lane >> 4;
    float bg = 0.f, bu = 0.f;
    if (a.bias && nok) {
      bg = __ldg(a.bias + n);
      bu = __ldg(a.bias + a.N + n);
    }
    float u[CW / 2];
#pragma unroll
    for (int c = 0; c < CW; c += 2) {
      const float other = __shfl_xor_sync(0xffffffffu, hi ? v[c] : v[c + 1], 16);
      u[c / 2] = swiglu_f32((hi ? other : v[c]) + bg, (hi ? v[c + 1] : other) + bu);
    }
    const int cnt = (nc - hi + 1) / 2;
    if (nok && cnt > 0) emit_rows<CW / 2>(a, u, t0 + hi, 2, cnt, n);
    return;
  }
  const float b = (a.bias && nok) ? __ldg(a.bias + n) : 0.f;
#pragma unroll
  for (int c = 0; c < CW; ++c) v[c] += b;
  if (a.act == MOE_ACT_SILU) {
#pragma unroll
    for (int c = 0; c < CW; ++c) v[c] = silu_f32(v[c]);
  } else if (a.act == MOE_ACT_GELU) {
#pragma unroll
    for (int c = 0; c < CW; ++c) v[c] = gelu_f32(v[c]);
  }
  if (nok) emit_rows<CW>(a, v, t0, 1, nc, n);
}

template <int CG, int NT>
__global__ void __launch_bounds__(kThreads, 1) linear_tc_kernel(const __grid_constant__ CUtensorMap tm_w,
                                                                const __grid_constant__ CUtensorMap tm_x,
                                                                const __grid_constant__ TcParams P) {
  constexpr int kStage = stage_bytes<CG, NT>();
  constexpr int ST = num_stages<CG, NT>();
  constexpr uint32_t kCols = NT >= 128 ? 512 : 4 * NT;  // two accumulators and (NT <= 128) the running sum
  constexpr int CW = NT / 2 < 32 ? NT / 2 : 32;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint64_t* full = reinterpret_cast<uint64_t*>(smem);  // [ST] stage landed (CG = 2: both CTAs' halves, on the first)
  uint64_t* empty = full + ST;                          // [ST] the stage's MMAs done
  uint64_t* acc_full = empty + ST;                      // [2]
  uint64_t* acc_empty = acc_full + 2;                   // [2] read by 8 warps per CTA (CG = 2: on the first)
  uint32_t* tmem_s = reinterpret_cast<uint32_t*>(acc_empty + 2);
  const uint32_t base = smem_u32(smem);
  const uint32_t tiles_off = ((base + kCtl + 1023u) & ~1023u) - base;
  uint8_t* stages = smem + tiles_off;

  const LinearArgs& a = P.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const bool glu = a.act == MOE_ACT_SWIGLU;
  const uint32_t rank = (CG == 2 || P.split > 1) ? cluster_rank() : 0;
  const int csize = CG == 2 ? 2 : P.split;
  const int unit = blockIdx.x / csize, units = gridDim.x / csize;  // the cluster walks tiles unit, unit + units, ...
  const int kb0 = CG == 2 ? 0 : static_cast<int>(static_cast<int64_t>(P.kblocks) * rank / P.split);
  const int kb1 = CG == 2 ? P.kblocks : static_cast<int>(static_cast<int64_t>(P.kblocks) * (rank + 1) / P.split);
  const int nchunk = (kb1 - kb0 + P.chunk - 1) / P.chunk;

  if (tid == 0) {
    for (int i = 0; i < ST; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&acc_full[i], 1);
      mbar_init(&acc_empty[i], 8 * CG);
    }
    fence_barrier_init();
  }
  if (warp == 1) {
    tm_alloc_cg<CG>(tmem_s, kCols);
    tm_relinquish_cg<CG>();
  }
  tm_fence_before();
  __syncthreads();
  if (csize > 1) cluster_sync_all();
  tm_fence_after();
  const uint32_t tmem = *tmem_s;
  pdl_wait();
  pdl_trigger();

  auto tile_of = [&](int tile, int& mb, int& tb) {
    if (P.mfast) {
      tb = tile / P.mblocks;
      mb = tile - tb * P.mblocks;
    } else {
      mb = tile / P.tblocks;
      tb = tile - mb * P.tblocks;
    }
  };

  if (warp == 0 && lane == 0) {  // ---------------------------------------- TMA
    int it = 0;
    bool ok = true;
    for (int tile = unit; ok && tile < P.tiles; tile += units) {
      int mb, tb;
      tile_of(tile, mb, tb);
      const int rb = mb * CG + (CG == 2 ? static_cast<int>(rank) : 0);          // 128-row block of this CTA
      const int tok = tb * NT + (CG == 2 ? static_cast<int>(rank) * (NT / 2) : 0);  // its first token
      for (int kb = kb0; kb < kb1; ++kb, ++it) {
        const int s = it % ST;
        ok = mbar_wait(&empty[s], ((it / ST) & 1) ^ 1, a.wait);
        if (!ok) break;
        const uint32_t dst = smem_u32(stages + s * kStage);
        uint32_t bar = smem_u32(&full[s]);
        if (rank == 0 || CG == 1) mbar_arrive_expect_tx(&full[s], CG * kStage);
        if (CG == 2) bar = map_rank(bar, 0);
        if (glu)
          tma_4d<CG>(dst, &tm_w, kb * kBK, 0, 0, rb * 4, bar);
        else
          tma_2d<CG>(dst, &tm_w, kb * kBK, rb * 128, bar);
        tma_2d<CG>(dst + kATile, &tm_x, kb * kBK, tok, bar);
      }
    }
    if (!ok) {
      set_err(a.dev_err, MOE_DEVERR_TIMEOUT);
      if (rank == 0 || CG == 1)  // the copies in flight land before the CTA ends
        for (int i = it > ST ? it - ST : 0; i < it; ++i) mbar_wait(&full[i % ST], (i / ST) & 1, a.wait);
    }
  } else if (warp == 1 && lane == 0 && (CG == 1 || rank == 0)) {  // -------- MMA
    const uint32_t idesc = idesc_bf16_mn(128 * CG, NT);
    int it = 0, ai = 0;
    bool ok = true;
    for (int tile = unit; ok && tile < P.tiles; tile += units) {
      for (int kc = kb0; ok && kc < kb1; kc += P.chunk, ++ai) {
        const int b = ai & 1;
        ok = CG == 2 ? mbar_wait_cluster(&acc_empty[b], ((ai >> 1) & 1) ^ 1, a.wait)
                     : mbar_wait(&acc_empty[b], ((ai >> 1) & 1) ^ 1, a.wait);
        if (!ok) break;
        tm_fence_after();
        const uint32_t d = tmem + b * NT;
        const int ke = kc + P.chunk < kb1 ? kc + P.chunk : kb1;
        for (int kb = kc; kb < ke; ++kb, ++it) {
          const int s = it % ST;
          ok = mbar_wait(&full[s], (it / ST) & 1, a.wait);
          if (!ok) break;
          tm_fence_after();
          const uint64_t ad = desc_sw128(smem_u32(stages + s * kStage));
          const uint64_t bd = desc_sw128(smem_u32(stages + s * kStage + kATile));
#pragma unroll
          for (int k = 0; k < kBK / 16; ++k)  // 16 elements of K = 32 bytes inside the swizzled row
            mma_ss<CG>(d, ad + 2 * k, bd + 2 * k, idesc, (kb > kc || k > 0) ? 1u : 0u);
          mma_commit<CG>(&empty[s]);
        }
        if (ok) mma_commit<CG>(&acc_full[b]);
      }
    }
    if (!ok) set_err(a.dev_err, MOE_DEVERR_TIMEOUT);
  } else if (warp >= 2) {  // ------------------------------------------- epilogue
    const int q = warp & 3, half = (warp - 2) >> 2;  // a warp reaches the TMEM lanes of its number mod 4
    const uint32_t lanes = static_cast<uint32_t>(q) << 21;  // lane 32 q in the address's upper half
    const uint32_t t_sum = tmem + lanes + 2 * NT;
    int ai = 0;
    bool ok = true;
    float* part = reinterpret_cast<float*>(stages);  // split: [NT][128] partial sums
    for (int tile = unit; ok && tile < P.tiles; tile += units) {
      int mb, tb;
      tile_of(tile, mb, tb);
      const int rb = mb * CG + (CG == 2 ? static_cast<int>(rank) : 0);
      const int64_t n = glu ? static_cast<int64_t>(rb) * 64 + q * 16 + (lane & 15)
                            : static_cast<int64_t>(rb) * 128 + q * 32 + lane;
      const bool nok = n < a.N;
      for (int kc = 0; kc < nchunk; ++kc, ++ai) {
        const int b = ai & 1;
        ok = mbar_wait(&acc_full[b], (ai >> 1) & 1, a.wait);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tm_fence_after();
        const uint32_t t_acc = tmem + lanes + b * NT;
        for (int c0 = half * (NT / 2); c0 < (half + 1) * (NT / 2); c0 += CW) {
          uint32_t r[CW];
          float v[CW];
          __syncwarp();
          tm_ld(t_acc + c0, r);
          tm_ld_wait();
#pragma unroll
          for (int c = 0; c < CW; ++c) v[c] = __uint_as_float(r[c]);
          if (kc > 0) {
            tm_ld(t_sum + c0, r);
            tm_ld_wait();
#pragma unroll
            for (int c = 0; c < CW; ++c) v[c] += __uint_as_float(r[c]);
          }
          if (kc < nchunk - 1) {
#pragma unroll
            for (int c = 0; c < CW; ++c) r[c] = __float_as_uint(v[c]);
            tm_st(t_sum + c0, r);
            tm_st_wait();
          } else if (CG == 1 && P.split > 1) {
#pragma unroll
            for (int c = 0; c < CW; ++c) part[(c0 + c) * 128 + q * 32 + lane] = v[c];
          } else {
            emit<CW>(a, v, static_cast<int64_t>(tb) * NT + c0, n, nok, lane);
          }
        }
        tm_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (CG == 2)
            mbar_arrive_remote(map_rank(smem_u32(&acc_empty[b]), 0));
          else
            mbar_arrive(&acc_empty[b]);
        }
      }
    }
    if (!ok && lane == 0) set_err(a.dev_err, MOE_DEVERR_TIMEOUT);
  }
  __syncwarp();

  if (CG == 1 && P.split > 1) {  // one tile per cluster: add the parts, a share of the columns per CTA
    cluster_sync_all();
    if (warp >= 2) {
      int mb, tb;
      tile_of(unit, mb, tb);
      const int q = warp & 3, half = (warp - 2) >> 2;
      const int64_t n = glu ? static_cast<int64_t>(mb) * 64 + q * 16 + (lane & 15)
                            : static_cast<int64_t>(mb) * 128 + q * 32 + lane;
      const int c0 = NT * static_cast<int>(rank) / P.split, c1 = NT * static_cast<int>(rank + 1) / P.split;
      for (int c = c0 + half; c < c1; c += 2) {
        const uint32_t off = smem_u32(stages) + (c * 128 + q * 32 + lane) * 4;
        float v = 0.f;
        for (int r = 0; r < P.split; ++r) v += ld_cluster_f32(map_rank(off, r));
        const int64_t t = static_cast<int64_t>(tb) * NT + c;
        bool nok = n < a.N && t < a.T;
        float bias = 0.f;
        if (a.bias && nok) bias = a.bias[(glu && lane >= 16 ? a.N : 0) + n];
        v += bias;
        if (glu) {
          v = swiglu_f32(v, __shfl_xor_sync(0xffffffffu, v, 16));
          nok = nok && lane < 16;
        } else {
          v = linear_act(v, a.act);
        }
        if (nok) linear_store(a, t, n, v);
      }
    }
  }
  tm_fence_before();
  __syncthreads();
  if (csize > 1) cluster_sync_all();  // no CTA leaves while another reads its shared memory or signals its barriers
  tm_fence_after();
  if (warp == 1) tm_free_cg<CG>(tmem, kCols);
}

// ------------------------------------------------------------------ host side
bool tma_rows(const void* p, int64_t ld, int rows) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && (rows <= 1 || (ld % 8 == 0 && ld < (1LL << 38)));
}

cudaError_t encode(CUtensorMap* m, const void* p, int nd, const cuuint64_t* dims, const cuuint64_t* strides,
                   const cuuint32_t* box) {
  EncodeFn enc = encode_fn();
  if (!enc) return cudaErrorNotSupported;
  const cuuint32_t one[4] = {1, 1, 1, 1};
  const CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, nd, const_cast<void*>(p), dims, strides, box, one,
                         CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <int CG, int NT>
cudaError_t launch(const LinearArgs& a, int split, cudaStream_t s) {
  const bool glu = a.act == MOE_ACT_SWIGLU;
  CUtensorMap tw, tx;
  const cuuint64_t ldw = static_cast<cuuint64_t>(a.N > 1 || glu ? a.ldw : a.K) * 2;
  const cuuint64_t ldx = static_cast<cuuint64_t>(a.T > 1 ? a.ldx : a.K) * 2;
  cudaError_t e;
  if (glu) {  // (k, row of 16, gate / up, 16-row group)
    const cuuint64_t dims[4] = {static_cast<cuuint64_t>(a.K), 16, 2, static_cast<cuuint64_t>(a.N / 16)};
    const cuuint64_t str[3] = {ldw, static_cast<cuuint64_t>(a.N) * ldw, 16 * ldw};
    const cuuint32_t box[4] = {kBK, 16, 2, 4};
    e = encode(&tw, a.w, 4, dims, str, box);
  } else {
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(a.K), static_cast<cuuint64_t>(a.N)};
    const cuuint32_t box[2] = {kBK, 128};
    e = encode(&tw, a.w, 2, dims, &ldw, box);
  }
  if (e != cudaSuccess) return e;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(a.K), static_cast<cuuint64_t>(a.T)};
  const cuuint32_t box[2] = {kBK, NT / CG};
  e = encode(&tx, a.x, 2, dims, &ldx, box);
  if (e != cudaSuccess) return e;

  TcParams P;
  P.a = a;
  const int64_t rows = glu ? 2 * static_cast<int64_t>(a.N) : a.N;
  P.mblocks = static_cast<int>((rows + 128 * CG - 1) / (128 * CG));
  P.tblocks = (a.T + NT - 1) / NT;
  if (static_cast<int64_t>(P.mblocks) * P.tblocks * (CG == 2 ? 2 : split) >= (1LL << 31)) return cudaErrorInvalidValue;
  P.tiles = P.mblocks * P.tblocks;
  P.kblocks = (a.K + kBK - 1) / kBK;
  P.chunk = a.out_fmt == MOE_FMT_F32 && NT <= 128 ? kChunk : P.kblocks;
  P.split = split;
  P.mfast = rows <= a.T;  // the smaller operand is the one read again from L2

  const int csize = CG == 2 ? 2 : split;
  int units = P.tiles;
  if (split == 1) {
    const int most = matmul_ctas() / csize > 0 ? matmul_ctas() / csize : 1;
    units = units < most ? units : most;
  }
  e = set_smem_limit(linear_tc_kernel<CG, NT>, smem_bytes<CG, NT>());
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(units * csize);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem_bytes<CG, NT>();
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = csize;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = csize > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, linear_tc_kernel<CG, NT>, tw, tx, P);
}

}  // namespace

bool linear_tc_supported(const LinearArgs& a) {
  const bool glu = a.act == MOE_ACT_SWIGLU;
  return a.K % 8 == 0 && tma_rows(a.x, a.ldx, a.T) && tma_rows(a.w, a.ldw, glu ? 2 * a.N : a.N) &&
         (!glu || a.N % 16 == 0);
}

cudaError_t launch_linear_tc(const LinearArgs& a, cudaStream_t s) {
  const int rows = a.act == MOE_ACT_SWIGLU ? 2 * a.N : a.N;
  const int mb = (rows + 127) / 128, kb = (a.K + kBK - 1) / kBK;
  const int sms = matmul_ctas();
  // split K while the tiles leave SMs idle and every part keeps two stages or more
  auto split_for = [&](int tiles) {
    int split = 1;
    while (split < 8 && tiles * split * 2 <= sms && kb >= split * 4) split *= 2;
    return split;
  };
  if (a.T <= 16) return launch<1, 16>(a, split_for(mb), s);
  if (a.T <= 32) return launch<1, 32>(a, split_for(mb), s);
  if (a.T <= 64) return launch<1, 64>(a, split_for(mb), s);
  const int64_t t128 = static_cast<int64_t>(mb) * ((a.T + 127) / 128);
  if (t128 <= sms) return launch<1, 128>(a, split_for(static_cast<int>(t128)), s);
  if (a.out_fmt == MOE_FMT_F32) return launch<2, 128>(a, 1, s);
  return launch<2, 256>(a, 1, s);
}

}  // namespace moe
