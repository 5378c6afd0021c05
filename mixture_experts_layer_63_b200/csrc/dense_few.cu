// The dense operators' forward products for few rows (decoding, small
// batches): the time is the stream of the weights.
//
//   out[t, n] = epilogue(sum_k x(t, k) W(n, k)),  bf16, both K-major
//
// The weights take the MMA's M side (128 rows of W a CTA) and the tokens its
// N side (a multiple of 16), so one token costs no more than the weights'
// bytes.  To keep enough bytes in flight on all SMs the contraction is split
// over a cluster of up to eight CTAs: each streams its share of k through a
// TMA ring, leaves its fp32 partial tile in its shared memory, and the CTAs of
// the cluster then add the tokens among them in rank order, reading one
// another's partials (distributed shared memory).  No atomics and no second
// pass over global memory: the same bits on every call.  The gated block
// streams W1 and W3 side by side into two accumulators.
//
//   warp 0  TMA producer, warp 1  MMA issuer, all eight warps  epilogue
#include <algorithm>
#include <atomic>

#include "dense_few_plan.h"
#include "dense_internal.h"
#include "dense_math.cuh"
#include "sm100_ptx.cuh"

namespace moe {
namespace {

constexpr int BN = kFewBN, BK = kFewBK;
constexpr int kThreads = 256;
constexpr int kMaxStages = kFewMaxStages;
constexpr uint32_t kWBytes = kFewWBytes;

struct FewParams {
  CUtensorMap x, w, w3;
  int32_t M, N, KB;                 // k-blocks in all
  int32_t tt;                    // tokens (the MMA's N): M rounded up to 16
  int32_t planes;                // of x: stacked on the MMA's N side, joined when the accumulator is read
  int32_t stages, split, tmem_cols, act;
  const void *bias, *bias3, *residual;
  void *out, *pre, *pre3;
  int64_t ld_r, ld_o, lo_stride;
  uint32_t *err;
};

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap *map, uint32_t bar, int c0, int c1,
                                            int c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2)
      : "memory");
}

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

__device__ __forceinline__ void prefetch_tile(const CUtensorMap *map, int c0, int c1) {
  asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global [%0, {%1, %2, %3}];" ::"l"(reinterpret_cast<uint64_t>(map)),
               "r"(c0), "r"(c1), "r"(0)
               : "memory");
}

__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr));
  return v;
}

// U: tokens a thread joins at a time
template <bool GATED, int U>
__global__ void __launch_bounds__(kThreads) dense_few_kernel(const __grid_constant__ FewParams P) {
  using T = __nv_bfloat16;
  constexpr int NW = GATED ? 2 : 1;                // weight tiles of a stage
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t full_bar[kMaxStages];
  __shared__ __align__(8) uint64_t empty_bar[kMaxStages];
  __shared__ __align__(8) uint64_t acc_bar;
  __shared__ __align__(8) uint64_t drain_bar;
  __shared__ uint32_t s_tmem_base;
  __shared__ volatile int s_abort;
  __shared__ uint64_t s_limit_sh;

  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  const uint32_t x_bytes = (uint32_t)P.tt * BK * 2, stage_bytes = NW * kWBytes + P.planes * x_bytes;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int split = P.split, rank = (int)(blockIdx.x % (unsigned)split);
  const int n0 = (int)(blockIdx.x / (unsigned)split) * BN;
  const int kb0 = (int)((int64_t)P.KB * rank / split), kb1 = (int)((int64_t)P.KB * (rank + 1) / split);

  if (tid == 32) {
    for (int i = 0; i < P.stages; ++i) {
      mbar_init(&full_bar[i], 1);
      mbar_init(&empty_bar[i], 1);
    }
    mbar_init(&acc_bar, 1);
    mbar_init(&drain_bar, 1);
    s_abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 2) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&s_tmem_base)),
                 "r"(P.tmem_cols));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  if (tid == 0) {
    tma_prefetch_map(&P.x);
    tma_prefetch_map(&P.w);
    if (GATED) tma_prefetch_map(&P.w3);
  }
  // The first weights towards L2 while the kernel before this one ends: a hint
  // that reads nothing (what that kernel may still write to them is written
  // through L2); 23.5 us against 24.5 for one row at 14336 x 4096.
  if (tid == 64) {
    for (int kb = kb0; kb < min(kb1, kb0 + 4); ++kb) {
      prefetch_tile(&P.w, kb * BK, n0);
      if (GATED) prefetch_tile(&P.w3, kb * BK, n0);
    }
  }
  pdl_wait();
  pdl_trigger();
  if (tid == 0) s_limit_sh = wait_limit_ns(P.err);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = s_tmem_base;
  const uint64_t s_limit = s_limit_sh;
  const uint32_t smem0 = smem_u32(smem);

  if (warp == 0 && lane == 0) {
    int stage = 0, kb = kb0;
    uint32_t phase = 0;
    for (; kb < kb1; ++kb) {
      if (!mbar_wait(&empty_bar[stage], phase ^ 1u, &s_abort, P.err, s_limit)) break;
      const uint32_t s0 = smem0 + (uint32_t)stage * stage_bytes, fb = smem_u32(&full_bar[stage]);
      mbar_expect_tx(&full_bar[stage], stage_bytes);
      tma_load_3d(s0, &P.w, fb, kb * BK, n0, 0);
      if (GATED) tma_load_3d(s0 + kWBytes, &P.w3, fb, kb * BK, n0, 0);
      tma_load_3d(s0 + NW * kWBytes, &P.x, fb, kb * BK, 0, 0);                 // all planes
      if (++stage == P.stages) { stage = 0; phase ^= 1u; }
    }
    // aborting: the last round of each stage has to land before the exit
    if (kb < kb1)
      for (int i = kb - 1, n = 0; i >= kb0 && n < P.stages; --i, ++n)
        mbar_wait_drain(&full_bar[(i - kb0) % P.stages], (uint32_t)((i - kb0) / P.stages) & 1u);
  } else if (warp == 1 && lane == 0) {
    const uint32_t idesc = idesc_bf16(BN, P.planes * P.tt);
    int stage = 0;
    uint32_t phase = 0;
    for (int kb = kb0; kb < kb1; ++kb) {
      if (!mbar_wait(&full_bar[stage], phase, &s_abort, P.err, s_limit)) break;
      tc_fence_after();
      const uint32_t s0 = smem0 + (uint32_t)stage * stage_bytes;
      const uint64_t wd = sw128_desc(s0), xd = sw128_desc(s0 + NW * kWBytes);
#pragma unroll
      for (int k = 0; k < BK / 16; ++k) {
        const uint32_t on = kb > kb0 || k > 0 ? 1u : 0u;
        umma_bf16(tmem_base, wd + 2 * k, xd + 2 * k, idesc, on);
        if (GATED) umma_bf16(tmem_base + P.tt, wd + (kWBytes >> 4) + 2 * k, xd + 2 * k, idesc, on);
      }
      umma_commit(&empty_bar[stage]);
      if (++stage == P.stages) { stage = 0; phase ^= 1u; }
    }
    umma_commit(&acc_bar);
    umma_commit(&drain_bar);
    mbar_wait_drain(&drain_bar, 0);
  }
  __syncwarp();

  // the partial tile, [matrix][token][row of W] fp32, over the stages (all of
  // them have been read: the accumulator is complete)
  const bool done = __syncthreads_and(mbar_wait(&acc_bar, 0, &s_abort, P.err, s_limit)) && !s_abort;
  tc_fence_after();
  float *part = reinterpret_cast<float *>(smem);
  const int row = tid % BN;                        // of W
  if (done) {
    // (a warp reaches TMEM lanes 32 (warp mod 4) ...; its half of the columns)
    const uint32_t ta = tmem_base + ((uint32_t)((warp & 3) * 32) << 16);
    for (int c = 16 * (warp >> 2); c < NW * P.tt; c += 32) {
      uint32_t r[16];
      tmem_ld16(ta + c, r);
      tmem_ld_wait();
      if (!GATED && P.planes == 2) {
        uint32_t lo[16];
        tmem_ld16(ta + P.tt + c, lo);
        tmem_ld_wait();
        // (an infinite weight makes the high plane's sum infinite; times a low
        // part, which may be 0 or of the other sign, it would say NaN)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float hi = __uint_as_float(r[i]);
          if (isfinite(hi)) r[i] = __float_as_uint(hi + __uint_as_float(lo[i]));
        }
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) part[(c + i) * BN + row] = kb1 > kb0 ? __uint_as_float(r[i]) : 0.0f;
    }
  }
  tc_fence_before();
  cluster_sync_all();
  if (done) {
    // tokens by rank, two thread halves within a rank
    const int n = n0 + row, step = 2 * split;
    const bool in = n < P.N;
    const float b = in && P.bias ? to_f32(static_cast<const T *>(P.bias)[n]) : 0.0f;
    const float b3 = GATED && in && P.bias3 ? to_f32(static_cast<const T *>(P.bias3)[n]) : 0.0f;
    const uint32_t p0 = smem0 + 4u * row, m3 = (uint32_t)P.tt * BN * 4;
    // U tokens at a time, with everything they read in flight (a token past the
    // last one reads the last one again); partials of four ranks at a time,
    // added in rank order
    for (int t = 2 * rank + tid / BN; t < P.M; t += U * step) {
      float v[U] = {}, u[U] = {}, res[U] = {};
      if (!GATED && P.residual && in) {
#pragma unroll
        for (int i = 0; i < U; ++i)
          res[i] = to_f32(static_cast<const T *>(P.residual)[(int64_t)min(t + i * step, P.M - 1) * P.ld_r + n]);
      }
      for (int r = 0; r < split; r += 4) {
        float pv[4][U], pu[4][U];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          if (r + q >= split) break;
          const uint32_t p = mapa_shared(p0, (uint32_t)(r + q));
#pragma unroll
          for (int i = 0; i < U; ++i) {
            const int ti = min(t + i * step, P.M - 1);
            pv[q][i] = ld_cluster_f32(p + (uint32_t)ti * BN * 4);
            if (GATED) pu[q][i] = ld_cluster_f32(p + m3 + (uint32_t)ti * BN * 4);
          }
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          if (r + q >= split) break;
#pragma unroll
          for (int i = 0; i < U; ++i) {
            v[i] += pv[q][i];
            if (GATED) u[i] += pu[q][i];
          }
        }
      }
      if (!in) continue;
      const int live = (P.M - 1 - t) / step + 1;               // tokens of these U that exist
#pragma unroll
      for (int i = 0; i < U; ++i) {
        v[i] += b;
        if (GATED) u[i] += b3;
      }
      if (P.pre) {
#pragma unroll
        for (int i = 0; i < U; ++i)
          if (i < live) {
            const int64_t at = (int64_t)(t + i * step) * P.N + n;
            from_f32(static_cast<T *>(P.pre)[at], v[i]);
            if (GATED && P.pre3) from_f32(static_cast<T *>(P.pre3)[at], u[i]);
          }
      }
      with_act(P.act, [&](auto A) {
#pragma unroll
        for (int i = 0; i < U; ++i) v[i] = act_fwd<true, decltype(A)::value>(v[i]);
      });
#pragma unroll
      for (int i = 0; i < U; ++i)
        if (i < live) {
          T *o = static_cast<T *>(P.out) + (int64_t)(t + i * step) * P.ld_o + n;
          const float y = GATED ? v[i] * u[i] : v[i] + res[i];
          from_f32(*o, y);
          if (P.lo_stride) from_f32(o[P.lo_stride], rest_of(y, to_f32(*o)));
        }
    }
  }
  cluster_sync_all();              // no CTA leaves while another may read its partial tile
  tc_fence_after();
  if (warp == 2)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(P.tmem_cols));
}

constexpr int kMaxDevices = 64;
constexpr size_t kMaxSmem = kFewMaxSmem;

template <auto kern>
cudaError_t allow_smem() {
  static std::atomic<bool> done[kMaxDevices];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || (dev < kMaxDevices && done[dev].load(std::memory_order_acquire))) return e;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kMaxSmem);
  if (e == cudaSuccess && dev < kMaxDevices) done[dev].store(true, std::memory_order_release);
  return e;
}

// CTAs of `split` a cluster that are resident at once, per_sm of them an SM: the
// GPCs hold whole clusters only.  One an SM: 132 CTAs in fours, 120 in eights (a
// 16th cluster of eight ran alone: 31 us for 128 rows of 2048 x 5632, 20 in fours),
// asked once a device.  Several an SM leave less over, about one SM in 64 a
// step of the size (two an SM: 284 in fours, 264 in eights); the occupancy
// query does not tell: it counts one CTA an SM for a kernel that allocates TMEM.
int64_t resident(int split, int per_sm) {
  if (per_sm > 1) return (int64_t)device_sms() * per_sm * (65 - split) / 64;
  static std::atomic<int> cache[kMaxDevices][4];
  int dev = 0, log = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  while (1 << log < split) ++log;
  int n = dev < kMaxDevices ? cache[dev][log].load(std::memory_order_acquire) : 0;
  if (n == 0) {
    constexpr auto kern = dense_few_kernel<false, 1>;
    if (allow_smem<kern>() != cudaSuccess) return 0;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)split);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kMaxSmem;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim = {(unsigned)split, 1, 1};
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess || n <= 0) {
      cudaGetLastError();
      n = std::max(1, device_sms() / split);
    }
    n *= split;
    if (dev < kMaxDevices) cache[dev][log].store(n, std::memory_order_release);
  }
  return n;
}

template <bool GATED, int U>
cudaError_t launch_few_as(const FewParams &P, unsigned tiles, size_t smem, cudaStream_t s) {
  constexpr auto kern = dense_few_kernel<GATED, U>;
  cudaError_t e = allow_smem<kern>();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(tiles * (unsigned)P.split);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim = {(unsigned)P.split, 1, 1};
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = MOE_PDL ? 2 : 1;
  e = cudaLaunchKernelEx(&cfg, kern, P);
  if (e == cudaSuccess) count_launch();
  return e;
}

}  // namespace

bool dense_few_ok(const DenseGemm &g) {
  return (g.epi == kDenseLinear || g.epi == kDenseGated) && g.dtype == MOE_BF16 && g.M <= kFewRows &&
         (g.a.planes < 2 || (g.epi == kDenseLinear && 2 * g.M <= kFewRows)) && g.b.planes < 2 && g.b3.planes < 2 && dense_tc_ok(g);
}

cudaError_t launch_dense_few(const DenseGemm &g, uint32_t *err, cudaStream_t s) {
  const bool gated = g.epi == kDenseGated;
  FewParams P{};
  P.planes = std::max(1, g.a.planes);
  const FewPlan plan = few_plan(g.M, g.K, g.N, gated, P.planes, resident);
  P.tt = plan.tt;
  P.KB = plan.KB;
  P.stages = plan.stages;
  P.split = plan.split;
  P.tmem_cols = plan.tmem_cols;
  auto map = [&](CUtensorMap *m, const Operand &o, int64_t rows, int box) {
    const int64_t ld = rows == 1 ? pack_ld(g.K) : o.rs;
    return make_map3d(m, o.p, g.K, rows, std::max(1, o.planes), ld, o.planes > 1 ? o.plane_stride : ld * rows, box,
                      std::max(1, o.planes));
  };
  if (!map(&P.x, g.a, g.M, P.tt) || !map(&P.w, g.b, g.N, BN) || (gated && !map(&P.w3, g.b3, g.N, BN)))
    return cudaErrorInvalidValue;
  P.M = (int32_t)g.M;
  P.N = g.N;
  P.act = g.act;
  P.bias = g.bias;
  P.bias3 = g.bias3;
  P.residual = g.residual;
  P.out = g.out;
  P.pre = g.pre;
  P.pre3 = g.pre3;
  P.ld_r = g.ld_r;
  P.ld_o = g.ld_o;
  P.lo_stride = g.lo_stride;
  P.err = err;
  // a thread's tokens at a time: all of them, up to four (eight with one
  // matrix), so that their loads are in flight together; more would be idle loads
  const unsigned nt = (unsigned)plan.tiles;
  const size_t smem = plan.smem;
  const int64_t each = (g.M + 2 * P.split - 1) / (2 * P.split);
  if (each <= 1) return gated ? launch_few_as<true, 1>(P, nt, smem, s) : launch_few_as<false, 1>(P, nt, smem, s);
  if (each <= 2) return gated ? launch_few_as<true, 2>(P, nt, smem, s) : launch_few_as<false, 2>(P, nt, smem, s);
  if (gated) return launch_few_as<true, 4>(P, nt, smem, s);
  return each <= 4 ? launch_few_as<false, 4>(P, nt, smem, s) : launch_few_as<false, 8>(P, nt, smem, s);
}

}  // namespace moe
