// The dense operators' forward products for few rows on CUDA cores: fp32, and
// bf16 matrices that TMA cannot read as they lie.  The time is the stream of
// the weights, which are read once, straight into registers (the tensor-core
// paths would write and read a copy of them first).
//
//   out[m, n] = epilogue(sum_k x(m, k) W(n, k))
//
// A warp keeps kRows rows of W against MT rows of x (all of a small batch):
// its lanes run along k, 16 bytes each where the lines allow it, and add in
// fp32; a butterfly of shuffles joins the lanes.  `ks` warps of a block share
// the k range of the same rows when there are too few rows of W to fill the
// GPU; their sums are added in order through shared memory.
#include <algorithm>

#include "dense_internal.h"
#include "dense_math.cuh"

namespace moe {
namespace {

constexpr int kWarps = 8;
constexpr int kRows = 4;               // rows of W a warp (gated: two of W1, the same two of W3)

// V consecutive elements (VEC), or the V elements 32 apart that a lane owns
// STREAM: without a place in L1 (the weights; x stays there)
template <typename T, bool VEC, bool STREAM>
__device__ __forceinline__ void load_k(const T *p, int64_t k, int64_t K, float (&v)[16 / sizeof(T)]) {
  constexpr int V = 16 / sizeof(T);
  const int lane = threadIdx.x % 32;
  if (VEC) {
    if (k + (lane + 1) * V <= K) {
      const uint4 *q = reinterpret_cast<const uint4 *>(p + k) + lane;
      uint4 w;
      if (STREAM)
        asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w)
                     : "l"(q));
      else
        w = __ldg(q);
      unpack16<T>(w, v);
      return;
    }
#pragma unroll
    for (int j = 0; j < V; ++j) v[j] = k + lane * V + j < K ? to_f32(p[k + lane * V + j]) : 0.0f;
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j) v[j] = k + 32 * j + lane < K ? to_f32(p[k + 32 * j + lane]) : 0.0f;
  }
}

// PLANES: x is two planes (bf16)
template <typename T, bool GATED, int MT, bool VEC, bool PLANES>
__global__ void __launch_bounds__(32 * kWarps) dense_rows_kernel(const DenseGemm P, int ks) {
  constexpr int V = 16 / sizeof(T), NR = GATED ? kRows / 2 : kRows;
  constexpr bool FAST = sizeof(T) == 2;
  __shared__ float red[kWarps][kRows][MT];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int mt = (int)((P.M + MT - 1) / MT);
  const int64_t m0 = (int64_t)(blockIdx.x % (unsigned)mt) * MT;
  const int nw = kWarps / ks;                                      // row groups of the block
  const int64_t n0 = ((int64_t)(blockIdx.x / (unsigned)mt) * nw + warp / ks) * NR;
  const int64_t step = 32 * V, chunks = (P.K + step - 1) / step;
  const int wk = warp % ks;
  const int64_t k0 = chunks * wk / ks * step, k1 = min(P.K, chunks * (wk + 1) / ks * step);
  pdl_wait();
  pdl_trigger();
  const T *x = static_cast<const T *>(P.a.p), *w1 = static_cast<const T *>(P.b.p), *w3 = static_cast<const T *>(P.b3.p);
  float acc[kRows][MT] = {};
  // rows past the last one read the last one again: nothing of it is stored
  const T *wr[kRows];
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    const int64_t n = min(n0 + (GATED ? r % NR : r), (int64_t)P.N - 1);
    wr[r] = GATED && r >= NR ? w3 + n * P.b3.rs : w1 + n * P.b.rs;
  }
  const T *xr[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) xr[m] = x + min(m0 + m, P.M - 1) * P.a.rs;
#pragma unroll 2
  for (int64_t k = k0; k < k1; k += step) {
    float w[kRows][V];
#pragma unroll
    for (int r = 0; r < kRows; ++r) load_k<T, VEC, true>(wr[r], k, k1, w[r]);
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      float v[V];
      load_k<T, VEC, false>(xr[m], k, k1, v);
      if (PLANES) {
        float lo[V];
        load_k<T, VEC, false>(xr[m] + P.a.plane_stride, k, k1, lo);
#pragma unroll
        for (int j = 0; j < V; ++j) v[j] += lo[j];
      }
#pragma unroll
      for (int r = 0; r < kRows; ++r)
#pragma unroll
        for (int j = 0; j < V; ++j) acc[r][m] = fmaf(w[r][j], v[j], acc[r][m]);
    }
  }
#pragma unroll
  for (int r = 0; r < kRows; ++r)
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      float v = acc[r][m];
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
      if (lane == 0) red[warp][r][m] = v;
    }
  __syncthreads();
  for (int i = threadIdx.x; i < nw * NR * MT; i += 32 * kWarps) {
    const int r = i % NR, q = i / NR % nw;
    const int m = i / (NR * nw);
    const int64_t n = ((int64_t)(blockIdx.x / (unsigned)mt) * nw + q) * NR + r, row = m0 + m;
    if (n >= P.N || row >= P.M) continue;
    float a = 0.0f, u = 0.0f;
    for (int s = 0; s < ks; ++s) {
      a += red[q * ks + s][r][m];
      if (GATED) u += red[q * ks + s][NR + r][m];
    }
    if (P.bias) a += to_f32(static_cast<const T *>(P.bias)[n]);
    if (P.pre) from_f32(static_cast<T *>(P.pre)[row * P.N + n], a);
    with_act(P.act, [&](auto A) { a = act_fwd<FAST, decltype(A)::value>(a); });
    if (GATED) {
      if (P.bias3) u += to_f32(static_cast<const T *>(P.bias3)[n]);
      if (P.pre3) from_f32(static_cast<T *>(P.pre3)[row * P.N + n], u);
      a *= u;
    } else if (P.residual) {
      a += to_f32(static_cast<const T *>(P.residual)[row * P.ld_r + n]);
    }
    T *o = static_cast<T *>(P.out) + row * P.ld_o + n;
    from_f32(*o, a);
    if (P.lo_stride) from_f32(o[P.lo_stride], rest_of(a, to_f32(*o)));
  }
}

template <typename T, bool GATED, int MT>
cudaError_t rows_as(const DenseGemm &g, cudaStream_t s) {
  constexpr int NR = GATED ? kRows / 2 : kRows;
  auto lines16 = [&](const Operand &o) {
    return !o.p || ((reinterpret_cast<uintptr_t>(o.p) | (uintptr_t)((o.rs | o.plane_stride) * (int64_t)sizeof(T))) & 15) == 0;
  };
  const bool vec = lines16(g.a) && lines16(g.b) && lines16(g.b3);
  const int64_t mt = (g.M + MT - 1) / MT, groups = (g.N + NR - 1) / NR;
  auto blocks = [&](int ks) { return (groups + kWarps / ks - 1) / (kWarps / ks) * mt; };
  int ks = 1;
  while (ks < kWarps && blocks(ks) < (int64_t)device_sms() * 4 && g.K / (2 * ks) >= 512) ks *= 2;
  if (blocks(ks) > 0x7fffffff) return cudaErrorInvalidValue;
  auto run = [&](auto kern) { return launch_kernel(kern, (unsigned)blocks(ks), 32 * kWarps, 0, s, g, ks); };
  if constexpr (sizeof(T) == 2 && !GATED)
    if (g.a.planes == 2)
      return vec ? run(dense_rows_kernel<T, GATED, MT, true, true>) : run(dense_rows_kernel<T, GATED, MT, false, true>);
  return vec ? run(dense_rows_kernel<T, GATED, MT, true, false>) : run(dense_rows_kernel<T, GATED, MT, false, false>);
}

// Rows of x a block.  bf16, whose lines are read element by element: up to three
// rows one each, in blocks side by side that share the weights in L2 (two rows of
// 4099 x 8192: 36 us, 52 with both in a block; three of 1411 x 2049: 7 against 13).
template <typename T, bool GATED>
cudaError_t rows_of(const DenseGemm &g, cudaStream_t s) {
  if (g.M == 1 || (sizeof(T) == 2 && g.M <= 3)) return rows_as<T, GATED, 1>(g, s);
  if constexpr (sizeof(T) == 4)
    if (g.M == 2) return rows_as<T, GATED, 2>(g, s);
  return g.M <= 4 ? rows_as<T, GATED, 4>(g, s) : rows_as<T, GATED, 8>(g, s);
}

}  // namespace

// Rows up to which the stream through registers beats a copy for the tensor
// cores and their launch.  fp32, K = 4096, N = 8192: 28 us (1 row; 4.8 TB/s), 52
// (8), 93 (16) against 145 whatever the rows, about 180 against 145 at 32; 1024 x
// 1024: 9 against 31 at 32 rows.  bf16 with unaligned lines, K = 4099, N = 8192:
// 23 against 46 us (1 row), 36 (2), 46 (3); 2051 x 4096: 16 against 17 at 3 rows, 21
// at 4; gated 1411 / 5003: 49 against 41 at 3; 1027 x 1024: 8 against 10 at 8.
bool dense_rows_ok(const DenseGemm &g) {
  if (g.epi != kDenseLinear && g.epi != kDenseGated) return false;
  const int64_t size = g.K * g.N;
  const bool small = size <= (int64_t)1 << 21;
  if (g.dtype == MOE_F32) return g.M <= (small ? 2 * kRegisterRows : kRegisterRows);
  return g.M <= (small ? 8 : size * (g.epi == kDenseGated || g.a.planes == 2 ? 2 : 1) <= (int64_t)5 << 21 ? 3 : 2);
}

cudaError_t launch_dense_rows(const DenseGemm &g, cudaStream_t s) {
  const bool gated = g.epi == kDenseGated;
  if (g.dtype == MOE_F32) return gated ? rows_of<float, true>(g, s) : rows_of<float, false>(g, s);
  return gated ? rows_of<__nv_bfloat16, true>(g, s) : rows_of<__nv_bfloat16, false>(g, s);
}

}  // namespace moe
