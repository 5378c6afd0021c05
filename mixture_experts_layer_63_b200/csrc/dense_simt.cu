// The dense operators' products on CUDA cores, for any strides and sizes,
// and their elementwise and column-sum passes.
//
//   acc[m, n] = sum_k A(m, k) B(n, k)
//
// One block of 256 threads computes a 64 x 64 tile of acc (4 x 4 outputs a
// thread) from 64 x 16 slices of A and B staged in shared memory as fp32.
// Sums run over 512 values of k at a time and the pieces are added to a
// second accumulator, so that a sum of K terms carries the rounding of
// 512 + K / 512 additions instead of K.
#include <algorithm>

#include "dense_internal.h"
#include "dense_math.cuh"

namespace moe {
namespace {

constexpr int TM = 64, TN = 64, TK = 16;
constexpr int kChunk = 512 / TK;        // slices summed before they join the second accumulator

// rows r0..r0+63, columns k0..k0+15 of an operand into dst[k][row]; zero
// outside [0, rows) x [0, K).  The 256 threads run along the contiguous
// index (K-major: 16 k by 16 rows; else 64 rows by 4 k).
template <typename T>
__device__ __forceinline__ void load_slice(const Operand &o, int64_t r0, int64_t rows, int64_t k0,
                                           int64_t K, float (*dst)[TM + 1]) {
  const T *p = static_cast<const T *>(o.p);
  const bool kmajor = o.ks == 1;
#pragma unroll
  for (int i = 0; i < TM * TK / 256; ++i) {
    const int e = threadIdx.x + 256 * i;
    const int k = kmajor ? e % TK : e / TM, r = kmajor ? e / TK : e % TM;
    float v = 0.0f;
    if (r0 + r < rows && k0 + k < K) v = to_f32(p[(r0 + r) * o.rs + (k0 + k) * o.ks]);
    dst[k][r] = v;
  }
}

template <typename T>
__device__ __forceinline__ void store1(const DenseGemm &P, int64_t m, int n, float acc, float acc3) {
  constexpr bool FAST = sizeof(T) == 2;
  const int64_t at = m * P.N + n;                          // packed [M, N]
  T *out = static_cast<T *>(P.out) + m * P.ld_o + n;
  switch (P.epi) {
    case kDenseLinear: {
      const float z = P.bias ? acc + to_f32(static_cast<const T *>(P.bias)[n]) : acc;
      float y = act_fwd<FAST>(z, P.act);
      if (P.residual) y += to_f32(static_cast<const T *>(P.residual)[m * P.ld_r + n]);
      if (P.pre) from_f32(static_cast<T *>(P.pre)[at], z);
      from_f32(*out, y);
      break;
    }
    case kDenseGated: {
      const float a = P.bias ? acc + to_f32(static_cast<const T *>(P.bias)[n]) : acc;
      const float u = P.bias3 ? acc3 + to_f32(static_cast<const T *>(P.bias3)[n]) : acc3;
      if (P.pre) from_f32(static_cast<T *>(P.pre)[at], a);
      if (P.pre3) from_f32(static_cast<T *>(P.pre3)[at], u);
      from_f32(*out, act_fwd<FAST>(a, P.act) * u);
      break;
    }
    case kDenseGatedGrad: {
      const float a = to_f32(static_cast<const T *>(P.pre_in)[at]);
      const float u = to_f32(static_cast<const T *>(P.pre3_in)[at]);
      float f, d;
      act_both<FAST>(a, P.act, f, d);
      from_f32(*out, acc * u * d);
      from_f32(static_cast<T *>(P.out2)[at], acc * f);
      from_f32(static_cast<T *>(P.out3)[at], f * u);
      break;
    }
    default: from_f32(*out, acc);
  }
}

template <typename T, bool GATED>
__global__ void __launch_bounds__(256) dense_simt_kernel(const DenseGemm P) {
  __shared__ float As[TK][TM + 1], Bs[TK][TN + 1], Cs[GATED ? TK : 1][TN + 1];
  const int64_t mt = (P.M + TM - 1) / TM;
  const int64_t tiles = mt * ((P.N + TN - 1) / TN);
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  pdl_wait();
  pdl_trigger();
  for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    const int64_t m0 = tile % mt * TM, n0 = tile / mt * TN;
    float acc[4][4] = {}, acc3[4][4] = {};
    for (int seg = 0; seg < (P.a2.p ? 2 : 1); ++seg) {
      const Operand a = seg ? P.a2 : P.a, b = seg ? P.b2 : P.b;
      for (int64_t k0 = 0; k0 < P.K; k0 += TK * kChunk) {
        float part[4][4] = {}, part3[4][4] = {};
        for (int64_t k = k0; k < P.K && k < k0 + TK * kChunk; k += TK) {
          __syncthreads();
          load_slice<T>(a, m0, P.M, k, P.K, As);
          load_slice<T>(b, n0, P.N, k, P.K, Bs);
          if (GATED) load_slice<T>(P.b3, n0, P.N, k, P.K, Cs);
          __syncthreads();
#pragma unroll
          for (int kk = 0; kk < TK; ++kk) {
            float av[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) av[i] = As[kk][ty + 16 * i];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float bv = Bs[kk][tx + 16 * j];
              const float cv = GATED ? Cs[kk][tx + 16 * j] : 0.0f;
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                part[i][j] = fmaf(av[i], bv, part[i][j]);
                if (GATED) part3[i][j] = fmaf(av[i], cv, part3[i][j]);
              }
            }
          }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            acc[i][j] += part[i][j];
            if (GATED) acc3[i][j] += part3[i][j];
          }
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int64_t m = m0 + ty + 16 * i, n = n0 + tx + 16 * j;
        if (m < P.M && n < P.N) store1<T>(P, m, (int)n, acc[i][j], acc3[i][j]);
      }
  }
}

template <typename T>
__global__ void __launch_bounds__(256) act_grad_kernel(int act, int64_t M, int N, const T *z, const T *dy,
                                                       int64_t ld_dy, T *dz) {
  pdl_wait();
  pdl_trigger();
  const int64_t total = M * N;
  for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < total; i += gridDim.x * 256ll) {
    const int64_t m = i / N;
    float f, d;
    act_both<sizeof(T) == 2>(to_f32(z[i]), act, f, d);
    from_f32(dz[i], to_f32(dy[m * ld_dy + (i - m * N)]) * d);
  }
}

// Column sums in two passes without atomics: block (x, y) adds the rows of
// part y in ascending order, 8 interleaved rows to a block, into part[y][n];
// the second kernel adds the parts in order.
constexpr int kColRows = 256;          // rows of a part at least
constexpr int kColParts = 64;          // parts at most

int colsum_parts(int64_t M) {
  return (int)std::min<int64_t>(kColParts, std::max<int64_t>(1, (M + kColRows - 1) / kColRows));
}

template <typename T>
__global__ void __launch_bounds__(256) colsum_part_kernel(int64_t M, int N, const T *src, int64_t ld,
                                                          float *part) {
  __shared__ float red[8][33];
  const int lane = threadIdx.x % 32, w = threadIdx.x / 32;
  const int n = blockIdx.x * 32 + lane;
  const int64_t per = (M + gridDim.y - 1) / gridDim.y;
  const int64_t r0 = blockIdx.y * per, r1 = min(M, r0 + per);
  pdl_wait();
  pdl_trigger();
  float v = 0.0f;
  if (n < N)
    for (int64_t r = r0 + w; r < r1; r += 8) v += to_f32(src[r * ld + n]);
  red[w][lane] = v;
  __syncthreads();
  if (w == 0 && n < N) {
    for (int i = 1; i < 8; ++i) v += red[i][lane];
    part[(int64_t)blockIdx.y * N + n] = v;
  }
}

template <typename T>
__global__ void __launch_bounds__(256) colsum_join_kernel(int parts, int N, const float *part, T *out) {
  const int n = blockIdx.x * 256 + threadIdx.x;
  pdl_wait();
  pdl_trigger();
  if (n >= N) return;
  float v = 0.0f;
  for (int p = 0; p < parts; ++p) v += part[(int64_t)p * N + n];
  from_f32(out[n], v);
}

unsigned grid_for(int64_t blocks, int per_sm) {
  return (unsigned)std::max<int64_t>(1, std::min<int64_t>(blocks, (int64_t)device_sms() * per_sm));
}

}  // namespace

cudaError_t launch_dense_simt(const DenseGemm &g, cudaStream_t s) {
  const int64_t tiles = ((g.M + TM - 1) / TM) * ((g.N + TN - 1) / TN);
  if (tiles == 0) return cudaSuccess;
  const unsigned grid = grid_for(tiles, 8);
  const bool gated = g.epi == kDenseGated;
  if (g.dtype == MOE_F32)
    return gated ? launch_kernel(dense_simt_kernel<float, true>, grid, 256, 0, s, g)
                 : launch_kernel(dense_simt_kernel<float, false>, grid, 256, 0, s, g);
  return gated ? launch_kernel(dense_simt_kernel<__nv_bfloat16, true>, grid, 256, 0, s, g)
               : launch_kernel(dense_simt_kernel<__nv_bfloat16, false>, grid, 256, 0, s, g);
}

cudaError_t launch_act_grad(int act, int dtype, int64_t M, int N, const void *z, const void *dy,
                            int64_t ld_dy, void *dz, cudaStream_t s) {
  if (M == 0) return cudaSuccess;
  const unsigned grid = grid_for((M * N + 255) / 256, 8);
  if (dtype == MOE_F32)
    return launch_kernel(act_grad_kernel<float>, grid, 256, 0, s, act, M, N, static_cast<const float *>(z),
                         static_cast<const float *>(dy), ld_dy, static_cast<float *>(dz));
  return launch_kernel(act_grad_kernel<__nv_bfloat16>, grid, 256, 0, s, act, M, N,
                       static_cast<const __nv_bfloat16 *>(z), static_cast<const __nv_bfloat16 *>(dy), ld_dy,
                       static_cast<__nv_bfloat16 *>(dz));
}

size_t colsum_scratch(int64_t M, int N) { return (size_t)colsum_parts(M) * N * 4; }

cudaError_t launch_colsum(int dtype, int64_t M, int N, const void *src, int64_t ld, float *part, void *out,
                          cudaStream_t s) {
  const int parts = colsum_parts(M);
  const dim3 grid((N + 31) / 32, parts);
  const unsigned gj = (N + 255) / 256;
  cudaError_t e;
  if (dtype == MOE_F32) {
    e = launch_kernel(colsum_part_kernel<float>, grid, 256, 0, s, M, N, static_cast<const float *>(src), ld,
                      part);
    if (e != cudaSuccess) return e;
    return launch_kernel(colsum_join_kernel<float>, gj, 256, 0, s, parts, N, part, static_cast<float *>(out));
  }
  e = launch_kernel(colsum_part_kernel<__nv_bfloat16>, grid, 256, 0, s, M, N,
                    static_cast<const __nv_bfloat16 *>(src), ld, part);
  if (e != cudaSuccess) return e;
  return launch_kernel(colsum_join_kernel<__nv_bfloat16>, gj, 256, 0, s, parts, N, part,
                       static_cast<__nv_bfloat16 *>(out));
}

}  // namespace moe
