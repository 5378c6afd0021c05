// The dense operators' products on CUDA cores, for any strides and sizes,
// and their column-sum passes.
//
//   acc[m, n] = sum_k A(m, k) B(n, k)
//
// One block of 256 threads computes a TS x TS tile of acc (TS / 16 squared
// outputs a thread) from TS x 32 slices of A and B staged in shared memory as
// fp32; the next slice is read into registers while this one is used.  Tiles
// of 32 where 64 would leave SMs without one: what runs here is small (fp32
// products below the tensor cores' break-even: 256 x 64 x 128 takes 6 us),
// or cannot be read by TMA.  Sums run over 512 values of k at a time and the
// pieces are added to a second accumulator, so that a sum of K terms carries
// the rounding of 512 + K / 512 additions instead of K.
#include <algorithm>

#include "dense_internal.h"
#include "dense_math.cuh"

namespace moe {
namespace {

constexpr int TK = 32;
constexpr int kChunk = 512;            // values of k summed before they join the second accumulator

// A thread's share of rows r0 ... r0 + TS - 1, columns k0 ... k0 + 31 of an
// operand; zero outside [0, rows) x [0, K).  The threads run along the
// contiguous index (K-major: 32 k by 8 rows; else TS rows by 256 / TS k).
template <typename T, int TS>
struct Slice {
  static constexpr int N = TS * TK / 256;
  float v[N];
  __device__ __forceinline__ static void at(const Operand &o, int i, int &r, int &k) {
    const int e = threadIdx.x + 256 * i;
    k = o.ks == 1 ? e % TK : e / TS;
    r = o.ks == 1 ? e / TK : e % TS;
  }
  __device__ __forceinline__ void fetch(const Operand &o, int64_t r0, int64_t rows, int64_t k0, int64_t K) {
    const T *p = static_cast<const T *>(o.p);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      int r, k;
      at(o, i, r, k);
      v[i] = 0.0f;
      if (r0 + r < rows && k0 + k < K) {
        const int64_t e = (r0 + r) * o.rs + (k0 + k) * o.ks;
        v[i] = to_f32(p[e]);
        if (o.planes == 2) v[i] += to_f32(p[e + o.plane_stride]);
      }
    }
  }
  __device__ __forceinline__ void put(const Operand &o, float (*dst)[TS + 1]) const {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      int r, k;
      at(o, i, r, k);
      dst[k][r] = v[i];
    }
  }
};

// v, and what its rounding leaves to the low plane
template <typename T>
__device__ __forceinline__ void store_planes(void *base, int64_t at, int64_t lo_stride, float v) {
  T *p = static_cast<T *>(base) + at;
  from_f32(*p, v);
  if (lo_stride) from_f32(p[lo_stride], rest_of(v, to_f32(*p)));
}

template <typename T>
__device__ __forceinline__ void store1(const DenseGemm &P, int64_t m, int n, float acc, float acc3) {
  constexpr bool FAST = sizeof(T) == 2;
  const int64_t at = m * P.N + n;                          // packed [M, N]
  T *out = static_cast<T *>(P.out) + m * P.ld_o + n;
  switch (P.epi) {
    case kDenseLinear: {
      const float z = P.bias ? acc + to_f32(static_cast<const T *>(P.bias)[n]) : acc;
      float y = 0.0f;
      with_act(P.act, [&](auto A) { y = act_fwd<FAST, decltype(A)::value>(z); });
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
      float f = 0.0f;
      with_act(P.act, [&](auto A) { f = act_fwd<FAST, decltype(A)::value>(a); });
      store_planes<T>(P.out, m * P.ld_o + n, P.lo_stride, f * u);
      break;
    }
    case kDenseGatedGrad: {
      const float a = to_f32(static_cast<const T *>(P.pre_in)[at]);
      const float u = to_f32(static_cast<const T *>(P.pre3_in)[at]);
      float f = 0.0f, d = 0.0f;
      with_act(P.act, [&](auto A) { act_both<FAST, decltype(A)::value>(a, f, d); });
      store_planes<T>(P.out, m * P.ld_o + n, P.lo_stride, acc * u * d);
      store_planes<T>(P.out2, m * P.ld_o + n, P.lo_stride, acc * f);
      store_planes<T>(P.out3, m * P.ld_o + n, P.lo_stride, f * u);
      break;
    }
    default: from_f32(*out, acc);
  }
}

template <typename T, bool GATED, int TS>
__global__ void __launch_bounds__(256) dense_simt_kernel(const __grid_constant__ DenseGemm P) {
  constexpr int R = TS / 16;
  __shared__ float As[TK][TS + 1], Bs[TK][TS + 1], Cs[GATED ? TK : 1][TS + 1];
  const int64_t mt = (P.M + TS - 1) / TS;
  const int64_t tiles = mt * ((P.N + TS - 1) / TS);
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  pdl_wait();
  pdl_trigger();
  for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    const int64_t m0 = tile % mt * TS, n0 = tile / mt * TS;
    float acc[R][R] = {}, acc3[R][R] = {};
    for (int seg = 0; seg < (P.a2.p ? 2 : 1); ++seg) {
      const Operand a = seg ? P.a2 : P.a, b = seg ? P.b2 : P.b;
      Slice<T, TS> sa, sb, sc;
      float part[R][R] = {}, part3[R][R] = {};
      auto fetch = [&](int64_t k) {
        sa.fetch(a, m0, P.M, k, P.K);
        sb.fetch(b, n0, P.N, k, P.K);
        if (GATED) sc.fetch(P.b3, n0, P.N, k, P.K);
      };
      if (P.K > 0) fetch(0);
      for (int64_t k = 0; k < P.K; k += TK) {
        __syncthreads();
        sa.put(a, As);
        sb.put(b, Bs);
        if (GATED) sc.put(P.b3, Cs);
        __syncthreads();
        if (k + TK < P.K) fetch(k + TK);
#pragma unroll
        for (int kk = 0; kk < TK; ++kk) {
          float av[R];
#pragma unroll
          for (int i = 0; i < R; ++i) av[i] = As[kk][ty + 16 * i];
#pragma unroll
          for (int j = 0; j < R; ++j) {
            const float bv = Bs[kk][tx + 16 * j];
            const float cv = GATED ? Cs[kk][tx + 16 * j] : 0.0f;
#pragma unroll
            for (int i = 0; i < R; ++i) {
              part[i][j] = fmaf(av[i], bv, part[i][j]);
              if (GATED) part3[i][j] = fmaf(av[i], cv, part3[i][j]);
            }
          }
        }
        if ((k + TK) % kChunk == 0 || k + TK >= P.K) {
#pragma unroll
          for (int i = 0; i < R; ++i)
#pragma unroll
            for (int j = 0; j < R; ++j) {
              acc[i][j] += part[i][j];
              part[i][j] = 0.0f;
              if (GATED) {
                acc3[i][j] += part3[i][j];
                part3[i][j] = 0.0f;
              }
            }
        }
      }
    }
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
      for (int j = 0; j < R; ++j) {
        const int64_t m = m0 + ty + 16 * i, n = n0 + tx + 16 * j;
        if (m < P.M && n < P.N) store1<T>(P, m, (int)n, acc[i][j], acc3[i][j]);
      }
  }
}

// Column sums, and dz = dy act'(z) on the way (ACT): a warp reads rows of 32
// pieces of V = 16 / sizeof(T) columns; block (x, y) adds the rows of part y,
// eight interleaved, and leaves their sums in part[y][n]; the second kernel
// adds the parts in order.  dz enters its sums before its rounding.  No
// atomics: the same bits on every call.
constexpr int kNoAct = -1;
struct ColSums {
  ColSum q[kMaxColSums];
  int64_t M;
  int parts;
  float *part;                 // [count][parts][max N]
  int64_t part_stride;
};

template <typename T, int ACT>          // ACT: the activation, or kNoAct
__global__ void __launch_bounds__(256, ACT == kNoAct ? 2 : 4) colsum_part_kernel(const ColSums P) {
  constexpr int V = 16 / sizeof(T);
  __shared__ float red[8][32 * V];
  const ColSum Q = P.q[blockIdx.z];
  const int lane = threadIdx.x % 32, w = threadIdx.x / 32;
  const int n0 = blockIdx.x * 32 * V;
  const int64_t per = (P.M + P.parts - 1) / P.parts;
  const int64_t r0 = blockIdx.y * per, r1 = min(P.M, r0 + per);
  pdl_wait();
  pdl_trigger();
  if (n0 >= Q.N) return;
  const T *src = static_cast<const T *>(Q.src), *z = static_cast<const T *>(Q.z);
  T *dz = static_cast<T *>(Q.dz);
  float sum[V] = {};
  uintptr_t at = reinterpret_cast<uintptr_t>(src) | (uintptr_t)(Q.ld * (int64_t)sizeof(T));
  constexpr bool GRAD = ACT != kNoAct;
  if (GRAD) at |= reinterpret_cast<uintptr_t>(z) | (uintptr_t)((int64_t)Q.N * sizeof(T));
  const int n = n0 + lane * V;
  if ((at & 15) == 0 && n0 + 32 * V <= Q.N) {
    // whole 16-byte pieces, R rows in flight a warp; the activations leave
    // fewer registers a warp and want more warps
    constexpr int R = GRAD ? 2 : 4;
    for (int64_t r = r0 + w; r < r1; r += 8 * R) {
      uint4 a[R], b[R];
#pragma unroll
      for (int i = 0; i < R; ++i)
        if (r + 8 * i < r1) {
          a[i] = *reinterpret_cast<const uint4 *>(src + (r + 8 * i) * Q.ld + n);
          if (GRAD) b[i] = *reinterpret_cast<const uint4 *>(z + (r + 8 * i) * Q.N + n);
        }
#pragma unroll
      for (int i = 0; i < R; ++i) {
        if (r + 8 * i >= r1) break;
        float v[V];
        unpack16<T>(a[i], v);
        if (Q.src_lo) {
          float lo[V];
          unpack16<T>(*reinterpret_cast<const uint4 *>(src + Q.src_lo + (r + 8 * i) * Q.ld + n), lo);
#pragma unroll
          for (int j = 0; j < V; ++j) v[j] += lo[j];
        }
        if (GRAD) {
          float zz[V];
          unpack16<T>(b[i], zz);
#pragma unroll
          for (int j = 0; j < V; j += 2) {
            float2 f, d;
            act_both2<sizeof(T) == 2, ACT>(make_float2(zz[j], zz[j + 1]), f, d);
            v[j] *= d.x;
            v[j + 1] *= d.y;
          }
          uint4 *o = reinterpret_cast<uint4 *>(dz + (r + 8 * i) * Q.ld_dz + n);
          const uint4 hi = pack16<T>(v);
          *o = hi;
          if (Q.lo_stride) {
            float h[V];
            unpack16<T>(hi, h);
#pragma unroll
            for (int j = 0; j < V; ++j) h[j] = rest_of(v[j], h[j]);
            *reinterpret_cast<uint4 *>(dz + Q.lo_stride + (r + 8 * i) * Q.ld_dz + n) = pack16<T>(h);
          }
        }
#pragma unroll
        for (int j = 0; j < V; ++j) sum[j] += v[j];
      }
    }
  } else {
    // column j of a lane is n0 + 32 j + lane
    for (int64_t r = r0 + w; r < r1; r += 8)
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int c = n0 + 32 * j + lane;
        if (c >= Q.N) break;
        float v = to_f32(src[r * Q.ld + c]);
        if (Q.src_lo) v += to_f32(src[r * Q.ld + c + Q.src_lo]);
        if (GRAD) {
          float f, d;
          act_both<sizeof(T) == 2, ACT>(to_f32(z[r * Q.N + c]), f, d);
          v *= d;
          T *o = dz + r * Q.ld_dz + c;
          from_f32(*o, v);
          if (Q.lo_stride) from_f32(o[Q.lo_stride], rest_of(v, to_f32(*o)));
        }
        sum[j] += v;
      }
  }
  if (!Q.out) return;                     // dz alone is wanted
  const bool pieces = (at & 15) == 0 && n0 + 32 * V <= Q.N;
#pragma unroll
  for (int j = 0; j < V; ++j) red[w][pieces ? lane * V + j : 32 * j + lane] = sum[j];
  __syncthreads();
  for (int c = threadIdx.x; c < 32 * V && n0 + c < Q.N; c += 256) {
    float v = red[0][c];
    for (int i = 1; i < 8; ++i) v += red[i][c];
    P.part[(blockIdx.z * (int64_t)P.parts + blockIdx.y) * P.part_stride + n0 + c] = v;
  }
}

// 32 columns a block: warp w adds parts w, w + 8, ..., then the eight sums join
template <typename T>
__global__ void __launch_bounds__(256) colsum_join_kernel(const ColSums P) {
  __shared__ float red[8][32];
  const ColSum Q = P.q[blockIdx.z];
  const int lane = threadIdx.x % 32, w = threadIdx.x / 32;
  const int n = blockIdx.x * 32 + lane;
  pdl_wait();
  pdl_trigger();
  if (blockIdx.x * 32 >= Q.N || !Q.out) return;
  float v = 0.0f;
  if (n < Q.N) {
    const float *p = P.part + blockIdx.z * (int64_t)P.parts * P.part_stride + n;
#pragma unroll 8
    for (int i = w; i < P.parts; i += 8) v += p[i * P.part_stride];
  }
  red[w][lane] = v;
  __syncthreads();
  if (w == 0 && n < Q.N) {
    for (int i = 1; i < 8; ++i) v += red[i][lane];
    from_f32(static_cast<T *>(Q.out)[n], v);
  }
}

// enough row parts for some eight blocks an SM, at least 32 rows each (4096 x
// 4096, GELU': 24 us; 8192 x 8192 sums alone: 23.5 us, 5.7 TB/s)
int colsum_parts(int64_t M, int N) {
  const int64_t cols = std::max(1, N / 256);
  return (int)std::max<int64_t>(1, std::min<int64_t>({256, (M + 31) / 32, (148 * 8 + cols - 1) / cols}));
}

template <typename T>
cudaError_t colsums_as(const ColSums &P, int count, int maxN, int act, bool join, cudaStream_t s) {
  constexpr int W = 32 * (16 / sizeof(T));
  const dim3 grid((maxN + W - 1) / W, P.parts, count);
  auto run = [&](auto kern) { return launch_kernel(kern, grid, 256, 0, s, P); };
  cudaError_t e;
  switch (act) {
    case MOE_DENSE_RELU: e = run(colsum_part_kernel<T, MOE_DENSE_RELU>); break;
    case MOE_DENSE_SILU: e = run(colsum_part_kernel<T, MOE_DENSE_SILU>); break;
    case MOE_DENSE_GELU: e = run(colsum_part_kernel<T, MOE_DENSE_GELU>); break;
    case MOE_DENSE_GELU_TANH: e = run(colsum_part_kernel<T, MOE_DENSE_GELU_TANH>); break;
    default: e = run(colsum_part_kernel<T, kNoAct>);
  }
  if (e != cudaSuccess || !join) return e;
  return launch_kernel(colsum_join_kernel<T>, dim3((maxN + 31) / 32, 1, count), 256, 0, s, P);
}

template <typename T, bool GATED>
cudaError_t simt_as(const DenseGemm &g, cudaStream_t s) {
  auto tiles = [&](int ts) { return ((g.M + ts - 1) / ts) * (((int64_t)g.N + ts - 1) / ts); };
  if (tiles(64) == 0) return cudaSuccess;
  const int64_t most = (int64_t)device_sms() * 8;
  return tiles(64) >= device_sms()
             ? launch_kernel(dense_simt_kernel<T, GATED, 64>, (unsigned)std::min(tiles(64), most), 256, 0, s, g)
             : launch_kernel(dense_simt_kernel<T, GATED, 32>, (unsigned)std::min(tiles(32), most), 256, 0, s, g);
}

}  // namespace

cudaError_t launch_dense_simt(const DenseGemm &g, cudaStream_t s) {
  const bool gated = g.epi == kDenseGated;
  if (g.dtype == MOE_F32) return gated ? simt_as<float, true>(g, s) : simt_as<float, false>(g, s);
  return gated ? simt_as<__nv_bfloat16, true>(g, s) : simt_as<__nv_bfloat16, false>(g, s);
}

size_t colsum_scratch(int64_t M, int N, int count) { return (size_t)colsum_parts(M, N) * N * 4 * count; }

cudaError_t launch_colsums(int act, int dtype, int64_t M, const ColSum *q, int count, float *part,
                           cudaStream_t s) {
  ColSums P{};
  int maxN = 0;
  bool grad = false, join = false;
  for (int i = 0; i < count; ++i) {
    P.q[i] = q[i];
    maxN = std::max(maxN, q[i].N);
    grad = grad || q[i].dz;
    join = join || q[i].out;
  }
  P.M = M;
  P.parts = colsum_parts(M, maxN);
  P.part = part;
  P.part_stride = maxN;
  return dtype == MOE_F32 ? colsums_as<float>(P, count, maxN, grad ? act : kNoAct, join, s)
                          : colsums_as<__nv_bfloat16>(P, count, maxN, grad ? act : kNoAct, join, s);
}

}  // namespace moe
