// Global gradient norm over a list of tensors, and clipping by it.
//
//   n = sqrt(sum over all tensors of g^2),  c = min(1, max_norm / (n + 1e-6)),
//   g <- c g
//
// Two kernels.  The first reads every element once: the list is cut into
// chunks, dealt round-robin over a fixed grid; each block leaves one partial
// sum.  In the second every block adds the partial sums in the same fixed
// order (so the norm is the same bits in every block and on every call) and
// scales its chunks.  Squares and sums are in fp64: an fp32 square overflows
// beyond 1.8e19 and a sum of 2^28 squares loses the small ones.
//
// Bound by DRAM: over 2^28 fp32 elements the norm takes 153 us (7.0 TB/s), the
// scaling 348 us (6.0 TB/s); a short list takes its two launches, 11 us with
// the binding.  512 threads with four 16-byte loads in flight each, two blocks
// an SM: 64 KB an SM in flight, which covers the latency at that rate.
#include <algorithm>

#include "dense_internal.h"
#include "dense_math.cuh"

namespace moe {
namespace {

constexpr int kClipThreads = 512;
constexpr int kClipTensors = 240;      // tensors of one launch (its table is a kernel argument)
constexpr int kClipBlocksPerSm = 2;
constexpr int kClipMaxBlocks = 160 * kClipBlocksPerSm;      // partial sums of one launch at most
constexpr double kClipEps = 1e-6;

struct ClipTable {
  const void *src[kClipTensors];
  void *dst[kClipTensors];
  int64_t n[kClipTensors];
  int32_t first[kClipTensors + 1];     // first chunk of each tensor
  uint8_t f32[kClipTensors];
  int32_t count;
  int32_t chunk;                       // elements of a chunk (a multiple of 8)
};

__device__ __forceinline__ int tensor_of(const ClipTable &t, int chunk) {
  int lo = 0, hi = t.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (t.first[mid] <= chunk) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// f(i, piece i) for the 16-byte pieces of p where it is 16-byte aligned (four
// loads in flight a thread; chunks start at multiples of 8 elements), and
// f(i, element i) for what is left, or for everything
template <typename T, typename F>
__device__ __forceinline__ void each(const T *p, int64_t n, bool vec, F f) {
  constexpr int V = 16 / sizeof(T), R = 4;
  int64_t done = 0;
  if (vec) {
    const int nv = (int)(n / V);
    const uint4 *q = reinterpret_cast<const uint4 *>(p);
    int i = threadIdx.x;
    for (; i + (R - 1) * kClipThreads < nv; i += R * kClipThreads) {
      uint4 w[R];
#pragma unroll
      for (int k = 0; k < R; ++k) w[k] = q[i + k * kClipThreads];
#pragma unroll
      for (int k = 0; k < R; ++k) f(i + k * kClipThreads, w[k]);
    }
    for (; i < nv; i += kClipThreads) f(i, q[i]);
    done = (int64_t)nv * V;
  }
  for (int64_t i = done + threadIdx.x; i < n; i += kClipThreads) f(i, p[i]);
}

template <typename T>
__device__ __forceinline__ double square_sum(const T *p, int64_t n) {
  double acc[2] = {0.0, 0.0};
  struct Add {
    double *acc;
    __device__ void one(float v, int i) { acc[i & 1] = fma((double)v, (double)v, acc[i & 1]); }
    __device__ void operator()(int64_t, T v) { one(to_f32(v), 0); }
    __device__ void operator()(int64_t, const uint4 &w) {
      const uint32_t q[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (sizeof(T) == 4) {
          one(__uint_as_float(q[i]), i);
        } else {
          one(bf16_lo(q[i]), 0);
          one(bf16_hi(q[i]), 1);
        }
      }
    }
  };
  each(p, n, (reinterpret_cast<uintptr_t>(p) & 15) == 0, Add{acc});
  return acc[0] + acc[1];
}

__device__ __forceinline__ double block_sum(double v, double *sh) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  if (threadIdx.x % 32 == 0) sh[threadIdx.x / 32] = v;
  __syncthreads();
  double t = 0.0;
  for (int i = 0; i < kClipThreads / 32; ++i) t += sh[i];
  return t;
}

__global__ void __launch_bounds__(kClipThreads) clip_norm_kernel(const __grid_constant__ ClipTable t,
                                                                 double *part) {
  __shared__ double sh[kClipThreads / 32];
  pdl_wait();
  pdl_trigger();
  double sum = 0.0;
  for (int c = blockIdx.x; c < t.first[t.count]; c += gridDim.x) {
    const int i = tensor_of(t, c);
    const int64_t at = (int64_t)(c - t.first[i]) * t.chunk, n = min((int64_t)t.chunk, t.n[i] - at);
    sum += t.f32[i] ? square_sum(static_cast<const float *>(t.src[i]) + at, n)
                    : square_sum(static_cast<const __nv_bfloat16 *>(t.src[i]) + at, n);
  }
  sum = block_sum(sum, sh);
  if (threadIdx.x == 0) part[blockIdx.x] = sum;
}

template <typename T>
__device__ __forceinline__ void scale(const T *p, T *q, int64_t n, float c) {
  struct Mul {
    T *q;
    float c;
    __device__ void operator()(int64_t i, T v) { from_f32(q[i], to_f32(v) * c); }
    __device__ void operator()(int64_t i, const uint4 &w) {
      uint32_t r[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int k = 0; k < 4; ++k)
        r[k] = sizeof(T) == 4 ? __float_as_uint(__uint_as_float(r[k]) * c)
                              : pack_bf16x2(bf16_lo(r[k]) * c, bf16_hi(r[k]) * c);
      reinterpret_cast<uint4 *>(q)[i] = make_uint4(r[0], r[1], r[2], r[3]);
    }
  };
  each(p, n, ((reinterpret_cast<uintptr_t>(p) | reinterpret_cast<uintptr_t>(q)) & 15) == 0, Mul{q, c});
}

// nparts partial sums -> norm; then dst = c * src (max_norm >= 0).  A tensor
// scaled in place by exactly 1 keeps its bits, so it is not touched.
__global__ void __launch_bounds__(kClipThreads) clip_scale_kernel(const __grid_constant__ ClipTable t,
                                                                  const double *part, int nparts,
                                                                  float max_norm, float *norm) {
  __shared__ double sh[kClipThreads / 32];
  pdl_wait();
  pdl_trigger();
  double sum = 0.0;
  for (int i = threadIdx.x; i < nparts; i += kClipThreads) sum += part[i];
  const double n = sqrt(block_sum(sum, sh));
  if (norm && blockIdx.x == 0 && threadIdx.x == 0) *norm = (float)n;
  if (max_norm < 0.0f) return;
  const double ratio = (double)max_norm / (n + kClipEps);
  // a NaN norm gives a NaN factor; no limit, no factor, whatever the norm
  const float c = ratio > 1.0 || isinf(max_norm) ? 1.0f : (float)ratio;
  // last chunks first: the norm's pass read them last, so they may still be in L2
  for (int k = t.first[t.count] - 1 - blockIdx.x; k >= 0; k -= gridDim.x) {
    const int i = tensor_of(t, k);
    if (c == 1.0f && t.dst[i] == t.src[i]) continue;
    const int64_t at = (int64_t)(k - t.first[i]) * t.chunk, m = min((int64_t)t.chunk, t.n[i] - at);
    if (t.f32[i])
      scale(static_cast<const float *>(t.src[i]) + at, static_cast<float *>(t.dst[i]) + at, m, c);
    else
      scale(static_cast<const __nv_bfloat16 *>(t.src[i]) + at, static_cast<__nv_bfloat16 *>(t.dst[i]) + at, m,
            c);
  }
}

int launches_of(int32_t count) { return (count + kClipTensors - 1) / kClipTensors; }

}  // namespace

size_t clip_scratch(int32_t count) {
  return (size_t)std::max(1, launches_of(count)) * kClipMaxBlocks * sizeof(double);
}

cudaError_t launch_clip(const moe_grad *g, int32_t count, float max_norm, float *norm, double *part,
                        cudaStream_t s) {
  int64_t total = 0;
  for (int32_t i = 0; i < count; ++i) total += g[i].n;
  const int blocks = std::min(kClipMaxBlocks, device_sms() * kClipBlocksPerSm);
  // several chunks a block on large lists, at least 4096 elements each
  const int64_t share = (total / blocks / 4 + 1023) / 1024 * 1024;
  const int32_t chunk = (int32_t)std::min<int64_t>(65536, std::max<int64_t>(4096, share));
  const int groups = std::max(1, launches_of(count));
  int nparts = 0;
  for (int pass = 0; pass < 2; ++pass) {
    for (int q = 0; q < (pass == 1 && max_norm < 0.0f ? 1 : groups); ++q) {
      ClipTable t;
      t.count = 0;
      t.chunk = chunk;
      t.first[0] = 0;
      int64_t chunks = 0;
      for (int32_t i = q * kClipTensors; i < std::min(count, (q + 1) * kClipTensors); ++i) {
        const int k = t.count;
        if (g[i].n == 0) continue;
        t.src[k] = g[i].src;
        t.dst[k] = g[i].dst;
        t.n[k] = g[i].n;
        t.f32[k] = g[i].dtype == MOE_F32;
        chunks += (g[i].n + chunk - 1) / chunk;
        t.first[k + 1] = (int32_t)chunks;
        ++t.count;
      }
      const int grid = (int)std::max<int64_t>(1, std::min<int64_t>(blocks, chunks));
      cudaError_t e;
      if (pass == 0) {
        e = launch_kernel(clip_norm_kernel, grid, kClipThreads, 0, s, t, part + nparts);
        nparts += grid;
      } else {
        e = launch_kernel(clip_scale_kernel, max_norm < 0.0f ? 1 : grid, kClipThreads, 0, s, t, part, nparts,
                          max_norm, q == 0 ? norm : nullptr);
      }
      if (e != cudaSuccess) return e;
    }
  }
  return cudaSuccess;
}

}  // namespace moe
