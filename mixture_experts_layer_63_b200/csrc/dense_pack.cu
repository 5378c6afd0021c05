// Operands of the tensor-core products that cannot be read as they lie.
//
// bf16 matrices whose lines are not 16-byte aligned are copied to aligned
// lines.  fp32 matrices are split into three bf16 matrices,
//   h = bf16(v),  m = bf16(v - h),  l = bf16(v - h - m),   v = h + m + l
// (each remainder is exact in fp32 and 3 x 8 significand bits hold fp32's
// 24), so that an fp32 product becomes six bf16 ones: h h', h m', m h', m m',
// h l', l h'; what is left out is below 2^-26 of the product.  An infinity or a
// NaN goes to the plane that meets one plane of the other operand only:
//   h = +-1 (NaN: 0),  m = 0,  l = v,
// so that it is multiplied by the other element's h, which has its sign, and
// never by a part that is 0 or of the other sign; two infinities meet each
// other's +-1.  The results are those of fp32 arithmetic.  The splits are
// bandwidth-bound (4 bytes read, 6 written an element; two 4096 x 4096 matrices
// in 55 us, 5.1 TB/s).
#include <algorithm>

#include "dense_internal.h"
#include "dense_math.cuh"

namespace moe {
namespace {

struct PackParams {
  PackJob job[kMaxPack];
  int64_t first[kMaxPack + 1];       // first 8-element piece of each job
  int n;
};

__device__ __forceinline__ void split3(float v, float &h, float &m, float &l) {
  h = __bfloat162float(__float2bfloat16_rn(v));
  if (isinf(h) && !isinf(v)) h = __bfloat162float(__float2bfloat16_rz(v));      // next to FLT_MAX
  const float r = v - h;
  m = __bfloat162float(__float2bfloat16_rn(r));
  l = r - m;
  if (!isfinite(v)) {
    h = isinf(v) ? copysignf(1.0f, v) : 0.0f;
    m = 0.0f;
    l = v;
  }
}

template <typename T>
__global__ void __launch_bounds__(256) pack_kernel(const __grid_constant__ PackParams P) {
  pdl_wait();
  pdl_trigger();
  for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < P.first[P.n]; i += gridDim.x * 256ll) {
    int j = 0;
    while (j + 1 < P.n && i >= P.first[j + 1]) ++j;
    const PackJob &J = P.job[j];
    const int64_t pieces = pack_ld(J.inner) / 8, at = i - P.first[j], line = at / pieces;
    const int64_t c = (at - line * pieces) * 8;
    const T *src = static_cast<const T *>(J.src) + line * J.ld + c;
    float v[8];
    if (c + 8 <= J.inner && (reinterpret_cast<uintptr_t>(src) & 15) == 0) {
#pragma unroll
      for (int q = 0; q < 8 * (int)sizeof(T) / 16; ++q)
        unpack16<T>(reinterpret_cast<const uint4 *>(src)[q], v + q * (16 / sizeof(T)));
    } else {
#pragma unroll
      for (int q = 0; q < 8; ++q) v[q] = c + q < J.inner ? to_f32(src[q]) : 0.0f;
    }
    __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(J.dst) + line * pack_ld(J.inner) + c;
    if (sizeof(T) == 2) {
      *reinterpret_cast<uint4 *>(dst) = pack16<__nv_bfloat16>(v);
    } else {
      const int64_t plane = J.lines * pack_ld(J.inner);
      float h[8], m[8], l[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) split3(v[q], h[q], m[q], l[q]);
      *reinterpret_cast<uint4 *>(dst) = pack16<__nv_bfloat16>(h);
      *reinterpret_cast<uint4 *>(dst + plane) = pack16<__nv_bfloat16>(m);
      *reinterpret_cast<uint4 *>(dst + 2 * plane) = pack16<__nv_bfloat16>(l);
    }
  }
}

}  // namespace

cudaError_t launch_pack(int dtype, const PackJob *jobs, int n, cudaStream_t s) {
  PackParams P{};
  P.n = n;
  for (int i = 0; i < n; ++i) {
    P.job[i] = jobs[i];
    P.first[i + 1] = P.first[i] + jobs[i].lines * (pack_ld(jobs[i].inner) / 8);
  }
  const unsigned grid = (unsigned)std::max<int64_t>(
      1, std::min<int64_t>((P.first[n] + 255) / 256, (int64_t)device_sms() * 8));
  return dtype == MOE_F32 ? launch_kernel(pack_kernel<float>, grid, 256, 0, s, P)
                          : launch_kernel(pack_kernel<__nv_bfloat16>, grid, 256, 0, s, P);
}

}  // namespace moe
