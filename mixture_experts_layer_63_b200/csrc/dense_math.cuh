// Element functions of the dense operators: activations, their derivatives,
// and loads / stores of one element in fp32.
#pragma once

#include "device_common.cuh"
#include "../../include/moe.h"

namespace moe {
namespace {

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void from_f32(float &d, float v) { d = v; }
__device__ __forceinline__ void from_f32(__nv_bfloat16 &d, float v) { d = __float2bfloat16_rn(v); }

// What rounding v to hi leaves for a low plane: nothing of what is no number or
// rounds to an infinity, so that the planes' sum is hi and not inf - inf.
__device__ __forceinline__ float rest_of(float v, float hi) { return fabsf(hi) <= 3.4028235e38f ? v - hi : 0.0f; }

// 16 bytes of T from fp32 values, and back
template <typename T>
__device__ __forceinline__ uint4 pack16(const float *v) {
  if (sizeof(T) == 4)
    return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
  return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                    pack_bf16x2(v[6], v[7]));
}

template <typename T>
__device__ __forceinline__ void unpack16(const uint4 &w, float *v) {
  const uint32_t q[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (sizeof(T) == 4) {
      v[i] = __uint_as_float(q[i]);
    } else {
      v[2 * i] = bf16_lo(q[i]);
      v[2 * i + 1] = bf16_hi(q[i]);
    }
  }
}

// Two fp32 operations an instruction (sm_100a), each rounded as its scalar form
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, z, w;\n\t"
      "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
      "fma.rn.f32x2 w, x, y, z;\n\tmov.b64 {%0, %1}, w;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, w;\n\t"
      "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "mul.rn.f32x2 w, x, y;\n\tmov.b64 {%0, %1}, w;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, w;\n\t"
      "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "add.rn.f32x2 w, x, y;\n\tmov.b64 {%0, %1}, w;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 two(float v) { return make_float2(v, v); }

// FAST (bf16 layers, whose results are rounded to 8 bits next): the hardware's
// approximate 2^v and 1 / v, 2^-22 off, denormals taken as zeros.  They spare
// the scaling around __expf and __fdividef.
__device__ __forceinline__ float ex2_fast(float v) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ float rcp_fast(float v) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
constexpr float kLog2e = 1.4426950408889634f;

// tanh-form GELU: 0.5 (1 + tanh(y)) = sigmoid(2 y), y = sqrt(2/pi) (v + 0.044715 v^3)
constexpr float kGeluA = 0.7978845608028654f;       // sqrt(2 / pi)
constexpr float kGeluB = 0.044715f;
constexpr float kGeluC = -2.0f * kGeluA * kLog2e;   // e^(-2 y) = 2^(v (C + C B v^2))

// 1 / (1 + e^-v), and of 2 y: SiLU's and the tanh form's factor of v
template <bool FAST, int ACT>
__device__ __forceinline__ float gate_of(float v) {
  constexpr bool TANH = ACT == MOE_DENSE_GELU_TANH;
  if (FAST) {
    const float g = TANH ? v * fmaf(kGeluC * kGeluB, v * v, kGeluC) : v * -kLog2e;
    return rcp_fast(ex2_fast(g) + 1.0f);
  }
  return 1.0f / (1.0f + expf(-(TANH ? 2.0f * kGeluA * (v + kGeluB * v * v * v) : v)));
}
template <int ACT>
__device__ __forceinline__ float2 gate_of2(float2 v) {
  const float2 g = ACT == MOE_DENSE_GELU_TANH
                       ? mul2(v, fma2(two(kGeluC * kGeluB), mul2(v, v), two(kGeluC)))
                       : mul2(v, two(-kLog2e));
  const float2 n = add2(make_float2(ex2_fast(g.x), ex2_fast(g.y)), two(1.0f));
  return make_float2(rcp_fast(n.x), rcp_fast(n.y));
}

// Normal distribution function for the bf16 layers' GELU, and e^(-v^2/2) on
// the way: Phi(-x) = e^(-x^2/2) t Q(t), t = 1 / (1 + x / (2 sqrt 2)), x >= 0,
// where t Q(t) is a degree-7 polynomial fitted (weighted least squares to a
// minimax error, float64) to half the scaled complementary error function of
// x / sqrt 2 on [0, 17]; relative error 2.4e-6 in fp32, in the tail too.
// Against erff and a second exponential: the column-sum pass over 4096 x 4096
// went from 33 to 28 us.
__device__ __forceinline__ float normal_cdf_fast(float v, float &e) {
  const float x = fabsf(v);
  e = ex2_fast(v * v * (-0.5f * kLog2e));
  const float t = rcp_fast(fmaf(0.35355339f, x, 1.0f));
  float q = 0.042448815f;
  q = fmaf(q, t, -0.17260440f);
  q = fmaf(q, t, 0.18664083f);
  q = fmaf(q, t, 0.024500929f);
  q = fmaf(q, t, 0.13870965f);
  q = fmaf(q, t, 0.13916363f);
  q = fmaf(q, t, 0.14113952f);
  const float tail = q * t * e;
  return v > 0.0f ? 1.0f - tail : tail;
}

// The same of two values, most of it two operations an instruction (the
// epilogues and the column sums are bound by instructions under GELU)
__device__ __forceinline__ float2 normal_cdf_fast2(float2 v, float2 &e) {
  const float2 x = make_float2(fabsf(v.x), fabsf(v.y));
  const float2 g = mul2(mul2(v, v), two(-0.5f * kLog2e));
  e = make_float2(ex2_fast(g.x), ex2_fast(g.y));
  const float2 y = fma2(two(0.35355339f), x, two(1.0f));
  const float2 t = make_float2(rcp_fast(y.x), rcp_fast(y.y));
  float2 q = two(0.042448815f);
  q = fma2(q, t, two(-0.17260440f));
  q = fma2(q, t, two(0.18664083f));
  q = fma2(q, t, two(0.024500929f));
  q = fma2(q, t, two(0.13870965f));
  q = fma2(q, t, two(0.13916363f));
  q = fma2(q, t, two(0.14113952f));
  const float2 tail = mul2(mul2(q, t), e), head = fma2(tail, two(-1.0f), two(1.0f));
  return make_float2(v.x > 0.0f ? head.x : tail.x, v.y > 0.0f ? head.y : tail.y);
}

// Call f with the activation as a compile-time constant: one branch for a
// whole row of elements (a switch an element, unrolled, cost more in branches
// and instruction fetches than the functions themselves: the gradient
// epilogue of 4096 x 2048 x 5632 took 192 us with it, against a 60 us product).
template <int V>
struct IntC {
  static constexpr int value = V;
};
template <typename F>
__device__ __forceinline__ void with_act(int act, F f) {
  switch (act) {
    case MOE_DENSE_RELU: f(IntC<MOE_DENSE_RELU>{}); break;
    case MOE_DENSE_SILU: f(IntC<MOE_DENSE_SILU>{}); break;
    case MOE_DENSE_GELU: f(IntC<MOE_DENSE_GELU>{}); break;
    case MOE_DENSE_GELU_TANH: f(IntC<MOE_DENSE_GELU_TANH>{}); break;
    default: f(IntC<MOE_DENSE_IDENTITY>{});
  }
}

// act(v).  A NaN stays a NaN (relu compares instead of taking a maximum).
template <bool FAST, int ACT>
__device__ __forceinline__ float act_fwd(float v) {
  if (ACT == MOE_DENSE_RELU) return v < 0.0f ? 0.0f : v;
  if (ACT == MOE_DENSE_SILU) return FAST ? v * gate_of<FAST, ACT>(v) : v / (1.0f + expf(-v));
  if (ACT == MOE_DENSE_GELU) {
    float e;
    return FAST ? v * normal_cdf_fast(v, e) : 0.5f * v * (1.0f + erff(v * 0.70710678118654752f));
  }
  if (ACT == MOE_DENSE_GELU_TANH) return v * gate_of<FAST, ACT>(v);
  return v;
}

// act(v) and act'(v); relu'(0) = 0, as in the MoE layer's backward pass, and a
// NaN stays a NaN in both
template <bool FAST, int ACT>
__device__ __forceinline__ void act_both(float v, float &f, float &d) {
  if (ACT == MOE_DENSE_RELU) {
    f = v < 0.0f ? 0.0f : v;
    d = v > 0.0f ? 1.0f : v <= 0.0f ? 0.0f : v;
  } else if (ACT == MOE_DENSE_SILU) {
    const float s = gate_of<FAST, ACT>(v);
    f = v * s;
    d = fmaf(f, 1.0f - s, s);
  } else if (ACT == MOE_DENSE_GELU) {
    float e, c;                            // e^(-v^2/2), normal distribution function
    if (FAST) {
      c = normal_cdf_fast(v, e);
    } else {
      e = expf(-0.5f * v * v);
      c = 0.5f * (1.0f + erff(v * 0.70710678118654752f));
    }
    f = v * c;
    d = fmaf(v, 0.3989422804014327f * e, c);
  } else if (ACT == MOE_DENSE_GELU_TANH) {
    const float s = gate_of<FAST, ACT>(v);
    f = v * s;
    // (s (1 - s) is 0 long before the bound, which keeps 0 * inf out)
    d = fmaf(f * (1.0f - s), fmaf(6.0f * kGeluA * kGeluB, fminf(v * v, 1e8f), 2.0f * kGeluA), s);
  } else {
    f = v;
    d = 1.0f;
  }
}

// Two values at once, to the same bits
template <bool FAST, int ACT>
__device__ __forceinline__ float2 act_fwd2(float2 v) {
  if (FAST && ACT == MOE_DENSE_GELU) {
    float2 e;
    return mul2(v, normal_cdf_fast2(v, e));
  }
  if (FAST && (ACT == MOE_DENSE_SILU || ACT == MOE_DENSE_GELU_TANH)) return mul2(v, gate_of2<ACT>(v));
  return make_float2(act_fwd<FAST, ACT>(v.x), act_fwd<FAST, ACT>(v.y));
}
template <bool FAST, int ACT>
__device__ __forceinline__ void act_both2(float2 v, float2 &f, float2 &d) {
  if (FAST && ACT == MOE_DENSE_GELU) {
    float2 e;
    const float2 c = normal_cdf_fast2(v, e);
    f = mul2(v, c);
    d = fma2(v, mul2(two(0.3989422804014327f), e), c);
  } else if (FAST && (ACT == MOE_DENSE_SILU || ACT == MOE_DENSE_GELU_TANH)) {
    const float2 s = gate_of2<ACT>(v), r = fma2(s, two(-1.0f), two(1.0f));
    f = mul2(v, s);
    if (ACT == MOE_DENSE_SILU) {
      d = fma2(f, r, s);
    } else {
      const float2 q = mul2(v, v);
      d = fma2(mul2(f, r),
               fma2(two(6.0f * kGeluA * kGeluB), make_float2(fminf(q.x, 1e8f), fminf(q.y, 1e8f)), two(2.0f * kGeluA)), s);
    }
  } else {
    act_both<FAST, ACT>(v.x, f.x, d.x);
    act_both<FAST, ACT>(v.y, f.y, d.y);
  }
}

}  // namespace
}  // namespace moe
