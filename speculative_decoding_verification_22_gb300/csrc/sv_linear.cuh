// sv_linear.cuh -- what the forms of the products with an epilogue share:
// activations, and loads and stores by element type.
#pragma once

#include "sv_target.cuh"
#include "sv_tmem.cuh"

namespace sv {

// 1 / x of the special-function unit (2^-23 relative; 0 for an infinity).
__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// v Phi(v) = v erfc(-v / sqrt 2) / 2.  With z = |v| / sqrt 2 and t = 1 / (1 + z / 2),
// erfc(z) = t exp(-z^2) 2^P(t), which is the form of a published approximation of erfc
// (Press et al., "Numerical Recipes", section 6.2); P is a polynomial of degree 9 that was
// fitted here to log2(erfc(z) exp(z^2) / t) for z from 0 to 13.5 (weighted least squares
// towards the least maximum), to 3e-7.  The rounded exponent adds about v^2 2^-24 where v
// is negative: measured against 64 bits 5e-7 relative from -2 to 6, 1.4e-6 down to -5,
// 3.5e-6 to -9, 8e-6 to -13.  erfcf takes three times the instructions.
__device__ __forceinline__ float gelu(float v) {
  const float t = rcp(fmaf(fabsf(v), 0.35355339059327376f, 1.0f));
  float q = 0.2301653027534485f;
  q = fmaf(q, t, -1.0967739820480347f);
  q = fmaf(q, t, 1.9376541376113892f);
  q = fmaf(q, t, -1.3609977960586548f);
  q = fmaf(q, t, 0.17759618163108826f);
  q = fmaf(q, t, -0.15300674736499786f);
  q = fmaf(q, t, 0.10209780931472778f);
  q = fmaf(q, t, 0.5470234751701355f);
  q = fmaf(q, t, 1.441956639289856f);
  q = fmaf(q, t, -1.8257149457931519f);
  const float tail = t * ex2(fmaf(v * -0.72134752044448170f, v, q));  // erfc(z)
  return 0.5f * v * (v > 0.0f ? 2.0f - tail : tail);
}

// The activations keep their relative accuracy where they come near zero for
// negative v: erfc in place of 1 + erf, a logistic function in place of 1 + tanh.
template <int kAct>
__device__ __forceinline__ float activate(float v) {
  if constexpr (kAct == SV_ACT_RELU) return v > 0.0f || isnan(v) ? v : 0.0f;
  if constexpr (kAct == SV_ACT_GELU) return gelu(v);
  if constexpr (kAct == SV_ACT_GELU_TANH)
    // (1 + tanh u) / 2 = 1 / (1 + exp(-2 u)), u = sqrt(2 / pi) (v + 0.044715 v^3)
    return v * rcp(1.0f + expf(-1.5957691216057308f * fmaf(0.044715f * v * v, v, v)));
  if constexpr (kAct == SV_ACT_SILU) return v * rcp(1.0f + expf(-v));
  return v;
}
__device__ __forceinline__ float activate(float v, int act) {
  switch (act) {
    case SV_ACT_RELU: return activate<SV_ACT_RELU>(v);
    case SV_ACT_GELU: return activate<SV_ACT_GELU>(v);
    case SV_ACT_GELU_TANH: return activate<SV_ACT_GELU_TANH>(v);
    case SV_ACT_SILU: return activate<SV_ACT_SILU>(v);
    default: return v;
  }
}

// Four values at a time and no inlining: unrolled over an epilogue's values the
// activations are tens of KB of code, which a tile that is a CTA's only one waits for.
template <int kAct>
__device__ __noinline__ float4 activate4_call(float4 v) {
  return make_float4(activate<kAct>(v.x), activate<kAct>(v.y), activate<kAct>(v.z),
                     activate<kAct>(v.w));
}
__device__ __forceinline__ float4 activate4(float4 v, int act) {
  switch (act) {
    case SV_ACT_RELU: return activate4_call<SV_ACT_RELU>(v);
    case SV_ACT_GELU: return activate4_call<SV_ACT_GELU>(v);
    case SV_ACT_GELU_TANH: return activate4_call<SV_ACT_GELU_TANH>(v);
    case SV_ACT_SILU: return activate4_call<SV_ACT_SILU>(v);
    default: return v;
  }
}

// Eight at a time: twice as many independent chains in a call.
struct Eight {
  float4 a, b;
};
template <int kAct>
__device__ __noinline__ Eight activate8_call(Eight v) {
  Eight r;
  r.a = make_float4(activate<kAct>(v.a.x), activate<kAct>(v.a.y), activate<kAct>(v.a.z),
                    activate<kAct>(v.a.w));
  r.b = make_float4(activate<kAct>(v.b.x), activate<kAct>(v.b.y), activate<kAct>(v.b.z),
                    activate<kAct>(v.b.w));
  return r;
}
__device__ __forceinline__ Eight activate8(Eight v, int act) {
  switch (act) {
    case SV_ACT_RELU: return activate8_call<SV_ACT_RELU>(v);
    case SV_ACT_GELU: return activate8_call<SV_ACT_GELU>(v);
    case SV_ACT_GELU_TANH: return activate8_call<SV_ACT_GELU_TANH>(v);
    case SV_ACT_SILU: return activate8_call<SV_ACT_SILU>(v);
    default: return v;
  }
}

__device__ __forceinline__ float load_any(const void *p, int64_t at, int dtype) {
  if (dtype == SV_BF16) return __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[at]);
  if (dtype == SV_FP16) return __half2float(static_cast<const __half *>(p)[at]);
  return static_cast<const float *>(p)[at];
}
__device__ __forceinline__ void store_any(void *p, int64_t at, float x, int dtype) {
  if (dtype == SV_BF16)
    static_cast<__nv_bfloat16 *>(p)[at] = __float2bfloat16_rn(x);
  else if (dtype == SV_FP16)
    static_cast<__half *>(p)[at] = __float2half_rn(x);
  else
    static_cast<float *>(p)[at] = x;
}

}  // namespace sv
