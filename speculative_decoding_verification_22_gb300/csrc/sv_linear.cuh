// sv_linear.cuh -- what the forms of the products with an epilogue share:
// activations, and loads and stores by element type.
#pragma once

#include "sv_target.cuh"

namespace sv {

// 1 / x of the special-function unit (2^-23 relative; 0 for an infinity).
__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The activations keep their relative accuracy where they come near zero for
// negative v: erfc in place of 1 + erf, a logistic function in place of 1 + tanh.
template <int kAct>
__device__ __forceinline__ float activate(float v) {
  if constexpr (kAct == SV_ACT_RELU) return v > 0.0f || isnan(v) ? v : 0.0f;
  if constexpr (kAct == SV_ACT_GELU) return 0.5f * v * erfcf(-0.70710678118654752f * v);
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
