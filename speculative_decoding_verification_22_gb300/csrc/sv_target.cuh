// sv_target.cuh -- definitions shared by the operators of spec_target.h and spec_layer.h:
// the handle, launch interfaces, and element conversions.
#pragma once

#include <cuda_bf16.h>

#include "../../include/spec_layer.h"
#include "sv_internal.cuh"

// The handle of the C ABI.
struct spec_target {
  int device = 0;
  int num_sms = 0;
  int smem_optin = 0;
  uint64_t wait_limit_ns = 1000000000ull;
  int *status = nullptr;   // device: first error since it was last read
  float *scratch = nullptr;  // device: partial results
  size_t scratch_bytes = 0;
  // Clusters of 1..8 CTAs that run at once, one CTA an SM: asked for the 8-bit product, and
  // the same for the 16-bit products' kernels (76, 46, 36, 28, 23, 15, 15 from two CTAs on).
  int clusters[9] = {};
};

namespace sv {

// ---- element conversions ---------------------------------------------------
template <class T>
__device__ __forceinline__ float to_float(T x);
template <>
__device__ __forceinline__ float to_float(float x) { return x; }
template <>
__device__ __forceinline__ float to_float(__half x) { return __half2float(x); }
template <>
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
template <class T>
__device__ __forceinline__ T from_float(float x);
template <>
__device__ __forceinline__ float from_float(float x) { return x; }
template <>
__device__ __forceinline__ __half from_float(float x) { return __float2half_rn(x); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_float(float x) { return __float2bfloat16_rn(x); }

// Eight consecutive elements as they lie in memory: 16 bytes of a 16-bit
// type, 32 of fp32.
template <class T>
struct alignas(16) Vec8 {
  T e[8];
};
template <class T>
__device__ __forceinline__ Vec8<T> load8(const T *p) {
  Vec8<T> v;
  constexpr int n = sizeof(Vec8<T>) / 16;
#pragma unroll
  for (int i = 0; i < n; ++i)
    reinterpret_cast<uint4 *>(&v)[i] = reinterpret_cast<const uint4 *>(p)[i];
  return v;
}
template <class T>
__device__ __forceinline__ void store8(T *p, const Vec8<T> &v) {
  constexpr int n = sizeof(Vec8<T>) / 16;
#pragma unroll
  for (int i = 0; i < n; ++i)
    reinterpret_cast<uint4 *>(p)[i] = reinterpret_cast<const uint4 *>(&v)[i];
}

// Maximum that keeps a NaN.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// ---- launch interfaces -----------------------------------------------------
struct NormParams {
  const void *x, *res, *w;
  void *out;         // dtype rows or E4M3 bytes
  void *res_out;
  float *scale;      // quant only
  int64_t xs, rs, os, ros, rows;
  int d, dtype, quant;  // quant: 0 none, 1 per 128 columns, 2 per row
  float eps;
};
cudaError_t launch_norm(const NormParams &P, int num_sms, cudaStream_t stream);

cudaError_t launch_rope_append(const sv_rope_append_t &a, int *status, cudaStream_t stream);

struct MatmulParams {
  const uint8_t *a, *w;
  const float *as, *ws;
  void *out;
  int64_t os;
  int M, N, K, kb, out_dtype;
};
// Fills h.clusters.
cudaError_t plan_matmul_fp8(spec_target &h);
int launch_matmul_fp8(const spec_target &h, const MatmulParams &P, cudaStream_t stream);

int launch_attention(const spec_target &h, const sv_attention_t &a, cudaStream_t stream);

cudaError_t launch_tree_mask(const int32_t *parents, int B, int N, int32_t *mask, int *status,
                             cudaStream_t stream);

// linear (wu NULL) and gated linear: w is the weight, or the gate's.
struct LinearParams {
  const void *x, *w, *wu, *bias, *bias_u, *res;
  void *out;
  int64_t xs, ws, wus, rs, os;
  int64_t M, N, K;
  int dtype, out_dtype, act;
};
int launch_linear(const spec_target &h, const LinearParams &P, cudaStream_t stream);

cudaError_t launch_block_norm(const sv_block_norm_t &a, int num_sms, cudaStream_t stream);

int log_probs_checks(const sv_log_probs_t &a);
cudaError_t launch_log_probs(const sv_log_probs_t &a, int num_sms, int *status,
                             cudaStream_t stream);

// Launch with programmatic stream serialisation: the kernel waits for what
// precedes it (griddepcontrol.wait) before it touches global memory.
template <class... K, class... A>
cudaError_t launch_chained(void (*fn)(K...), dim3 grid, dim3 block, size_t smem,
                           cudaStream_t stream, A... args) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, fn, static_cast<K>(args)...);
}

}  // namespace sv
