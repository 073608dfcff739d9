// sv_log_probs.cu -- log probabilities of given tokens, entropy and the top
// alternatives of logit rows:
//
//   z = x / T, lse = log sum exp z;  z_t - lse;  H = -sum p (z - lse)
//
// With m the row's maximum and d = (x - m) / T <= 0, s = sum exp d and
// t = sum d exp d: lse - m / T = log s and H = log s - t / s.
#include <cmath>

#include "sv_target.cuh"

namespace sv {
namespace {

constexpr int kThreads = 512;

// Order of the alternatives: the larger logit first, of equal ones the smaller
// id.  The logit's bits become an unsigned number of the same order; -0 counts
// as +0.
__device__ __forceinline__ uint64_t order_key(float x, int id) {
  const uint32_t b = __float_as_uint(x + 0.0f);
  const uint32_t u = b & 0x80000000u ? ~b : b | 0x80000000u;
  return static_cast<uint64_t>(u) << 32 | static_cast<uint32_t>(~id);
}

template <class V, class Op>
__device__ __forceinline__ V block_reduce(V v, V *red, Op op) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = op(v, __shfl_xor_sync(0xffffffffu, v, o));
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  V r = red[0];
  for (int i = 1; i < kThreads / 32; ++i) r = op(r, red[i]);
  return r;
}

template <class T>
__global__ void __launch_bounds__(kThreads)
    log_probs_kernel(const sv_log_probs_t P, int *status) {
  __shared__ float red[32];
  __shared__ uint64_t best[32];
  const int64_t row = blockIdx.x;
  const T *x = static_cast<const T *>(P.logits) + row * P.stride;
  const int V = static_cast<int>(P.V);
  pdl_wait();
  pdl_launch_dependents();
  float m = -INFINITY;
  for (int i = threadIdx.x; i < V; i += kThreads) m = max_nan(m, to_float(x[i]));
  m = block_reduce(m, red, [](float a, float b) { return max_nan(a, b); });
  const bool fine = isfinite(m);
  const float inv_t = 1.0f / P.temperature;
  float s = 0.0f, t = 0.0f;
  for (int i = threadIdx.x; i < V; i += kThreads) {
    const float d = (to_float(x[i]) - m) * inv_t;
    const float e = expf(d);
    s += e;
    if (e > 0.0f) t = fmaf(d, e, t);
  }
  const auto add = [](float a, float b) { return a + b; };
  s = block_reduce(s, red, add);
  t = block_reduce(t, red, add);
  const float log_s = fine ? logf(s) : NAN;
  if (threadIdx.x == 0 && P.entropy) P.entropy[row] = log_s - t / s;
  for (int i = threadIdx.x; i < P.n; i += kThreads) {
    const int id = P.tokens[row * P.n + i];
    float y = 0.0f;
    if (id >= 0 && id < V) {
      y = (to_float(x[id]) - m) * inv_t - log_s;
    } else if (id != -1) {
      y = NAN;
      set_status(status, SV_ERR_TOKEN);
    }
    P.log_probs[row * P.n + i] = y;
  }
  uint64_t last = ~0ull;
  for (int j = 0; j < P.top; ++j) {
    uint64_t b = 0;
    if (fine)
      for (int i = threadIdx.x; i < V; i += kThreads) {
        const uint64_t k = order_key(to_float(x[i]), i);
        if (k < last && k > b) b = k;
      }
    last = block_reduce(b, best, [](uint64_t a, uint64_t c) { return a > c ? a : c; });
    if (threadIdx.x == 0) {
      const int id = fine ? static_cast<int>(~static_cast<uint32_t>(last)) : -1;
      P.top_ids[row * P.top + j] = id;
      P.top_log_probs[row * P.top + j] =
          fine ? (to_float(x[id]) - m) * inv_t - log_s : NAN;
    }
  }
}

template <class T>
cudaError_t launch_typed(const sv_log_probs_t &a, int *status, cudaStream_t stream) {
  return launch_chained(log_probs_kernel<T>, dim3(static_cast<unsigned>(a.rows)),
                        dim3(kThreads), 0, stream, a, status);
}

}  // namespace

int log_probs_checks(const sv_log_probs_t &a) {
  if ((a.dtype != SV_BF16 && a.dtype != SV_FP16 && a.dtype != SV_FP32) ||
      !(a.temperature > 0.0f) || !std::isfinite(a.temperature) ||
      !std::isfinite(1.0f / a.temperature) || a.n < 0)
    return SV_ERR_ARG;
  constexpr int64_t kMost = int64_t(1) << 24;
  if (a.V < 1 || a.V > kMost || a.top < 0 || a.top > SV_MAX_TOP || a.top > a.V ||
      a.n > (1 << 16) || a.rows < 0 || a.rows > kMost)
    return SV_ERR_SHAPE;
  if (a.rows == 0) return SV_OK;
  if (!a.logits || (a.n && (!a.tokens || !a.log_probs)) ||
      (a.top && (!a.top_ids || !a.top_log_probs)))
    return SV_ERR_ARG;
  if (a.rows > 1 && a.stride < a.V) return SV_ERR_SHAPE;
  auto at = [](const void *p, size_t n) { return (reinterpret_cast<uintptr_t>(p) % n) == 0; };
  return at(a.logits, a.dtype == SV_FP32 ? 4 : 2) && at(a.tokens, 4) && at(a.log_probs, 4) &&
                 at(a.entropy, 4) && at(a.top_ids, 4) && at(a.top_log_probs, 4)
             ? SV_OK
             : SV_ERR_ALIGN;
}

cudaError_t launch_log_probs(const sv_log_probs_t &a, int num_sms, int *status,
                             cudaStream_t stream) {
  switch (a.dtype) {
    case SV_BF16: return launch_typed<__nv_bfloat16>(a, status, stream);
    case SV_FP16: return launch_typed<__half>(a, status, stream);
    default: return launch_typed<float>(a, status, stream);
  }
}

}  // namespace sv
