// sv_block_norm.cu -- the norms after and before a block with its gate, its
// scale and the residual:
//
//   y = x / sqrt(mean(x^2) + eps) * post,  h = residual + s * gate * y,
//   out = h / sqrt(mean(h^2) + eps) * weight
#include "sv_target.cuh"

namespace sv {
namespace {

constexpr int kThreads = 512;

template <class Op>
__device__ __forceinline__ float block_reduce(float v, float *red, Op op) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = op(v, __shfl_xor_sync(0xffffffffu, v, o));
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  float r = red[0];
  for (int i = 1; i < kThreads / 32; ++i) r = op(r, red[i]);
  return r;
}

// One block a row, the row read once for each of the sums, the maximum (row
// scale) and the output.  A thread rereads only elements that it writes itself
// and writes in the last pass alone, so the in-place forms hold.
template <class T>
__global__ void __launch_bounds__(kThreads) block_norm_any_kernel(const sv_block_norm_t P) {
  __shared__ float red[3][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t row = blockIdx.x;
  const int d = static_cast<int>(P.d);
  const T *x = static_cast<const T *>(P.x) + row * P.x_stride;
  const T *r = static_cast<const T *>(P.residual) + row * P.residual_stride;
  const T *gate = P.gate ? static_cast<const T *>(P.gate) + row * P.gate_row : nullptr;
  const T *post = static_cast<const T *>(P.post_weight), *w = static_cast<const T *>(P.weight);
  T *ro = P.residual_out ? static_cast<T *>(P.residual_out) + row * P.residual_out_stride
                         : nullptr;
  pdl_wait();
  pdl_launch_dependents();
  const auto add = [](float a, float b) { return a + b; };
  const auto most = [](float a, float b) { return max_nan(a, b); };
  // a warp takes 128 columns at a time, lane l the columns l, l + 32, ...
  auto each = [&](auto &&f) {
    for (int g = warp * 128; g < d; g += kThreads * 4) f(g);
  };
  float inv_x = 1.0f;
  if (post) {
    float ss = 0.0f;
    each([&](int g) {
      for (int i = g + lane; i < min(g + 128, d); i += 32) {
        const float v = to_float(x[i]);
        ss = fmaf(v, v, ss);
      }
    });
    inv_x = 1.0f / sqrtf(block_reduce(ss, red[0], add) / static_cast<float>(d) + P.eps);
  }
  auto at = [&](int i) {
    float y = to_float(x[i]);
    if (post) y = y * inv_x * to_float(post[i]);
    y *= P.branch_scale;
    if (gate) y *= to_float(gate[i * P.gate_col]);
    return to_float(r[i]) + y;
  };
  float ss = 0.0f;
  each([&](int g) {
    for (int i = g + lane; i < min(g + 128, d); i += 32) {
      const float h = at(i);
      ss = fmaf(h, h, ss);
    }
  });
  const float inv = 1.0f / sqrtf(block_reduce(ss, red[1], add) / static_cast<float>(d) + P.eps);
  float s = 0.0f, inv_s = 0.0f;
  if (P.group == 0) {
    float m = 0.0f;
    each([&](int g) {
      for (int i = g + lane; i < min(g + 128, d); i += 32)
        m = max_nan(m, fabsf(at(i) * inv * to_float(w[i])));
    });
    s = max_nan(block_reduce(m, red[2], most), 1e-30f) / 448.0f;
    inv_s = 1.0f / s;
    if (threadIdx.x == 0) P.scale[row] = s;
  }
  each([&](int g) {
    float y[4], m = 0.0f;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int i = g + 32 * k + lane;
      y[k] = 0.0f;
      if (i < d) {
        const float h = at(i);
        if (ro) ro[i] = from_float<T>(h);
        y[k] = h * inv * to_float(w[i]);
      }
      m = max_nan(m, fabsf(y[k]));
    }
    if (P.group > 0) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
      s = max_nan(m, 1e-30f) / 448.0f;
      inv_s = 1.0f / s;
      if (lane == 0) P.scale[row * ((d + 127) / 128) + g / 128] = s;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int i = g + 32 * k + lane;
      if (i >= d) break;
      if (P.group >= 0)
        static_cast<uint8_t *>(P.out)[row * d + i] = static_cast<uint8_t>(
            __nv_cvt_float_to_fp8(y[k] * inv_s, __NV_SATFINITE, __NV_E4M3));
      else
        static_cast<T *>(P.out)[row * P.out_stride + i] = from_float<T>(y[k]);
    }
  });
}

template <class T>
cudaError_t launch_typed(const sv_block_norm_t &a, cudaStream_t stream) {
  return launch_chained(block_norm_any_kernel<T>, dim3(static_cast<unsigned>(a.rows)),
                        dim3(kThreads), 0, stream, a);
}

}  // namespace

cudaError_t launch_block_norm(const sv_block_norm_t &a, int num_sms, cudaStream_t stream) {
  switch (a.dtype) {
    case SV_BF16: return launch_typed<__nv_bfloat16>(a, stream);
    case SV_FP16: return launch_typed<__half>(a, stream);
    default: return launch_typed<float>(a, stream);
  }
}

}  // namespace sv
