// sv_linear.cu -- products with an epilogue, general form:
//
//   out = act(x w^T + bias) + residual
//   out = act(x wg^T + bg) * (x wu^T + bu)
//
// fp32 arithmetic on operands of any type, stride and alignment: a block of 256
// threads holds a 64 x 64 tile of the output, 4 x 4 a thread, and walks K in
// steps of 16 through shared memory.
#include "sv_linear_tc.cuh"

namespace sv {
namespace {

constexpr int kTile = 64, kStep = 16, kGenThreads = 256;

template <class T, bool kGated>
__global__ void __launch_bounds__(kGenThreads) linear_general_kernel(const LinearParams P) {
  __shared__ float sx[kStep][kTile + 4], sw[kGated ? 2 : 1][kStep][kTile + 4];
  const int64_t m0 = static_cast<int64_t>(blockIdx.y) * kTile;
  const int64_t n0 = static_cast<int64_t>(blockIdx.x) * kTile;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;  // columns, rows 4 t ..
  const int lk = threadIdx.x & 15, lr = threadIdx.x >> 4;  // loads: K element, row
  const T *x = static_cast<const T *>(P.x);
  const T *w[2] = {static_cast<const T *>(P.w), static_cast<const T *>(P.wu)};
  const int64_t ws[2] = {P.ws, P.wus};
  pdl_wait();
  pdl_launch_dependents();
  float acc[kGated ? 2 : 1][4][4] = {};
  for (int64_t k0 = 0; k0 < P.K; k0 += kStep) {
    const bool kin = k0 + lk < P.K;
#pragma unroll
    for (int r = lr; r < kTile; r += 16) {
      sx[lk][r] = kin && m0 + r < P.M ? to_float(x[(m0 + r) * P.xs + k0 + lk]) : 0.0f;
#pragma unroll
      for (int g = 0; g < (kGated ? 2 : 1); ++g)
        sw[g][lk][r] = kin && n0 + r < P.N ? to_float(w[g][(n0 + r) * ws[g] + k0 + lk]) : 0.0f;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kStep; ++k) {
      const float4 a = *reinterpret_cast<const float4 *>(&sx[k][4 * ty]);
      const float av[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
      for (int g = 0; g < (kGated ? 2 : 1); ++g) {
        const float4 b = *reinterpret_cast<const float4 *>(&sw[g][k][4 * tx]);
        const float bv[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[g][i][j] = fmaf(av[i], bv[j], acc[g][i][j]);
      }
    }
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t m = m0 + 4 * ty + i;
    if (m >= P.M) break;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t n = n0 + 4 * tx + j;
      if (n >= P.N) break;
      float y = acc[0][i][j];
      if (P.bias) y += load_any(P.bias, n, P.dtype);
      y = activate(y, P.act);
      if constexpr (kGated) {
        float u = acc[1][i][j];
        if (P.bias_u) u += load_any(P.bias_u, n, P.dtype);
        y *= u;
      }
      if (P.res) y += load_any(P.res, m * P.rs + n, P.out_dtype);
      store_any(P.out, m * P.os + n, y, P.out_dtype);
    }
  }
}

template <class T>
cudaError_t launch_general(const LinearParams &P, cudaStream_t stream) {
  const dim3 grid(static_cast<unsigned>((P.N + kTile - 1) / kTile),
                  static_cast<unsigned>((P.M + kTile - 1) / kTile));
  return P.wu ? launch_chained(linear_general_kernel<T, true>, grid, dim3(kGenThreads), 0,
                               stream, P)
              : launch_chained(linear_general_kernel<T, false>, grid, dim3(kGenThreads), 0,
                               stream, P);
}

}  // namespace

int launch_linear(const spec_target &h, const LinearParams &P, cudaStream_t stream) {
  cudaError_t e;
  if (P.dtype != SV_FP32 && lin_rows_aligned(P.x, P.xs, P.M) && lin_rows_aligned(P.w, P.ws, P.N) &&
      (!P.wu || lin_rows_aligned(P.wu, P.wus, P.N)))
    return P.M <= 128 ? launch_linear_few(h, P, stream) : launch_linear_pair(h, P, stream);
  if ((P.M + kTile - 1) / kTile > 65535) return SV_ERR_SHAPE;
  switch (P.dtype) {
    case SV_BF16: e = launch_general<__nv_bfloat16>(P, stream); break;
    case SV_FP16: e = launch_general<__half>(P, stream); break;
    default: e = launch_general<float>(P, stream);
  }
  return e == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}

}  // namespace sv
