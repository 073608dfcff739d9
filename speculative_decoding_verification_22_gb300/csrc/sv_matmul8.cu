// sv_matmul8.cu -- 8-bit product with one fp32 scale per row and 128 columns
// of A and per 128 x 128 block of W.
#include "sv_target.cuh"

namespace sv {
namespace {

constexpr int kTile = 64, kStep = 32, kThreadsMM = 256;

__device__ __forceinline__ float e4m3(uint8_t b) {
  return __half2float(__half(__nv_cvt_fp8_to_halfraw(b, __NV_E4M3)));
}

// 64 x 64 outputs a block, 4 x 4 a thread.
template <class T>
__global__ void __launch_bounds__(kThreadsMM) matmul8_simple_kernel(const MatmulParams P) {
  __shared__ float sa[kStep][kTile + 4], sw[kStep][kTile + 4];
  const int m0 = blockIdx.y * kTile, n0 = blockIdx.x * kTile;
  const int tm = threadIdx.x / 16 * 4, tn = threadIdx.x % 16 * 4;
  float acc[4][4] = {}, blk[4][4] = {};
  pdl_wait();
  pdl_launch_dependents();
  for (int k0 = 0; k0 < P.K; k0 += kStep) {
    for (int i = threadIdx.x; i < kTile * kStep; i += kThreadsMM) {
      const int r = i / kStep, k = k0 + i % kStep;
      sa[i % kStep][r] = (m0 + r < P.M && k < P.K) ? e4m3(P.a[int64_t(m0 + r) * P.K + k]) : 0.0f;
      sw[i % kStep][r] = (n0 + r < P.N && k < P.K) ? e4m3(P.w[int64_t(n0 + r) * P.K + k]) : 0.0f;
    }
    __syncthreads();
    for (int k = 0; k < kStep; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) blk[i][j] = fmaf(sa[k][tm + i], sw[k][tn + j], blk[i][j]);
    __syncthreads();
    if ((k0 + kStep) % SV_SCALE_BLOCK == 0 || k0 + kStep >= P.K) {
      const int kb = k0 / SV_SCALE_BLOCK;
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int m = m0 + tm + i, n = n0 + tn + j;
          if (m < P.M && n < P.N)
            acc[i][j] = fmaf(blk[i][j], P.as[int64_t(m) * P.kb + kb] *
                                            P.ws[int64_t(n / SV_SCALE_BLOCK) * P.kb + kb],
                             acc[i][j]);
          blk[i][j] = 0.0f;
        }
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int m = m0 + tm + i, n = n0 + tn + j;
      if (m < P.M && n < P.N) static_cast<T *>(P.out)[m * P.os + n] = from_float<T>(acc[i][j]);
    }
}

}  // namespace

int launch_matmul_fp8(const spec_target &h, const MatmulParams &P, cudaStream_t stream) {
  const dim3 grid((P.N + kTile - 1) / kTile, (P.M + kTile - 1) / kTile), block(kThreadsMM);
  cudaError_t e;
  switch (P.out_dtype) {
    case SV_BF16:
      e = launch_chained(matmul8_simple_kernel<__nv_bfloat16>, grid, block, 0, stream, P);
      break;
    case SV_FP16:
      e = launch_chained(matmul8_simple_kernel<__half>, grid, block, 0, stream, P);
      break;
    default: e = launch_chained(matmul8_simple_kernel<float>, grid, block, 0, stream, P);
  }
  return e == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}

}  // namespace sv
