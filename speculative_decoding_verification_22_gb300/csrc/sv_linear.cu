// sv_linear.cu -- products with an epilogue, general form:
//
//   out = act(x w^T + bias) + residual
//   out = act(x wg^T + bg) * (x wu^T + bu)
//
// fp32 arithmetic on operands of any type, stride and alignment, for what the
// tensor-core forms do not take.  A block of 256 threads holds a tile of the output,
// 16 x 16 threads with every sixteenth row and column each, and walks K in steps of 32
// through shared memory, the next step's elements on their way in registers.  Where
// the tiles leave SMs idle a cluster shares one: each CTA takes a part of K, and the
// parts are added in the order of K through distributed shared memory.  Up to eight
// rows of x a warp takes a row of the weight and its lanes run along K.
//
// What bounds it: many rows the K step, two barriers and one step ahead, with loads of one
// element a lane (1024 x 4096 x 4096 in fp32 1.08 ms, 32 TFLOP/s; 512 x 4096 x 4095 in bf16
// 0.67 ms); few rows the same loads (5 x 4096 x 4096 in fp32 45 us, the weight's bytes 10).
#include <algorithm>

#include "sv_linear_tc.cuh"

namespace sv {
namespace {

constexpr int kThreads = 256;
constexpr int kStep = 32;  // K elements of a step
constexpr int kMaxSplit = 8;

// y and, gated, u of element [m, n] to the output.
template <bool kGated>
__device__ __forceinline__ void finish(const LinearParams &P, int64_t m, int64_t n, float y,
                                       float u) {
  if (P.bias) y += load_any(P.bias, n, P.dtype);
  y = activate(y, P.act);
  if constexpr (kGated) {
    if (P.bias_u) u += load_any(P.bias_u, n, P.dtype);
    y *= u;
  }
  if (P.res) y += load_any(P.res, m * P.rs + n, P.out_dtype);
  store_any(P.out, m * P.os + n, y, P.out_dtype);
}

// kTM x kTN elements a thread: a tile of 16 kTM rows of x and 16 kTN of each weight.
template <class T, bool kGated, int kTM, int kTN>
__global__ void __launch_bounds__(kThreads, 2) linear_general_kernel(const LinearParams P, int split) {
  constexpr int kW = kGated ? 2 : 1, kM = 16 * kTM, kN = 16 * kTN;
  constexpr int kLoadM = kM / 8, kLoadN = kN / 8;  // loads of a thread a step
  // (an odd stride: the lanes of a load are K elements, and their stores meet no bank
  // twice)
  __shared__ float sx[kStep][kM + 1], sw[kW][kStep][kN + 1];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int rank = split > 1 ? static_cast<int>(lin_cluster_rank()) : 0;
  const int64_t n0 = static_cast<int64_t>(blockIdx.x) / split * kN;
  const int64_t m0 = static_cast<int64_t>(blockIdx.y) * kM;
  const int64_t steps = (P.K + kStep - 1) / kStep;
  const int64_t s0 = steps * rank / split, s1 = steps * (rank + 1) / split;
  const T *x = static_cast<const T *>(P.x);
  const T *w[2] = {static_cast<const T *>(P.w), static_cast<const T *>(P.wu)};
  const int64_t ws[2] = {P.ws, P.wus};
  pdl_wait();
  pdl_launch_dependents();
  float px[kLoadM], pw[kW][kLoadN];
  auto load = [&](int64_t step) {
    const int64_t k = step * kStep + lane;
    const bool in = k < P.K && step < s1;
#pragma unroll
    for (int i = 0; i < kLoadM; ++i) {
      const int64_t m = m0 + warp + 8 * i;
      px[i] = in && m < P.M ? to_float(x[m * P.xs + k]) : 0.0f;
    }
#pragma unroll
    for (int g = 0; g < kW; ++g)
#pragma unroll
      for (int i = 0; i < kLoadN; ++i) {
        const int64_t n = n0 + warp + 8 * i;
        pw[g][i] = in && n < P.N ? to_float(w[g][n * ws[g] + k]) : 0.0f;
      }
  };
  float acc[kW][kTM][kTN] = {};
  load(s0);
  for (int64_t step = s0; step < s1; ++step) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kLoadM; ++i) sx[lane][warp + 8 * i] = px[i];
#pragma unroll
    for (int g = 0; g < kW; ++g)
#pragma unroll
      for (int i = 0; i < kLoadN; ++i) sw[g][lane][warp + 8 * i] = pw[g][i];
    __syncthreads();
    load(step + 1);
#pragma unroll 8
    for (int k = 0; k < kStep; ++k) {
      float a[kTM];
#pragma unroll
      for (int i = 0; i < kTM; ++i) a[i] = sx[k][ty + 16 * i];
#pragma unroll
      for (int g = 0; g < kW; ++g)
#pragma unroll
        for (int j = 0; j < kTN; ++j) {
          const float b = sw[g][k][tx + 16 * j];
#pragma unroll
          for (int i = 0; i < kTM; ++i) acc[g][i][j] = fmaf(a[i], b, acc[g][i][j]);
        }
    }
  }
  if (split == 1) {
#pragma unroll
    for (int i = 0; i < kTM; ++i)
#pragma unroll
      for (int j = 0; j < kTN; ++j) {
        const int64_t m = m0 + ty + 16 * i, n = n0 + tx + 16 * j;
        if (m < P.M && n < P.N) finish<kGated>(P, m, n, acc[0][i][j], acc[kW - 1][i][j]);
      }
    return;
  }
  // CTA r of the cluster finishes every split-th of a thread's elements from r on: its
  // peers leave theirs in their own shared memory.
  constexpr int kEach = kTM * kTN;
  __shared__ float parts[kEach <= 16 ? kW * kEach * kThreads : 1];
  if constexpr (kEach <= 16) {
#pragma unroll
    for (int g = 0; g < kW; ++g)
#pragma unroll
      for (int e = 0; e < kEach; ++e)
        parts[(g * kEach + e) * kThreads + threadIdx.x] = acc[g][e / kTN][e % kTN];
    lin_cluster_sync();
    const uint32_t own = smem_u32(parts) + threadIdx.x * 4;
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
      if (e % split != rank) continue;
      float y[kW] = {};
      for (int q = 0; q < split; ++q)
#pragma unroll
        for (int g = 0; g < kW; ++g) {
          float v;
          asm volatile("ld.shared::cluster.f32 %0, [%1];"
                       : "=f"(v)
                       : "r"(lin_remote(own + (g * kEach + e) * kThreads * 4, q))
                       : "memory");
          y[g] += v;
        }
      const int64_t m = m0 + ty + 16 * (e / kTN), n = n0 + tx + 16 * (e % kTN);
      if (m < P.M && n < P.N) finish<kGated>(P, m, n, y[0], y[kW - 1]);
    }
    lin_cluster_sync();  // nobody reads a CTA that is gone
  }
}

// Up to kFewRows rows of x: a row of the weight (of each) a warp.
constexpr int kFewRows = 8;

template <class T, bool kGated>
__global__ void __launch_bounds__(kThreads) linear_general_few_kernel(const LinearParams P) {
  constexpr int kW = kGated ? 2 : 1, kAhead = 4;
  const int lane = threadIdx.x & 31;
  const int64_t n = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
  const T *x = static_cast<const T *>(P.x);
  const int rows = static_cast<int>(P.M);
  pdl_wait();
  pdl_launch_dependents();
  if (n >= P.N) return;
  const T *w[2] = {static_cast<const T *>(P.w) + n * P.ws,
                   kGated ? static_cast<const T *>(P.wu) + n * P.wus : nullptr};
  float acc[kW][kFewRows] = {};
  for (int64_t k0 = lane; k0 < P.K; k0 += 32 * kAhead) {
    float wv[kW][kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
#pragma unroll
      for (int g = 0; g < kW; ++g)
        wv[g][i] = k0 + 32 * i < P.K ? to_float(w[g][k0 + 32 * i]) : 0.0f;
#pragma unroll
    for (int m = 0; m < kFewRows; ++m) {
      if (m >= rows) break;
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const float xv = k0 + 32 * i < P.K ? to_float(x[m * P.xs + k0 + 32 * i]) : 0.0f;
#pragma unroll
        for (int g = 0; g < kW; ++g) acc[g][m] = fmaf(xv, wv[g][i], acc[g][m]);
      }
    }
  }
#pragma unroll
  for (int m = 0; m < kFewRows; ++m) {
    if (m >= rows) break;
    const float y = warp_sum(acc[0][m]), u = warp_sum(acc[kW - 1][m]);
    if (lane == 0) finish<kGated>(P, m, n, y, u);
  }
}

template <class T, bool kGated, int kTM, int kTN>
int launch_tile(const spec_target &h, const LinearParams &P, cudaStream_t stream) {
  const int64_t rows = (P.M + 16 * kTM - 1) / (16 * kTM), cols = (P.N + 16 * kTN - 1) / (16 * kTN);
  int split = 1;
  if (kTM * kTN <= 16)
    while (2 * split <= kMaxSplit && rows * cols * split < 4 * h.num_sms &&
           P.K >= 4 * kStep * split)
      split *= 2;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = split;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(cols * split), static_cast<unsigned>(rows));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = split > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, linear_general_kernel<T, kGated, kTM, kTN>, P, split) ==
                 cudaSuccess
             ? SV_OK
             : SV_ERR_CUDA;
}

template <class T, bool kGated>
int launch_general(const spec_target &h, const LinearParams &P, cudaStream_t stream) {
  // (4096 x 4096 in fp32, the weight from HBM and x in L2: 1 row 20.5 us, 5 45, 8 63, as a
  // tile 71 whatever the rows)
  if (P.M <= kFewRows) {
    const int64_t blocks = (P.N + kThreads / 32 - 1) / (kThreads / 32);
    return launch_chained(linear_general_few_kernel<T, kGated>, dim3(static_cast<unsigned>(blocks)),
                          dim3(kThreads), 0, stream, P) == cudaSuccess
               ? SV_OK
               : SV_ERR_CUDA;
  }
  // Large tiles where they are enough for every SM, else smaller ones whose K is shared
  // (32 x 4096 x 4096 in fp32: 74 us; 256 rows 312, 422 with the smallest tile).
  const int64_t large = ((P.M + 127) / 128) * ((P.N + (kGated ? 63 : 127)) / (kGated ? 64 : 128));
  if (large >= h.num_sms) return launch_tile<T, kGated, 8, kGated ? 4 : 8>(h, P, stream);
  return P.M <= 32 ? launch_tile<T, kGated, 2, 4>(h, P, stream)
                   : launch_tile<T, kGated, 4, kGated ? 2 : 4>(h, P, stream);
}
template <class T>
int launch_typed(const spec_target &h, LinearParams P, cudaStream_t stream) {
  // Row tiles lie on a grid's y, which ends at 65535 of them: rows beyond are further
  // launches. (All tiles on x, with a division by their columns, cost the 16-bit rows of
  // 512 x 4096 x 4095 743 us in place of 668, through the registers.)
  constexpr int64_t kMost = int64_t(65535) * 128;
  const int64_t M = P.M, size = P.out_dtype == SV_FP32 ? 4 : 2;
  for (int64_t m0 = 0; m0 < M; m0 += kMost) {
    P.M = std::min(M - m0, kMost);
    const int code =
        P.wu ? launch_general<T, true>(h, P, stream) : launch_general<T, false>(h, P, stream);
    if (code != SV_OK) return code;
    P.x = static_cast<const T *>(P.x) + kMost * P.xs;
    P.out = static_cast<char *>(P.out) + kMost * P.os * size;
    if (P.res) P.res = static_cast<const char *>(P.res) + kMost * P.rs * size;
  }
  return SV_OK;
}

}  // namespace

int launch_linear(const spec_target &h, const LinearParams &P, cudaStream_t stream) {
  if (P.dtype != SV_FP32 && lin_rows_aligned(P.x, P.xs, P.M) && lin_rows_aligned(P.w, P.ws, P.N) &&
      (!P.wu || lin_rows_aligned(P.wu, P.wus, P.N)))
    return P.M <= 128 ? launch_linear_few(h, P, stream) : launch_linear_pair(h, P, stream);
  switch (P.dtype) {
    case SV_BF16: return launch_typed<__nv_bfloat16>(h, P, stream);
    case SV_FP16: return launch_typed<__half>(h, P, stream);
    default: return launch_typed<float>(h, P, stream);
  }
}

}  // namespace sv
