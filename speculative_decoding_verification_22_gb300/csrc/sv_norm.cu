// sv_norm.cu -- residual RMS norm, with the result in the rows' type or in
// E4M3 with one scale per 128 columns or per row.
//
//   h = x + residual,  y = h / sqrt(mean(h^2) + eps) * weight
//
// One pass: a row stays in registers between the sum of squares and the
// output, so x and the residual are read once and the results written once
// (the bytes the operator cannot do without); HBM bounds it for many rows,
// the launch for few (times in this file are of kernels in a CUDA graph; a call adds
// 2 us).  A thread holds kVec vectors of eight elements; a row
// takes `wpr` whole warps, and a block several short rows.  Sixteen lanes
// hold the 128 columns of one scale, so the block maximum is four shuffles.
#include "sv_target.cuh"

namespace sv {
namespace {

__device__ __forceinline__ float warp_max_nan(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x = max_nan(x, __shfl_xor_sync(0xffffffffu, x, o));
  return x;
}

// scale = max(amax, 1e-30) / 448
__device__ __forceinline__ float e4m3_scale(float amax) { return max_nan(amax, 1e-30f) / 448.0f; }

// y * (1 / scale) in place of y / scale: one more rounding in fp32, 2^-24
// against E4M3's 2^-4, for a tenth of the instructions.
__device__ __forceinline__ uint8_t to_e4m3(float y, float inv) {
  return static_cast<uint8_t>(__nv_cvt_float_to_fp8(y * inv, __NV_SATFINITE, __NV_E4M3));
}
__device__ __forceinline__ uint2 to_e4m3x8(const float (&y)[8], float inv) {
  uint32_t h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    h[i] = __nv_cvt_float2_to_fp8x2(make_float2(y[2 * i] * inv, y[2 * i + 1] * inv),
                                    __NV_SATFINITE, __NV_E4M3);
  return make_uint2(h[0] | h[1] << 16, h[2] | h[3] << 16);
}

// `red` holds one value for each of a row's wpr warps; all threads of the
// block take part.
template <class Op>
__device__ __forceinline__ float row_reduce(float v, float *red, int wpr, int warp, int lane,
                                            Op op) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = op(v, __shfl_xor_sync(0xffffffffu, v, o));
  if (wpr == 1) return v;
  if (lane == 0) red[warp] = v;
  __syncthreads();
  const int first = warp / wpr * wpr;
  float r = red[first];
  for (int i = 1; i < wpr; ++i) r = op(r, red[first + i]);
  return r;
}

template <class T, int kVec, int kQuant, int kThreads>
__global__ void __launch_bounds__(kThreads, kThreads <= 256 && kVec == 2 ? 5 : 1)
    norm_kernel(const NormParams P, int wpr) {
  __shared__ float red[2][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * ((blockDim.x >> 5) / wpr) + warp / wpr;
  const bool live = row < P.rows;
  const int t = (warp % wpr) * 32 + lane, step = wpr * 32;
  const int nvec = P.d >> 3;
  const T *w = static_cast<const T *>(P.w);
  pdl_wait();
  pdl_launch_dependents();
  // The weight is read ahead where that costs no resident blocks (5 rows of
  // 4096: 1.9 us against 2.1; with it the many-row form takes 102 us, not 94).
  constexpr bool kAhead = kVec == 1 || (kVec == 2 && kThreads > 256);
  Vec8<T> wv[kVec];
  float h[kVec][8];
  float ss = 0.0f;
  {
    const T *x = static_cast<const T *>(P.x) + row * P.xs;
    const T *r = static_cast<const T *>(P.res) + row * P.rs;
    Vec8<T> xv[kVec], rv[kVec];
#pragma unroll
    for (int v = 0; v < kVec; ++v) {
      const int i = t + v * step;
      if (live && i < nvec) {
        xv[v] = load8(x + 8 * i);
        if (P.res) rv[v] = load8(r + 8 * i);
        if constexpr (kAhead) wv[v] = load8(w + 8 * i);
      }
    }
#pragma unroll
    for (int v = 0; v < kVec; ++v) {
      const bool in = live && t + v * step < nvec;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        float s = in ? to_float(xv[v].e[e]) : 0.0f;
        if (P.res && in) s += to_float(rv[v].e[e]);
        h[v][e] = s;
        ss = fmaf(s, s, ss);
      }
      if (P.res_out && in) {
        Vec8<T> o;
#pragma unroll
        for (int e = 0; e < 8; ++e) o.e[e] = from_float<T>(h[v][e]);
        store8(static_cast<T *>(P.res_out) + row * P.ros + 8 * (t + v * step), o);
      }
    }
  }
  ss = row_reduce(ss, red[0], wpr, warp, lane, [](float a, float b) { return a + b; });
  const float inv = 1.0f / sqrtf(ss / static_cast<float>(P.d) + P.eps);

  float rmax = 0.0f;
#pragma unroll
  for (int v = 0; v < kVec; ++v) {
    const int i = t + v * step;
    const bool in = live && i < nvec;
    if (in) {
      if constexpr (!kAhead) wv[v] = load8(w + 8 * i);
#pragma unroll
      for (int e = 0; e < 8; ++e) h[v][e] = h[v][e] * inv * to_float(wv[v].e[e]);
    }
    if constexpr (kQuant == 0) {
      if (in) {
        Vec8<T> o;
#pragma unroll
        for (int e = 0; e < 8; ++e) o.e[e] = from_float<T>(h[v][e]);
        store8(static_cast<T *>(P.out) + row * P.os + 8 * i, o);
      }
    } else {
      // lanes past the row hold zeros
      float m = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) m = max_nan(m, fabsf(h[v][e]));
      if constexpr (kQuant == 1) {
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
        const float s = e4m3_scale(m);
        if (in) {
          *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(P.out) + row * P.os + 8 * i) =
              to_e4m3x8(h[v], 1.0f / s);
          if ((i & 15) == 0) P.scale[row * ((P.d + 127) / 128) + (i >> 4)] = s;
        }
      } else {
        rmax = max_nan(rmax, m);
      }
    }
  }
  if constexpr (kQuant == 2) {
    rmax = row_reduce(rmax, red[1], wpr, warp, lane,
                      [](float a, float b) { return max_nan(a, b); });
    const float s = e4m3_scale(rmax), inv_s = 1.0f / s;
#pragma unroll
    for (int v = 0; v < kVec; ++v) {
      const int i = t + v * step;
      if (live && i < nvec)
        *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(P.out) + row * P.os + 8 * i) =
            to_e4m3x8(h[v], inv_s);
    }
    if (live && t == 0) P.scale[row] = s;
  }
}

// What is left, rows of more columns: one block a row, the row read once for
// each of sum, maximum (row scale) and output (the later reads come from
// cache).  A thread rereads only elements that it writes itself, so the
// in-place forms hold here too.
constexpr int kAnyThreads = 512;
template <class T>
__global__ void __launch_bounds__(kAnyThreads) norm_any_kernel(const NormParams P) {
  __shared__ float red[2][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t row = blockIdx.x;
  const T *x = static_cast<const T *>(P.x) + row * P.xs;
  const T *r = P.res ? static_cast<const T *>(P.res) + row * P.rs : nullptr;
  const T *w = static_cast<const T *>(P.w);
  T *ro = P.res_out ? static_cast<T *>(P.res_out) + row * P.ros : nullptr;
  pdl_wait();
  pdl_launch_dependents();
  auto at = [&](int i) { return r ? to_float(x[i]) + to_float(r[i]) : to_float(x[i]); };
  // a warp takes 128 columns at a time, lane l the columns l, l + 32, ...
  auto each = [&](auto &&f) {
    for (int g = warp * 128; g < P.d; g += kAnyThreads * 4) f(g);
  };
  float ss = 0.0f;
  each([&](int g) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int i = g + 32 * k + lane;
      if (i < P.d) {
        const float h = at(i);
        ss = fmaf(h, h, ss);
      }
    }
  });
  ss = row_reduce(ss, red[0], kAnyThreads / 32, warp, lane,
                  [](float a, float b) { return a + b; });
  const float inv = 1.0f / sqrtf(ss / static_cast<float>(P.d) + P.eps);
  float s = 0.0f;
  if (P.quant == 2) {
    float m = 0.0f;
    each([&](int g) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int i = g + 32 * k + lane;
        if (i < P.d) m = max_nan(m, fabsf(at(i) * inv * to_float(w[i])));
      }
    });
    s = e4m3_scale(row_reduce(m, red[1], kAnyThreads / 32, warp, lane,
                              [](float a, float b) { return max_nan(a, b); }));
    if (threadIdx.x == 0) P.scale[row] = s;
  }
  float inv_s = 1.0f / s;
  each([&](int g) {
    float y[4], m = 0.0f;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int i = g + 32 * k + lane;
      y[k] = 0.0f;
      if (i < P.d) {
        const float h = at(i);
        if (ro) ro[i] = from_float<T>(h);
        y[k] = h * inv * to_float(w[i]);
      }
      m = max_nan(m, fabsf(y[k]));
    }
    if (P.quant == 1) {
      s = e4m3_scale(warp_max_nan(m));
      inv_s = 1.0f / s;
      if (lane == 0) P.scale[row * ((P.d + 127) / 128) + g / 128] = s;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int i = g + 32 * k + lane;
      if (i >= P.d) break;
      if (P.quant)
        static_cast<uint8_t *>(P.out)[row * P.os + i] = to_e4m3(y[k], inv_s);
      else
        static_cast<T *>(P.out)[row * P.os + i] = from_float<T>(y[k]);
    }
  });
}

// Rows of any stride and alignment up to 8192 columns: one pass, as above, but
// an element at a time.  A warp takes kGroups runs of 128 columns, lane l of
// them the columns l, l + 32, ...
template <class T, int kGroups>
__global__ void __launch_bounds__(512) norm_odd_kernel(const NormParams P) {
  __shared__ float red[2][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  const int64_t row = blockIdx.x;
  const T *x = static_cast<const T *>(P.x) + row * P.xs;
  const T *r = P.res ? static_cast<const T *>(P.res) + row * P.rs : nullptr;
  const T *w = static_cast<const T *>(P.w);
  T *ro = P.res_out ? static_cast<T *>(P.res_out) + row * P.ros : nullptr;
  const int first = warp * (128 * kGroups) + lane;
  pdl_wait();
  pdl_launch_dependents();
  float h[4 * kGroups], ss = 0.0f;
#pragma unroll
  for (int k = 0; k < 4 * kGroups; ++k) {
    const int i = first + 32 * k;
    h[k] = i < P.d ? to_float(x[i]) : 0.0f;
  }
  if (r) {
#pragma unroll
    for (int k = 0; k < 4 * kGroups; ++k) {
      const int i = first + 32 * k;
      if (i < P.d) h[k] += to_float(r[i]);
    }
  }
#pragma unroll
  for (int k = 0; k < 4 * kGroups; ++k) ss = fmaf(h[k], h[k], ss);
  ss = row_reduce(ss, red[0], warps, warp, lane, [](float a, float b) { return a + b; });
  const float inv = 1.0f / sqrtf(ss / static_cast<float>(P.d) + P.eps);
  float m = 0.0f;
#pragma unroll
  for (int k = 0; k < 4 * kGroups; ++k) {
    const int i = first + 32 * k;
    if (i < P.d) {
      if (ro) ro[i] = from_float<T>(h[k]);
      h[k] = h[k] * inv * to_float(w[i]);
      m = max_nan(m, fabsf(h[k]));
    }
  }
  float s = 0.0f, inv_s = 0.0f;
  if (P.quant == 2) {
    s = e4m3_scale(row_reduce(m, red[1], warps, warp, lane,
                              [](float a, float b) { return max_nan(a, b); }));
    inv_s = 1.0f / s;
    if (threadIdx.x == 0) P.scale[row] = s;
  }
#pragma unroll
  for (int g = 0; g < kGroups; ++g) {
    const int block = warp * kGroups + g;
    if (block * 128 >= P.d) break;
    if (P.quant == 1) {
      float mb = 0.0f;
#pragma unroll
      for (int k = 4 * g; k < 4 * g + 4; ++k) mb = max_nan(mb, fabsf(h[k]));
      s = e4m3_scale(warp_max_nan(mb));
      inv_s = 1.0f / s;
      if (lane == 0) P.scale[row * ((P.d + 127) / 128) + block] = s;
    }
#pragma unroll
    for (int k = 4 * g; k < 4 * g + 4; ++k) {
      const int i = first + 32 * k;
      if (i >= P.d) break;
      if (P.quant)
        static_cast<uint8_t *>(P.out)[row * P.os + i] = to_e4m3(h[k], inv_s);
      else
        static_cast<T *>(P.out)[row * P.os + i] = from_float<T>(h[k]);
    }
  }
}
template <class T, int kGroups>
cudaError_t launch_odd(const NormParams &P, cudaStream_t stream) {
  const int warps = (P.d + 128 * kGroups - 1) / (128 * kGroups);
  return launch_chained(norm_odd_kernel<T, kGroups>, dim3(static_cast<unsigned>(P.rows)),
                        dim3(32 * warps), 0, stream, P);
}

template <class T, int kVec, int kThreads>
cudaError_t launch_block(const NormParams &P, int wpr, int per_block, cudaStream_t stream) {
  const dim3 grid(static_cast<unsigned>((P.rows + per_block - 1) / per_block));
  const dim3 block(32 * wpr * per_block);
  switch (P.quant) {
    case 0:
      return launch_chained(norm_kernel<T, kVec, 0, kThreads>, grid, block, 0, stream, P, wpr);
    case 1:
      return launch_chained(norm_kernel<T, kVec, 1, kThreads>, grid, block, 0, stream, P, wpr);
    default:
      return launch_chained(norm_kernel<T, kVec, 2, kThreads>, grid, block, 0, stream, P, wpr);
  }
}
template <class T, int kVec>
cudaError_t launch_vec(const NormParams &P, cudaStream_t stream) {
  const int wpr = (P.d / 8 + 32 * kVec - 1) / (32 * kVec);
  const int per_block = wpr >= 4 ? 1 : 4 / wpr;
  return wpr * per_block <= 8 ? launch_block<T, kVec, 256>(P, wpr, per_block, stream)
                              : launch_block<T, kVec, 1024>(P, wpr, per_block, stream);
}

template <class T>
cudaError_t launch_typed(const NormParams &P, int num_sms, cudaStream_t stream) {
  auto ok = [](const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; };
  const int es = sizeof(T);
  const bool vec = P.d % 8 == 0 && P.d <= 32768 && P.xs * es % 16 == 0 && ok(P.x) && ok(P.w) &&
                   (!P.res || (P.rs * es % 16 == 0 && ok(P.res))) &&
                   (!P.res_out || (P.ros * es % 16 == 0 && ok(P.res_out))) &&
                   (P.quant ? (reinterpret_cast<uintptr_t>(P.out) & 7u) == 0
                            : P.os * es % 16 == 0 && ok(P.out));
  // One pass against the reads again: 16384 rows of 4095 in bf16 140 us against
  // 196 (to E4M3 164 against 234), 100000 of 500 103 against 583.  Four runs a
  // warp take 193 us for the former, and the wider rows that they are for 11.1
  // against 12.5 (384 of 8190); above that (4000 rows of 16383: 266 us against
  // 201) too few rows fit an SM at once.
  if (!vec && P.d <= 4096) return launch_odd<T, 2>(P, stream);
  if (!vec && P.d <= 8192) return launch_odd<T, 4>(P, stream);
  if (!vec)
    return launch_chained(norm_any_kernel<T>, dim3(static_cast<unsigned>(P.rows)),
                          dim3(kAnyThreads), 0, stream, P);
  const int nvec = P.d / 8;
  // Few rows: one vector a thread, as many threads as that takes (5 rows of
  // 4096: 1.9 us; 2.4 with two).  Many: two a thread, which leaves room for five
  // blocks of eight warps on an SM (16384 rows of 4096 in bf16 to E4M3: 94 us,
  // 5.0 TB/s; 113 with one vector, 117 with four).
  const int kvec = nvec > 2048 ? 4 : (P.rows <= num_sms && nvec <= 1024) || nvec <= 128 ? 1 : 2;
  switch (kvec) {
    case 1: return launch_vec<T, 1>(P, stream);
    case 2: return launch_vec<T, 2>(P, stream);
    default: return launch_vec<T, 4>(P, stream);
  }
}

}  // namespace

cudaError_t launch_norm(const NormParams &P, int num_sms, cudaStream_t stream) {
  switch (P.dtype) {
    case SV_BF16: return launch_typed<__nv_bfloat16>(P, num_sms, stream);
    case SV_FP16: return launch_typed<__half>(P, num_sms, stream);
    default: return launch_typed<float>(P, num_sms, stream);
  }
}

}  // namespace sv
