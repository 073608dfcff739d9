// sv_block_norm.cu -- the norms after and before a block with its gate, its
// scale and the residual:
//
//   y = x / sqrt(mean(x^2) + eps) * post,  h = residual + s * gate * y,
//   out = h / sqrt(mean(h^2) + eps) * weight
//
// One pass: a row stays in registers from its load to the stores, through two
// sums (and the maximum of an E4M3 row), so every input is read once and every
// output written once; HBM bounds it for many rows (16384 x 4096 in bf16 to bf16 89 us,
// 6.0 TB/s; to E4M3 with a gate 93, where instructions count too: 71% of the SM's
// issue), the launch for few (5 x 4096: 2.8 us).  Times in this file are of kernels in
// a CUDA graph.  A thread
// holds kVec vectors of eight elements; a row takes `wpr` whole warps, and a block
// several short rows.  Sixteen lanes hold the 128 columns of one scale, so a
// block's maximum is four shuffles.
#include "sv_target.cuh"
#include "sv_tmem.cuh"

namespace sv {
namespace {

// `red` holds one value for each of a row's wpr warps; all threads of the block
// take part.
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
// scale = max(amax, 1e-30) / 448
__device__ __forceinline__ float e4m3_scale(float amax) { return max_nan(amax, 1e-30f) / 448.0f; }

// Two neighbouring elements as fp32 pairs and back: the arithmetic below takes two
// columns an instruction.
template <class T>
__device__ __forceinline__ uint64_t widen(const Vec8<T> &v, int i) {
  return pair2(to_float(v.e[2 * i]), to_float(v.e[2 * i + 1]));
}
template <>
__device__ __forceinline__ uint64_t widen(const Vec8<__nv_bfloat16> &v, int i) {
  const uint32_t w = reinterpret_cast<const uint32_t *>(&v)[i];
  return pair2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
__device__ __forceinline__ void narrow(Vec8<float> &o, int i, uint64_t x) {
  const float2 f = unpair2(x);
  o.e[2 * i] = f.x;
  o.e[2 * i + 1] = f.y;
}
__device__ __forceinline__ void narrow(Vec8<__half> &o, int i, uint64_t x) {
  const float2 f = unpair2(x);
  reinterpret_cast<__half2 *>(&o)[i] = __floats2half2_rn(f.x, f.y);
}
__device__ __forceinline__ void narrow(Vec8<__nv_bfloat16> &o, int i, uint64_t x) {
  const float2 f = unpair2(x);
  reinterpret_cast<__nv_bfloat162 *>(&o)[i] = __floats2bfloat162_rn(f.x, f.y);
}
// y * (1 / scale) in place of y / scale: one more rounding in fp32, 2^-24 against
// E4M3's 2^-4.
__device__ __forceinline__ uint2 to_e4m3x8(const uint64_t (&y)[4], float inv) {
  const uint64_t inv2 = pair2(inv, inv);
  uint32_t h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    h[i] = __nv_cvt_float2_to_fp8x2(unpair2(mul2(y[i], inv2)), __NV_SATFINITE, __NV_E4M3);
  return make_uint2(h[0] | h[1] << 16, h[2] | h[3] << 16);
}
__device__ __forceinline__ float sum2(uint64_t x) {
  const float2 f = unpair2(x);
  return f.x + f.y;
}

template <class T, int kVec, int kQuant, int kMost>
__global__ void __launch_bounds__(kMost, kMost > 256 ? 1 : kVec >= 2 ? 4 : 1)
    block_norm_kernel(const sv_block_norm_t P, int wpr, float inv_d) {
  __shared__ float red[3][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * ((blockDim.x >> 5) / wpr) + warp / wpr;
  const bool live = row < P.rows;
  const int t0 = (warp % wpr) * 32 + lane, step = wpr * 32;
  const int d = static_cast<int>(P.d);
  const int nvec = live ? d >> 3 : 0;  // of this thread's row
  const T *post = static_cast<const T *>(P.post_weight), *w = static_cast<const T *>(P.weight);
  const T *gate = P.gate ? static_cast<const T *>(P.gate) + row * P.gate_row : nullptr;
  pdl_wait();
  pdl_launch_dependents();
  const auto add = [](float a, float b) { return a + b; };
  uint64_t h[kVec][4];
  Vec8<T> rv[kVec];
  {
    const T *x = static_cast<const T *>(P.x) + row * P.x_stride;
    const T *r = static_cast<const T *>(P.residual) + row * P.residual_stride;
    Vec8<T> xv[kVec];
#pragma unroll
    for (int v = 0; v < kVec; ++v) {
      const int i = t0 + v * step;
      if (i < nvec) {
        xv[v] = load8(x + 8 * i);
        rv[v] = load8(r + 8 * i);
      }
    }
    uint64_t ss = 0;
#pragma unroll
    for (int v = 0; v < kVec; ++v) {
      const bool in = t0 + v * step < nvec;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        h[v][e] = in ? widen(xv[v], e) : 0;
        ss = fma2(h[v][e], h[v][e], ss);
      }
    }
    if (post) {
      const float all = row_reduce(sum2(ss), red[0], wpr, warp, lane, add);
      const float inv = rsqrtf(fmaf(all, inv_d, P.eps));
      const uint64_t inv2 = pair2(inv, inv);
#pragma unroll
      for (int v = 0; v < kVec; ++v) {
        const int i = t0 + v * step;
        if (i < nvec) {
          const Vec8<T> pv = load8(post + 8 * i);
#pragma unroll
          for (int e = 0; e < 4; ++e) h[v][e] = mul2(mul2(h[v][e], inv2), widen(pv, e));
        }
      }
    }
  }
  float scale = P.branch_scale;
  if (gate && P.gate_col == 0) {
    if (live) scale *= to_float(gate[0]);
    gate = nullptr;
  }
  const uint64_t scale2 = pair2(scale, scale);
  uint64_t ss = 0;
#pragma unroll
  for (int v = 0; v < kVec; ++v) {
    const int i = t0 + v * step;
    if (i < nvec) {
      if (gate) {
        const Vec8<T> gv = load8(gate + 8 * i);
#pragma unroll
        for (int e = 0; e < 4; ++e) h[v][e] = mul2(h[v][e], widen(gv, e));
      }
      Vec8<T> o;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        h[v][e] = fma2(scale2, h[v][e], widen(rv[v], e));
        ss = fma2(h[v][e], h[v][e], ss);
        narrow(o, e, h[v][e]);
      }
      if (P.residual_out)
        store8(static_cast<T *>(P.residual_out) + row * P.residual_out_stride + 8 * i, o);
    }
  }
  const float all = row_reduce(sum2(ss), red[1], wpr, warp, lane, add);
  const float inv = rsqrtf(fmaf(all, inv_d, P.eps));
  const uint64_t inv2 = pair2(inv, inv);

  float rmax = 0.0f;
#pragma unroll
  for (int v = 0; v < kVec; ++v) {
    const int i = t0 + v * step;
    const bool in = i < nvec;
    if (in) {
      const Vec8<T> wv = load8(w + 8 * i);
#pragma unroll
      for (int e = 0; e < 4; ++e) h[v][e] = mul2(mul2(h[v][e], inv2), widen(wv, e));
    }
    if constexpr (kQuant == 0) {
      if (in) {
        Vec8<T> o;
#pragma unroll
        for (int e = 0; e < 4; ++e) narrow(o, e, h[v][e]);
        store8(static_cast<T *>(P.out) + row * P.out_stride + 8 * i, o);
      }
    } else {
      // lanes past the row hold zeros
      float m = 0.0f;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 f = unpair2(h[v][e]);
        m = max3_nan(m, fabsf(f.x), fabsf(f.y));
      }
      if constexpr (kQuant == 1) {
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
        const float s = e4m3_scale(m);
        if (in) {
          *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(P.out) + row * d + 8 * i) =
              to_e4m3x8(h[v], 1.0f / s);
          if ((i & 15) == 0) P.scale[row * ((d + 127) / 128) + (i >> 4)] = s;
        }
      } else {
        rmax = max_nan(rmax, m);
      }
    }
  }
  if constexpr (kQuant == 2) {
    rmax = row_reduce(rmax, red[2], wpr, warp, lane,
                      [](float a, float b) { return max_nan(a, b); });
    const float s = e4m3_scale(rmax), inv_s = 1.0f / s;
#pragma unroll
    for (int v = 0; v < kVec; ++v) {
      const int i = t0 + v * step;
      if (i < nvec)
        *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(P.out) + row * d + 8 * i) =
            to_e4m3x8(h[v], inv_s);
    }
    if (live && t0 == 0) P.scale[row] = s;
  }
}

// Rows of any stride and alignment up to 8192 columns: one pass, as above, but an
// element at a time.  A warp takes kGroups runs of 128 columns, lane l of them the
// columns l, l + 32, ...
template <class T, int kGroups>
__global__ void __launch_bounds__(512, 2) block_norm_odd_kernel(const sv_block_norm_t P,
                                                                float inv_d) {
  constexpr int kEach = 4 * kGroups;
  __shared__ float red[3][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  const int64_t row = blockIdx.x;
  const int d = static_cast<int>(P.d);
  const T *x = static_cast<const T *>(P.x) + row * P.x_stride;
  const T *r = static_cast<const T *>(P.residual) + row * P.residual_stride;
  const T *gate = P.gate ? static_cast<const T *>(P.gate) + row * P.gate_row : nullptr;
  const T *post = static_cast<const T *>(P.post_weight), *w = static_cast<const T *>(P.weight);
  T *ro = P.residual_out ? static_cast<T *>(P.residual_out) + row * P.residual_out_stride
                         : nullptr;
  const int first = warp * (128 * kGroups) + lane;
  pdl_wait();
  pdl_launch_dependents();
  const auto add = [](float a, float b) { return a + b; };
  float h[kEach], res[kEach], ss = 0.0f;
#pragma unroll
  for (int k = 0; k < kEach; ++k) {
    const int i = first + 32 * k;
    h[k] = i < d ? to_float(x[i]) : 0.0f;
    res[k] = i < d ? to_float(r[i]) : 0.0f;
  }
#pragma unroll
  for (int k = 0; k < kEach; ++k) ss = fmaf(h[k], h[k], ss);
  if (post) {
    ss = row_reduce(ss, red[0], warps, warp, lane, add);
    const float inv = rsqrtf(fmaf(ss, inv_d, P.eps));
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
      const int i = first + 32 * k;
      if (i < d) h[k] = h[k] * inv * to_float(post[i]);
    }
  }
  float scale = P.branch_scale;
  if (gate && P.gate_col == 0) {
    scale *= to_float(gate[0]);
    gate = nullptr;
  }
  ss = 0.0f;
#pragma unroll
  for (int k = 0; k < kEach; ++k) {
    const int i = first + 32 * k;
    if (i < d) {
      if (gate) h[k] *= to_float(gate[i]);
      h[k] = fmaf(scale, h[k], res[k]);
      ss = fmaf(h[k], h[k], ss);
      if (ro) ro[i] = from_float<T>(h[k]);
    }
  }
  ss = row_reduce(ss, red[1], warps, warp, lane, add);
  const float inv = rsqrtf(fmaf(ss, inv_d, P.eps));
  float m = 0.0f;
#pragma unroll
  for (int k = 0; k < kEach; ++k) {
    const int i = first + 32 * k;
    if (i < d) {
      h[k] = h[k] * inv * to_float(w[i]);
      m = max_nan(m, fabsf(h[k]));
    }
  }
  float s = 0.0f, inv_s = 0.0f;
  if (P.group == 0) {
    s = e4m3_scale(row_reduce(m, red[2], warps, warp, lane,
                              [](float a, float b) { return max_nan(a, b); }));
    inv_s = 1.0f / s;
    if (threadIdx.x == 0) P.scale[row] = s;
  }
#pragma unroll
  for (int g = 0; g < kGroups; ++g) {
    const int block = warp * kGroups + g;
    if (block * 128 >= d) break;
    if (P.group > 0) {
      float mb = 0.0f;
#pragma unroll
      for (int k = 4 * g; k < 4 * g + 4; ++k) mb = max_nan(mb, first + 32 * k < d ? fabsf(h[k]) : 0.0f);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) mb = max_nan(mb, __shfl_xor_sync(0xffffffffu, mb, o));
      s = e4m3_scale(mb);
      inv_s = 1.0f / s;
      if (lane == 0) P.scale[row * ((d + 127) / 128) + block] = s;
    }
#pragma unroll
    for (int k = 4 * g; k < 4 * g + 4; ++k) {
      const int i = first + 32 * k;
      if (i >= d) break;
      if (P.group >= 0)
        static_cast<uint8_t *>(P.out)[row * d + i] = static_cast<uint8_t>(
            __nv_cvt_float_to_fp8(h[k] * inv_s, __NV_SATFINITE, __NV_E4M3));
      else
        static_cast<T *>(P.out)[row * P.out_stride + i] = from_float<T>(h[k]);
    }
  }
}
template <class T, int kGroups>
cudaError_t launch_odd(const sv_block_norm_t &a, cudaStream_t stream) {
  const int warps = static_cast<int>((a.d + 128 * kGroups - 1) / (128 * kGroups));
  return launch_chained(block_norm_odd_kernel<T, kGroups>, dim3(static_cast<unsigned>(a.rows)),
                        dim3(32 * warps), 0, stream, a, 1.0f / static_cast<float>(a.d));
}

constexpr int kThreads = 512;  // of the form below

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

// What is left, rows of more columns: one block a row, the row read once for each of the sums, the maximum (row
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

template <class T, int kVec, int kMost>
cudaError_t launch_block(const sv_block_norm_t &a, int wpr, int per_block, cudaStream_t stream) {
  const dim3 grid(static_cast<unsigned>((a.rows + per_block - 1) / per_block));
  const dim3 block(32 * wpr * per_block);
  const float inv_d = 1.0f / static_cast<float>(a.d);
  if (a.group < 0)
    return launch_chained(block_norm_kernel<T, kVec, 0, kMost>, grid, block, 0, stream, a, wpr,
                          inv_d);
  if (a.group > 0)
    return launch_chained(block_norm_kernel<T, kVec, 1, kMost>, grid, block, 0, stream, a, wpr,
                          inv_d);
  return launch_chained(block_norm_kernel<T, kVec, 2, kMost>, grid, block, 0, stream, a, wpr,
                          inv_d);
}
template <class T, int kVec>
cudaError_t launch_vec(const sv_block_norm_t &a, cudaStream_t stream) {
  const int wpr = static_cast<int>((a.d / 8 + 32 * kVec - 1) / (32 * kVec));
  const int per_block = wpr >= 4 ? 1 : 4 / wpr;
  return wpr * per_block <= 8 ? launch_block<T, kVec, 256>(a, wpr, per_block, stream)
                              : launch_block<T, kVec, 1024>(a, wpr, per_block, stream);
}

template <class T>
cudaError_t launch_typed(const sv_block_norm_t &a, int num_sms, cudaStream_t stream) {
  auto ok = [&](const void *p, int64_t stride) {
    return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 &&
           (a.rows == 1 || stride * static_cast<int64_t>(sizeof(T)) % 16 == 0);
  };
  const bool vec = a.d % 8 == 0 && a.d <= 32768 && ok(a.x, a.x_stride) &&
                   ok(a.residual, a.residual_stride) && ok(a.weight, 0) && ok(a.post_weight, 0) &&
                   (a.gate_col == 0 || ok(a.gate, a.gate_row)) &&
                   (!a.residual_out || ok(a.residual_out, a.residual_out_stride)) &&
                   (a.group >= 0 ? (reinterpret_cast<uintptr_t>(a.out) & 7u) == 0
                                 : ok(a.out, a.out_stride));
  // One pass against the reads again: 16384 rows of 4095 in bf16 205 us against 295.
  if (!vec && a.d <= 4096) return launch_odd<T, 2>(a, stream);
  if (!vec && a.d <= 8192) return launch_odd<T, 4>(a, stream);
  if (!vec)
    return launch_chained(block_norm_any_kernel<T>, dim3(static_cast<unsigned>(a.rows)),
                          dim3(kThreads), 0, stream, a);
  const int64_t nvec = a.d / 8;
  // Few rows: one vector a thread, as many threads as that takes.  Many: four of 16-bit
  // rows (16384 rows of 4096 in bf16 to E4M3 with a gate: 93 us, 5.1 TB/s; 112 with
  // two; 4000 of 8192 to E4M3 49 against 65), two of fp32 rows (16384 of 4096 with a
  // full gate: 212 us; 241 with four) while 1024 threads hold one.
  if (a.rows <= num_sms && nvec <= 1024) return launch_vec<T, 1>(a, stream);
  if constexpr (sizeof(T) == 2) {
    return launch_vec<T, 4>(a, stream);
  } else {
    if (nvec <= 2048) return launch_vec<T, 2>(a, stream);
    return launch_block<T, 4, 1024>(a, static_cast<int>((nvec + 127) / 128), 1, stream);
  }
}

}  // namespace

cudaError_t launch_block_norm(const sv_block_norm_t &a, int num_sms, cudaStream_t stream) {
  switch (a.dtype) {
    case SV_BF16: return launch_typed<__nv_bfloat16>(a, num_sms, stream);
    case SV_FP16: return launch_typed<__half>(a, num_sms, stream);
    default: return launch_typed<float>(a, num_sms, stream);
  }
}

}  // namespace sv
