// sv_target_api.cu -- the C ABI declared in include/spec_target.h: handle
// lifetime, argument checks and launches.
#include <cmath>
#include <cstdint>
#include <new>

#include "sv_target.cuh"

namespace {

// Scratch of the attention's partial results.
constexpr size_t kScratchBytes = size_t(44) << 20;

size_t elem_size(int32_t dtype) { return dtype == SV_FP32 ? 4 : 2; }
bool float_type(int32_t dtype) {
  return dtype == SV_BF16 || dtype == SV_FP16 || dtype == SV_FP32;
}
bool aligned(const void *p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// The handle's device has to be the current one.
int check_handle(const spec_target *h) {
  if (!h) return SV_ERR_ARG;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return SV_ERR_CUDA;
  return dev == h->device ? SV_OK : SV_ERR_ARG;
}

int done(cudaError_t e) { return e == cudaSuccess ? SV_OK : SV_ERR_CUDA; }

int norm_checks(const void *x, int64_t xs, const void *res, int64_t rs, const void *w, float eps,
                int64_t rows, int64_t d, int32_t dtype, const void *out, int64_t os,
                const void *ro, int64_t ros) {
  if (!float_type(dtype) || !(eps >= 0.0f) || !std::isfinite(eps) || rows < 0) return SV_ERR_ARG;
  if (d < 1 || d > (1 << 20) || rows > INT32_MAX) return SV_ERR_SHAPE;
  if (rows == 0) return SV_OK;
  if (!x || !w || !out) return SV_ERR_ARG;
  if (rows > 1 && (xs < d || os < d || (res && rs < d) || (ro && ros < d))) return SV_ERR_SHAPE;
  const size_t es = elem_size(dtype);
  if (!aligned(x, es) || !aligned(w, es) || (res && !aligned(res, es)) || (ro && !aligned(ro, es)))
    return SV_ERR_ALIGN;
  return SV_OK;
}

}  // namespace

extern "C" {

int spec_target_create(spec_target_t **out) {
  if (!out) return SV_ERR_ARG;
  *out = nullptr;
  int dev = 0, major = 0, minor = 0, sms = 0, smem = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&smem, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev) != cudaSuccess)
    return SV_ERR_CUDA;
  if (major != 10 || minor != 3) return SV_ERR_ARCH;
  spec_target *h = new (std::nothrow) spec_target();
  if (!h) return SV_ERR_CUDA;
  h->device = dev;
  h->num_sms = sms;
  h->smem_optin = smem;
  h->scratch_bytes = kScratchBytes;
  if (cudaMalloc(&h->status, sizeof(int)) != cudaSuccess ||
      cudaMalloc(&h->scratch, h->scratch_bytes) != cudaSuccess ||
      cudaMemset(h->status, 0, sizeof(int)) != cudaSuccess ||
      cudaMemset(h->scratch, 0, h->scratch_bytes) != cudaSuccess ||
      cudaStreamSynchronize(nullptr) != cudaSuccess ||
      sv::plan_matmul_fp8(*h) != cudaSuccess) {
    spec_target_destroy(h);
    return SV_ERR_CUDA;
  }
  *out = h;
  return SV_OK;
}

void spec_target_destroy(spec_target_t *h) {
  if (!h) return;
  cudaFree(h->status);
  cudaFree(h->scratch);
  delete h;
}

int spec_target_status(spec_target_t *h, void *stream) {
  const int c = check_handle(h);
  if (c != SV_OK) return c;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  int code = 0;
  if (cudaMemcpyAsync(&code, h->status, sizeof(int), cudaMemcpyDeviceToHost, s) != cudaSuccess ||
      cudaMemsetAsync(h->status, 0, sizeof(int), s) != cudaSuccess ||
      cudaStreamSynchronize(s) != cudaSuccess)
    return SV_ERR_CUDA;
  return code;
}

int spec_target_set_wait_limit(spec_target_t *h, uint64_t limit_ns) {
  if (!h) return SV_ERR_ARG;
  h->wait_limit_ns = limit_ns;
  return SV_OK;
}

int spec_target_rms_norm(spec_target_t *h, const void *x, int64_t x_stride, const void *residual,
                         int64_t residual_stride, const void *weight, float eps, int64_t rows,
                         int64_t d, int32_t dtype, void *out, int64_t out_stride,
                         void *residual_out, int64_t residual_out_stride, void *stream) {
  if (!h) return SV_ERR_ARG;
  int c = norm_checks(x, x_stride, residual, residual_stride, weight, eps, rows, d, dtype, out,
                      out_stride, residual_out, residual_out_stride);
  if (c != SV_OK || rows == 0) return c;
  if (!aligned(out, elem_size(dtype))) return SV_ERR_ALIGN;
  if ((c = check_handle(h)) != SV_OK) return c;
  sv::NormParams P{x, residual, weight, out, residual_out, nullptr, x_stride, residual_stride,
                   out_stride, residual_out_stride, rows, static_cast<int>(d), dtype, 0, eps};
  return done(sv::launch_norm(P, h->num_sms, static_cast<cudaStream_t>(stream)));
}

int spec_target_rms_norm_fp8(spec_target_t *h, const void *x, int64_t x_stride,
                             const void *residual, int64_t residual_stride, const void *weight,
                             float eps, int64_t rows, int64_t d, int32_t dtype, int32_t group,
                             void *out8, float *scale, void *residual_out,
                             int64_t residual_out_stride, void *stream) {
  if (!h || (group != 0 && group != SV_SCALE_BLOCK)) return SV_ERR_ARG;
  int c = norm_checks(x, x_stride, residual, residual_stride, weight, eps, rows, d, dtype, out8,
                      d, residual_out, residual_out_stride);
  if (c != SV_OK || rows == 0) return c;
  if (!scale) return SV_ERR_ARG;
  if (!aligned(scale, 4)) return SV_ERR_ALIGN;
  if ((c = check_handle(h)) != SV_OK) return c;
  sv::NormParams P{x, residual, weight, out8, residual_out, scale, x_stride, residual_stride,
                   d, residual_out_stride, rows, static_cast<int>(d), dtype, group ? 1 : 2, eps};
  return done(sv::launch_norm(P, h->num_sms, static_cast<cudaStream_t>(stream)));
}

int spec_target_matmul_fp8(spec_target_t *h, const void *a8, const float *a_scale, const void *w8,
                           const float *w_scale, int64_t M, int64_t N, int64_t K,
                           int32_t out_dtype, void *out, int64_t out_stride, void *stream) {
  if (!h || !float_type(out_dtype)) return SV_ERR_ARG;
  constexpr int64_t kMost = int64_t(1) << 24;
  if (M < 0 || N < 1 || K < 1 || M > kMost || N > kMost || K > kMost || K % 16 != 0)
    return SV_ERR_SHAPE;
  if (M == 0) return SV_OK;
  if (!a8 || !a_scale || !w8 || !w_scale || !out) return SV_ERR_ARG;
  if (M > 1 && out_stride < N) return SV_ERR_SHAPE;
  if (!aligned(a8, 16) || !aligned(w8, 16) || !aligned(a_scale, 4) || !aligned(w_scale, 4) ||
      !aligned(out, elem_size(out_dtype)))
    return SV_ERR_ALIGN;
  const int c = check_handle(h);
  if (c != SV_OK) return c;
  sv::MatmulParams P{static_cast<const uint8_t *>(a8), static_cast<const uint8_t *>(w8), a_scale,
                     w_scale, out, out_stride, static_cast<int>(M), static_cast<int>(N),
                     static_cast<int>(K), static_cast<int>((K + 127) / 128), out_dtype};
  return sv::launch_matmul_fp8(*h, P, static_cast<cudaStream_t>(stream));
}

int spec_target_rope_freqs(const sv_rope_t *cfg, double *freqs, double *magnitude) {
  if (!cfg || !freqs || !magnitude) return SV_ERR_ARG;
  const sv_rope_t &c = *cfg;
  if (c.rot_dim < 2 || c.rot_dim > SV_MAX_HEAD_DIM || c.rot_dim % 2 != 0) return SV_ERR_SHAPE;
  if (c.scaling < SV_ROPE_PLAIN || c.scaling > SV_ROPE_YARN || !(c.base > 1.0) ||
      !std::isfinite(c.base))
    return SV_ERR_ARG;
  if (c.scaling != SV_ROPE_PLAIN && (!(c.factor >= 1.0) || !std::isfinite(c.factor)))
    return SV_ERR_ARG;
  if (c.scaling >= SV_ROPE_BANDED && (!(c.original_len >= 1.0) || !std::isfinite(c.original_len)))
    return SV_ERR_ARG;
  if (c.scaling == SV_ROPE_BANDED && !(c.low > 0.0 && c.high > c.low && std::isfinite(c.high)))
    return SV_ERR_ARG;
  if (c.scaling == SV_ROPE_YARN &&
      !(c.beta_slow > 0.0 && c.beta_fast > c.beta_slow && std::isfinite(c.beta_fast)))
    return SV_ERR_ARG;
  const double two_pi = 6.283185307179586476925286766559;
  const int half = c.rot_dim / 2;
  double base = c.base;
  if (c.scaling == SV_ROPE_NTK && c.rot_dim > 2)
    base *= std::pow(c.factor, static_cast<double>(c.rot_dim) / (c.rot_dim - 2));
  double lo = 0.0, hi = 1.0;
  *magnitude = 1.0;
  if (c.scaling == SV_ROPE_YARN) {
    // the (fractional) pair that turns `turns` times over original_len
    auto pair = [&](double turns) {
      return c.rot_dim * std::log(c.original_len / (turns * two_pi)) / (2.0 * std::log(c.base));
    };
    lo = std::fmax(std::floor(pair(c.beta_fast)), 0.0);
    hi = std::fmin(std::ceil(pair(c.beta_slow)), c.rot_dim - 1.0);
    *magnitude = 0.1 * std::log(c.factor) + 1.0;
  }
  for (int i = 0; i < half; ++i) {
    const double f0 = std::pow(base, -2.0 * i / c.rot_dim) / two_pi;
    double t;
    switch (c.scaling) {
      case SV_ROPE_LINEAR: freqs[i] = f0 / c.factor; break;
      case SV_ROPE_BANDED:
        t = std::fmin(std::fmax((c.original_len * f0 - c.low) / (c.high - c.low), 0.0), 1.0);
        freqs[i] = (1.0 - t) * f0 / c.factor + t * f0;
        break;
      case SV_ROPE_YARN:
        t = std::fmin(std::fmax((i - lo) / std::fmax(hi - lo, 0.001), 0.0), 1.0);
        freqs[i] = t * f0 / c.factor + (1.0 - t) * f0;
        break;
      default: freqs[i] = f0;
    }
  }
  return SV_OK;
}

int spec_target_rope_append(spec_target_t *h, const sv_rope_append_t *a, void *stream) {
  if (!h || !a || !float_type(a->dtype) || !std::isfinite(a->magnitude)) return SV_ERR_ARG;
  if (a->T < 0 || a->Hq < 1 || a->Hkv < 1 || a->Hq > 4096 || a->Hkv > 4096 || a->D < 1 ||
      a->D > SV_MAX_HEAD_DIM || a->rot_dim < 0 || a->rot_dim > a->D || a->rot_dim % 2 != 0 ||
      a->page_size < 1 || a->num_pages < 1)
    return SV_ERR_SHAPE;
  if (a->T == 0) return SV_OK;
  if (!a->q || !a->k || !a->v || !a->positions || !a->slots || (a->rot_dim && !a->freqs) ||
      !a->q_out || !a->k_cache || !a->v_cache)
    return SV_ERR_ARG;
  const size_t es = elem_size(a->dtype);
  for (const void *p : {a->q, a->k, a->v, static_cast<const void *>(a->q_out),
                        static_cast<const void *>(a->k_cache),
                        static_cast<const void *>(a->v_cache)})
    if (!aligned(p, es)) return SV_ERR_ALIGN;
  if (!aligned(a->positions, 8) || !aligned(a->slots, 8) || !aligned(a->freqs, 8))
    return SV_ERR_ALIGN;
  const int c = check_handle(h);
  if (c != SV_OK) return c;
  return done(sv::launch_rope_append(*a, h->status, static_cast<cudaStream_t>(stream)));
}

int spec_target_attention(spec_target_t *h, const sv_attention_t *a, void *stream) {
  if (!h || !a || !float_type(a->dtype) || !std::isfinite(a->scale) || a->window < 0 ||
      (a->tree_mask && (a->window > 0 || a->tree_words < 1)))
    return SV_ERR_ARG;
  if (a->T < 0 || a->B < 1 || a->B > SV_MAX_B || a->Hq < 1 || a->Hkv < 1 || a->Hq > 65536 ||
      a->D < 1 || a->D > SV_MAX_HEAD_DIM || a->page_size < 1 || a->max_pages < 1 ||
      a->num_pages < 1 || a->num_pages > INT32_MAX ||
      static_cast<int64_t>(a->max_pages) * a->page_size > (int64_t(1) << 30) ||
      static_cast<int64_t>(a->T) * a->Hq > (int64_t(1) << 30))
    return SV_ERR_SHAPE;
  if (a->Hq % a->Hkv != 0) return SV_ERR_ARG;
  if (a->T == 0) return SV_OK;
  if (!a->q || !a->k_cache || !a->v_cache || !a->page_table || !a->q_start || !a->kv_len ||
      !a->out)
    return SV_ERR_ARG;
  const size_t es = elem_size(a->dtype);
  if (!aligned(a->q, es) || !aligned(a->k_cache, es) || !aligned(a->v_cache, es) ||
      !aligned(a->out, es) || !aligned(a->page_table, 4) || !aligned(a->q_start, 4) ||
      !aligned(a->kv_len, 4) || !aligned(a->tree_mask, 4) || !aligned(a->lse, 4))
    return SV_ERR_ALIGN;
  const int c = check_handle(h);
  if (c != SV_OK) return c;
  return sv::launch_attention(*h, *a, static_cast<cudaStream_t>(stream));
}

int spec_target_tree_mask(spec_target_t *h, const int32_t *tree_parents, int32_t B, int32_t N,
                          int32_t *mask, void *stream) {
  if (!h || !tree_parents || !mask || B < 1 || B > SV_MAX_B || N < 1 || N > SV_MAX_K)
    return SV_ERR_ARG;
  if (!aligned(tree_parents, 4) || !aligned(mask, 4)) return SV_ERR_ALIGN;
  const int c = check_handle(h);
  if (c != SV_OK) return c;
  return done(sv::launch_tree_mask(tree_parents, B, N, mask, h->status,
                                   static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
