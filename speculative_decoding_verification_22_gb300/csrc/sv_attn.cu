// sv_attn.cu -- attention of new tokens over the pages: the form for every
// type, head size, page size and stride.
//
//   o = sum_j softmax_j(scale q . k_j) v_j over the keys that a token sees
//
// One warp takes one token and query head and walks its keys 32 at a time
// with a running maximum and sum: each lane forms one key's score, the lanes
// agree on the maximum, and the values are added up with the lanes spread
// over the head's elements.  A key that is not seen is never multiplied, so
// what the cache holds there does not count.
#include "sv_attn.cuh"

namespace sv {
namespace {

constexpr int kAnyWarps = 4;

template <class T>
__device__ void attend_row(const sv_attention_t &a, const SeqGeom &s, int b, int i, int head,
                           int lane, float *sq, int *status) {
  const int t = s.t0 + i;
  const T *q = static_cast<const T *>(a.q) + t * a.q_token + head * a.q_head;
  for (int d = lane; d < a.D; d += 32) sq[d] = to_float(q[d]);
  __syncwarp();
  const int kvh = head / (a.Hq / a.Hkv);
  const T *kc = static_cast<const T *>(a.k_cache) + kvh * a.kc_head;
  const T *vc = static_cast<const T *>(a.v_cache) + kvh * a.vc_head;
  const int32_t *pages = a.page_table + b * a.table_stride;
  const int32_t *tree = a.tree_mask ? a.tree_mask + static_cast<int64_t>(t) * a.tree_words
                                    : nullptr;
  int lo, hi;
  key_range(a, s, i, lo, hi);
  constexpr int kPer = SV_MAX_HEAD_DIM / 32;
  float m = -INFINITY, l = 0.0f, acc[kPer] = {};
  for (int j0 = lo; j0 < hi; j0 += 32) {
    const int j = j0 + lane;
    bool see = j < hi;
    if (see && tree && j >= s.ctx) see = tree_sees(tree, a.tree_words, j - s.ctx);
    int page = -1, off = 0;
    float x = -INFINITY;
    if (see) {
      page = pages[j / a.page_size];
      off = j % a.page_size;
      if (page < 0 || page >= a.num_pages) {
        set_status(status, SV_ERR_CACHE);
        page = -1;
      }
      x = 0.0f;
      if (page >= 0) {
        const T *k = kc + page * a.kc_page + off * a.kc_token;
        for (int d = 0; d < a.D; ++d) x = fmaf(sq[d], to_float(k[d]), x);
      }
      x *= a.scale;
    }
    // a NaN score has to reach the sums: fmaxf drops it from the maximum only
    const float top = fmaxf(m, warp_max(x));
    const float ref = top > -INFINITY ? top : 0.0f;
    const float p = see ? expf(x - ref) : 0.0f;
    const float c = m > -INFINITY ? expf(m - ref) : (l != 0.0f ? 1.0f : 0.0f);
    l = l * c + warp_sum(p);
    m = top;
#pragma unroll
    for (int e = 0; e < kPer; ++e) acc[e] *= c;
    unsigned live = __ballot_sync(0xffffffffu, see);
    while (live) {
      const int src = __ffs(live) - 1;
      live &= live - 1;
      const float ps = __shfl_sync(0xffffffffu, p, src);
      const int pg = __shfl_sync(0xffffffffu, page, src), of = __shfl_sync(0xffffffffu, off, src);
      if (pg < 0) continue;
      const T *v = vc + pg * a.vc_page + of * a.vc_token;
#pragma unroll
      for (int e = 0; e < kPer; ++e)
        if (lane + 32 * e < a.D) acc[e] = fmaf(ps, to_float(v[lane + 32 * e]), acc[e]);
    }
  }
  // nothing seen, or every score -inf: no mass
  const float inv = l != 0.0f ? 1.0f / l : 0.0f;
  T *o = static_cast<T *>(a.out) + t * a.o_token + head * a.o_head;
#pragma unroll
  for (int e = 0; e < kPer; ++e)
    if (lane + 32 * e < a.D)
      o[lane + 32 * e] = from_float<T>(l != 0.0f ? acc[e] * inv : 0.0f);
  if (a.lse && lane == 0)
    a.lse[static_cast<int64_t>(t) * a.Hq + head] = l != 0.0f ? m + logf(l) : -INFINITY;
}

template <class T>
__global__ void __launch_bounds__(32 * kAnyWarps)
    attention_any_kernel(const sv_attention_t a, int *status) {
  __shared__ float sq[kAnyWarps][SV_MAX_HEAD_DIM];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int b = blockIdx.y;
  pdl_wait();
  pdl_launch_dependents();
  bool bad;
  const SeqGeom s = seq_geom(a, b, &bad);
  if (bad && threadIdx.x == 0) set_status(status, SV_ERR_CACHE);
  const int64_t rows = static_cast<int64_t>(s.n) * a.Hq;
  for (int64_t r = static_cast<int64_t>(blockIdx.x) * kAnyWarps + warp; r < rows;
       r += static_cast<int64_t>(gridDim.x) * kAnyWarps) {
    const int i = static_cast<int>(r / a.Hq);
    __syncwarp();
    attend_row<T>(a, s, b, i, static_cast<int>(r - static_cast<int64_t>(i) * a.Hq), lane,
                  sq[warp], status);
  }
}

}  // namespace

int launch_attention(const spec_target &h, const sv_attention_t &a, cudaStream_t stream) {
  // enough blocks for every row of an even split of the tokens, at most a
  // few waves
  const int64_t want = (static_cast<int64_t>(a.T) * a.Hq + kAnyWarps - 1) / kAnyWarps;
  const int64_t cap = (16LL * h.num_sms + a.B - 1) / a.B;
  const dim3 grid(static_cast<unsigned>(want < cap ? want : cap), a.B), block(32 * kAnyWarps);
  cudaError_t e;
  switch (a.dtype) {
    case SV_BF16:
      e = launch_chained(attention_any_kernel<__nv_bfloat16>, grid, block, 0, stream, a, h.status);
      break;
    case SV_FP16:
      e = launch_chained(attention_any_kernel<__half>, grid, block, 0, stream, a, h.status);
      break;
    default:
      e = launch_chained(attention_any_kernel<float>, grid, block, 0, stream, a, h.status);
  }
  return e == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}

}  // namespace sv
