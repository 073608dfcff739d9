// sv_rope.cu -- rotary positions of the new tokens' queries and keys, and the
// append of K and V to their cache pages, in one launch; and the tree mask of
// the attention.
//
// One block takes one token: its rot/2 angles are formed once (64-bit product
// and reduction to a fraction of a turn, then sin and cos of pi times twice
// that in fp32, so a far position loses nothing) and shared by all heads.
// Every element is read once and written once; with many tokens HBM bounds
// it, with few the launch.
#include "sv_target.cuh"

namespace sv {
namespace {

constexpr int kRopeThreads = 256;

template <class T>
__device__ __forceinline__ void rotate_pair(T &a, T &b, float2 cs) {
  const float x = to_float(a), y = to_float(b);
  a = from_float<T>(x * cs.x - y * cs.y);
  b = from_float<T>(x * cs.y + y * cs.x);
}

// Vectors of eight elements (kVecs): a unit is the two vectors of eight
// half-layout pairs, one vector of four interleaved pairs, or one vector that
// is copied.  Otherwise single elements: a unit is one pair or one element.
template <class T, bool kVecs>
__global__ void __launch_bounds__(kRopeThreads) rope_append_kernel(const sv_rope_append_t a,
                                                                   int *status) {
  __shared__ float2 cs[SV_MAX_HEAD_DIM / 2];
  const int64_t t = blockIdx.x;
  const int half = a.rot_dim / 2;
  pdl_wait();
  pdl_launch_dependents();
  const double pos = static_cast<double>(a.positions[t]);
  for (int i = threadIdx.x; i < half; i += kRopeThreads) {
    const double turns = pos * a.freqs[i];
    const float f = static_cast<float>(turns - rint(turns));  // -1/2 .. 1/2
    float s, c;
    sincospif(2.0f * f, &s, &c);
    cs[i] = make_float2(c * a.magnitude, s * a.magnitude);
  }
  const int64_t slot = a.slots[t];
  const bool keep = slot >= 0 && slot < a.num_pages * a.page_size;
  if (threadIdx.x == 0 && !keep && slot != -1) set_status(status, SV_ERR_CACHE);
  const int64_t page = keep ? slot / a.page_size : 0;
  const int64_t off = keep ? slot - page * a.page_size : 0;
  const T *q = static_cast<const T *>(a.q) + t * a.q_token;
  const T *k = static_cast<const T *>(a.k) + t * a.k_token;
  const T *v = static_cast<const T *>(a.v) + t * a.v_token;
  T *qo = static_cast<T *>(a.q_out) + t * a.qo_token;
  T *kc = static_cast<T *>(a.k_cache) + page * a.kc_page + off * a.kc_token;
  T *vc = static_cast<T *>(a.v_cache) + page * a.vc_page + off * a.vc_token;
  __syncthreads();

  constexpr int W = kVecs ? 8 : 1;
  const int turn = kVecs ? (a.interleaved ? a.rot_dim / 8 : half / 8) : half;  // rotating units
  const int rest = (a.D - a.rot_dim) / W;                                      // copied units
  const int per = turn + rest, nqk = (a.Hq + a.Hkv) * per;
  const int total = nqk + a.Hkv * (a.D / W);
  for (int u = threadIdx.x; u < total; u += kRopeThreads) {
    if (u < nqk) {
      const int head = u / per, i = u - head * per;
      const bool isq = head < a.Hq;
      if (!isq && !keep) continue;
      const T *src = isq ? q + head * a.q_head : k + (head - a.Hq) * a.k_head;
      T *dst = isq ? qo + head * a.qo_head : kc + (head - a.Hq) * a.kc_head;
      if constexpr (kVecs) {
        if (i >= turn) {
          const int e = a.rot_dim + 8 * (i - turn);
          store8(dst + e, load8(src + e));
        } else if (a.interleaved) {
          Vec8<T> x = load8(src + 8 * i);
#pragma unroll
          for (int j = 0; j < 4; ++j) rotate_pair(x.e[2 * j], x.e[2 * j + 1], cs[4 * i + j]);
          store8(dst + 8 * i, x);
        } else {
          Vec8<T> x = load8(src + 8 * i), y = load8(src + half + 8 * i);
#pragma unroll
          for (int j = 0; j < 8; ++j) rotate_pair(x.e[j], y.e[j], cs[8 * i + j]);
          store8(dst + 8 * i, x);
          store8(dst + half + 8 * i, y);
        }
      } else {
        if (i >= turn) {
          const int e = a.rot_dim + i - turn;
          dst[e] = src[e];
        } else {
          const int e0 = a.interleaved ? 2 * i : i, e1 = a.interleaved ? 2 * i + 1 : half + i;
          T x = src[e0], y = src[e1];
          rotate_pair(x, y, cs[i]);
          dst[e0] = x;
          dst[e1] = y;
        }
      }
    } else if (keep) {
      const int w = u - nqk, per_v = a.D / W;
      const int head = w / per_v, e = (w - head * per_v) * W;
      if constexpr (kVecs)
        store8(vc + head * a.vc_head + e, load8(v + head * a.v_head + e));
      else
        vc[head * a.vc_head + e] = v[head * a.v_head + e];
    }
  }
}

template <class T>
cudaError_t launch_rope_typed(const sv_rope_append_t &a, int *status, cudaStream_t stream) {
  auto ok = [](const void *p, int64_t s0, int64_t s1, int64_t s2 = 0) {
    const int64_t es = sizeof(T);
    return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && s0 * es % 16 == 0 &&
           s1 * es % 16 == 0 && s2 * es % 16 == 0;
  };
  const bool vecs = a.D % 8 == 0 && a.rot_dim % (a.interleaved ? 8 : 16) == 0 &&
                    ok(a.q, a.q_token, a.q_head) && ok(a.k, a.k_token, a.k_head) &&
                    ok(a.v, a.v_token, a.v_head) && ok(a.q_out, a.qo_token, a.qo_head) &&
                    ok(a.k_cache, a.kc_page, a.kc_token, a.kc_head) &&
                    ok(a.v_cache, a.vc_page, a.vc_token, a.vc_head);
  const dim3 grid(static_cast<unsigned>(a.T)), block(kRopeThreads);
  if (vecs) return launch_chained(rope_append_kernel<T, true>, grid, block, 0, stream, a, status);
  return launch_chained(rope_append_kernel<T, false>, grid, block, 0, stream, a, status);
}

// Row r of a sequence: 0 the root, 1 + j node j.
__global__ void tree_mask_kernel(const int32_t *parents, int B, int N, int32_t *mask,
                                 int *status) {
  pdl_wait();
  pdl_launch_dependents();
  const int rows = N + 1, words = (rows + 31) / 32;
  const int i = blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= B * rows) return;
  const int b = i / rows;
  uint32_t m[(SV_MAX_K + 32) / 32] = {1u};
  for (int r = i - b * rows; r > 0;) {
    m[r >> 5] |= 1u << (r & 31);
    const int p = parents[static_cast<int64_t>(b) * N + r - 1];
    if (p < -1 || p >= r - 1) {
      set_status(status, SV_ERR_TOKEN);
      break;
    }
    r = p + 1;
  }
  for (int w = 0; w < words; ++w) mask[static_cast<int64_t>(i) * words + w] = m[w];
}

}  // namespace

cudaError_t launch_rope_append(const sv_rope_append_t &a, int *status, cudaStream_t stream) {
  switch (a.dtype) {
    case SV_BF16: return launch_rope_typed<__nv_bfloat16>(a, status, stream);
    case SV_FP16: return launch_rope_typed<__half>(a, status, stream);
    default: return launch_rope_typed<float>(a, status, stream);
  }
}

cudaError_t launch_tree_mask(const int32_t *parents, int B, int N, int32_t *mask, int *status,
                             cudaStream_t stream) {
  const int n = B * (N + 1);
  return launch_chained(tree_mask_kernel, dim3((n + 127) / 128), dim3(128), 0, stream, parents, B,
                        N, mask, status);
}

}  // namespace sv
