// sv_rope.cu -- rotary positions of the new tokens' queries and keys, and the
// append of K and V to their cache pages, in one launch; and the tree mask of
// the attention.
//
// One block takes one token: its rot/2 angles are formed once (the exact product
// in two 64-bit parts, reduced to a fraction of a turn, then sin and cos of pi
// times twice that in fp32, so a far position loses nothing) and shared by all
// heads.
// Every element is read once and written once; with many tokens HBM bounds
// it, with few the launch.  A thread has one unit in flight and few registers,
// so that eight blocks share an SM: 8192 tokens of 48 heads of 128 in 36.6 us
// (5.5 TB/s, in a CUDA graph); with two units a thread and six blocks 39 us, with
// three 40.
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

template <class T, bool kVecs>
struct Unit {
  using type = T;
};
template <class T>
struct Unit<T, true> {
  using type = Vec8<T>;
};
template <class U>
__device__ __forceinline__ U load_unit(const U *p) {
  if constexpr (sizeof(U) >= 16)
    return load8(p->e);
  else
    return *p;
}
template <class U>
__device__ __forceinline__ void store_unit(U *p, const U &x) {
  if constexpr (sizeof(U) >= 16)
    store8(p->e, x);
  else
    *p = x;
}

// u / d by d's 32-bit reciprocal (which is 0 for d = 1).
__device__ __forceinline__ int divide(int u, uint32_t by) {
  return by ? static_cast<int>(__umulhi(static_cast<uint32_t>(u), by)) : u;
}

// Vectors of eight elements (kVecs): a unit is the two vectors of eight
// half-layout pairs, one vector of four interleaved pairs, or one vector that
// is copied.  Otherwise single elements: a unit is one pair or one element.
template <class T, bool kVecs>
__global__ void __launch_bounds__(kRopeThreads, 8)
    rope_append_kernel(const sv_rope_append_t a, uint32_t by_per, uint32_t by_v, int *status) {
  __shared__ float2 cs[SV_MAX_HEAD_DIM / 2];
  __shared__ int64_t at_k, at_v;  // the token's place in the caches; -1: none
  const int64_t t = blockIdx.x;
  const int half = a.rot_dim / 2;
  const T *q = static_cast<const T *>(a.q) + t * a.q_token;
  const T *k = static_cast<const T *>(a.k) + t * a.k_token;
  const T *v = static_cast<const T *>(a.v) + t * a.v_token;
  T *qo = static_cast<T *>(a.q_out) + t * a.qo_token;
  constexpr int W = kVecs ? 8 : 1;
  const int turn = kVecs ? (a.interleaved ? a.rot_dim / 8 : half / 8) : half;  // rotating units
  const int per = turn + (a.D - a.rot_dim) / W;  // units of a head of q or k; the rest is copied
  const int nqk = (a.Hq + a.Hkv) * per, per_v = a.D / W;
  const int total = nqk + a.Hkv * per_v;
  using U = typename Unit<T, kVecs>::type;
  pdl_wait();
  pdl_launch_dependents();
  bool first = true;
  for (int u = threadIdx.x; u < total || first; u += kRopeThreads) {
    // the loads go out first; the first unit's hide the angles
    U x, y;
    int head = -1, unit = 0;  // head: q, then k, then v
    if (u < total) {
      if (u < nqk) {
        head = divide(u, by_per);
        unit = u - head * per;
        const T *src = head < a.Hq ? q + head * a.q_head : k + (head - a.Hq) * a.k_head;
        if (unit >= turn) {
          x = load_unit(reinterpret_cast<const U *>(src + a.rot_dim + W * (unit - turn)));
        } else if (a.interleaved) {
          src += (kVecs ? 8 : 2) * unit;
          x = load_unit(reinterpret_cast<const U *>(src));
          if constexpr (!kVecs) y = src[1];
        } else {
          src += W * unit;
          x = load_unit(reinterpret_cast<const U *>(src));
          y = load_unit(reinterpret_cast<const U *>(src + half));
        }
      } else {
        const int h = divide(u - nqk, by_v);
        head = a.Hq + a.Hkv + h;
        unit = u - nqk - h * per_v;
        x = load_unit(reinterpret_cast<const U *>(v + h * a.v_head + W * unit));
      }
    }
    if (first) {
      const double pos = static_cast<double>(a.positions[t]);
      for (int i = threadIdx.x; i < half; i += kRopeThreads) {
        // the product in two parts: its rounding to 64 bits counts among the
        // fractions of a turn from about 2^28 turns on
        const double by = a.freqs[i], turns = pos * by, rest = fma(pos, by, -turns);
        const float f = static_cast<float>((turns - rint(turns)) + rest);  // about -1/2 .. 1/2
        float s, c;
        sincospif(2.0f * f, &s, &c);
        cs[i] = make_float2(c * a.magnitude, s * a.magnitude);
      }
      if (threadIdx.x == kRopeThreads - 1) {
        const int64_t slot = a.slots[t];
        if (slot >= 0 && slot < a.num_pages * a.page_size) {
          const int64_t page = slot / a.page_size, off = slot - page * a.page_size;
          at_k = page * a.kc_page + off * a.kc_token;
          at_v = page * a.vc_page + off * a.vc_token;
        } else {
          at_k = at_v = -1;
          if (slot != -1) set_status(status, SV_ERR_CACHE);
        }
      }
      __syncthreads();
      first = false;
    }
    if (head < 0 || (head >= a.Hq && at_k < 0)) continue;
    if (head >= a.Hq + a.Hkv) {
      T *dst = static_cast<T *>(a.v_cache) + at_v + (head - a.Hq - a.Hkv) * a.vc_head;
      store_unit(reinterpret_cast<U *>(dst + W * unit), x);
      continue;
    }
    T *dst = head < a.Hq ? qo + head * a.qo_head
                         : static_cast<T *>(a.k_cache) + at_k + (head - a.Hq) * a.kc_head;
    const int i = unit;
    if (i >= turn) {
      store_unit(reinterpret_cast<U *>(dst + a.rot_dim + W * (i - turn)), x);
    } else if constexpr (kVecs) {
      if (a.interleaved) {
#pragma unroll
        for (int e = 0; e < 4; ++e) rotate_pair(x.e[2 * e], x.e[2 * e + 1], cs[4 * i + e]);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) rotate_pair(x.e[e], y.e[e], cs[8 * i + e]);
        store8(dst + half + 8 * i, y);
      }
      store8(dst + 8 * i, x);
    } else {
      rotate_pair(x, y, cs[i]);
      dst[a.interleaved ? 2 * i : i] = x;
      dst[a.interleaved ? 2 * i + 1 : half + i] = y;
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
  // ceil(2^32 / d) for divide(): exact while u * d < 2^32, and a unit's number
  // times the units of a head is below 3 * 4096 * 256 * 256
  const uint32_t w = vecs ? 8 : 1;
  const uint32_t turn = vecs ? (a.interleaved ? a.rot_dim / 8 : a.rot_dim / 16) : a.rot_dim / 2;
  const uint32_t per = turn + (a.D - a.rot_dim) / w, per_v = a.D / w;
  const uint32_t by_per = static_cast<uint32_t>(((uint64_t(1) << 32) + per - 1) / per);
  const uint32_t by_v = static_cast<uint32_t>(((uint64_t(1) << 32) + per_v - 1) / per_v);
  if (vecs)
    return launch_chained(rope_append_kernel<T, true>, grid, block, 0, stream, a, by_per, by_v,
                          status);
  return launch_chained(rope_append_kernel<T, false>, grid, block, 0, stream, a, by_per, by_v,
                        status);
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
