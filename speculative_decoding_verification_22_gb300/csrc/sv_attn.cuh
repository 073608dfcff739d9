// sv_attn.cuh -- what the attention's kernels share: the geometry of a
// sequence, and which keys a new token sees.
#pragma once

#include "sv_target.cuh"

namespace sv {

// The tensor-core form (16-bit types): its result, or kNotTaken where the
// layout is none of its own.
constexpr int kNotTaken = 1;
int launch_attention_tc(const spec_target &h, const sv_attention_t &a, cudaStream_t stream);

struct SeqGeom {
  int t0;   // first new token
  int n;    // new tokens
  int kv;   // cached tokens, the new ones included
  int ctx;  // kv - n: index of the first new token (negative if kv < n)
};

// Reads and checks one sequence's lengths.  A token range outside [0, T]
// counts as empty, a cache length out of bounds as 0; *bad is set for both.
__device__ __forceinline__ SeqGeom seq_geom(const sv_attention_t &a, int b, bool *bad) {
  int t0 = a.q_start[b], t1 = a.q_start[b + 1];
  int kv = a.kv_len[b];
  *bad = false;
  if (t0 < 0 || t1 < t0 || t1 > a.T) {
    *bad = true;
    t0 = t1 = 0;
  }
  if (kv < 0 || kv > static_cast<int64_t>(a.max_pages) * a.page_size) {
    *bad = true;
    kv = 0;
  }
  return SeqGeom{t0, t1 - t0, kv, kv - (t1 - t0)};
}

// New token i sees the keys [lo, hi) and, under a tree mask, of those from
// ctx on only the ones whose bit is set.
__device__ __forceinline__ void key_range(const sv_attention_t &a, const SeqGeom &s, int i,
                                          int &lo, int &hi) {
  const int at = s.ctx + i;
  hi = a.tree_mask ? s.kv : at + 1;  // kv bounds both
  if (hi > s.kv) hi = s.kv;
  if (hi < 0) hi = 0;
  lo = a.window > 0 && at >= a.window ? at + 1 - a.window : 0;
}
__device__ __forceinline__ bool tree_sees(const int32_t *row, int words, int jj) {
  return jj < 32 * words && ((static_cast<uint32_t>(row[jj >> 5]) >> (jj & 31)) & 1u);
}

// One warp attends with one token and query head over its keys, 32 at a time
// with a running maximum and sum: each lane forms one key's score, the lanes
// agree on the maximum, and the values are added up with the lanes spread
// over the head's elements.  A key that is not seen is never multiplied, so
// what the cache holds there does not count.  It writes the elements [d0, d1) of
// the row, and the lse with element 0.
template <class T>
__device__ __noinline__ void attend_row(const sv_attention_t &a, const SeqGeom &s, int b, int i,
                                        int head, int lane, int *status, int d0 = 0,
                                        int d1 = SV_MAX_HEAD_DIM) {
  const int t = s.t0 + i;
  const T *q = static_cast<const T *>(a.q) + t * a.q_token + head * a.q_head;
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
        for (int d = 0; d < a.D; ++d) x = fmaf(to_float(q[d]), to_float(k[d]), x);
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
    if (lane + 32 * e < a.D && lane + 32 * e >= d0 && lane + 32 * e < d1)
      o[lane + 32 * e] = from_float<T>(l != 0.0f ? acc[e] * inv : 0.0f);
  if (a.lse && lane == 0 && d0 == 0)
    a.lse[static_cast<int64_t>(t) * a.Hq + head] = l != 0.0f ? m + logf(l) : -INFINITY;
}

}  // namespace sv
