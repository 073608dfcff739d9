// sv_attn.cuh -- what the attention's kernels share: the geometry of a
// sequence, and which keys a new token sees.
#pragma once

#include "sv_target.cuh"

namespace sv {

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
  lo = a.window > 0 && at + 1 - a.window > 0 ? at + 1 - a.window : 0;
}
__device__ __forceinline__ bool tree_sees(const int32_t *row, int words, int jj) {
  return jj < 32 * words && ((static_cast<uint32_t>(row[jj >> 5]) >> (jj & 31)) & 1u);
}

}  // namespace sv
