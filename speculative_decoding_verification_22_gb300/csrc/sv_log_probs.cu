// sv_log_probs.cu -- log probabilities of given tokens, entropy and the top
// alternatives of logit rows:
//
//   z = x / T, lse = log sum exp z;  z_t - lse;  H = -sum p (z - lse)
//
// With m the row's maximum and d = (x - m) / T <= 0, s = sum exp d and
// t = sum d exp d: lse - m / T = log s and H = log s - t / s.
#include <cmath>
#include <type_traits>

#include "sv_target.cuh"
#include "sv_tmem.cuh"

namespace sv {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kBytes = 16;          // of a load
constexpr int kCap = 2048;          // candidates that wait to be ranked
constexpr int kFlush = 128;         // of these are ranked
constexpr int kMaxCluster = 8;

// Order of the alternatives: the larger logit first, of equal ones the smaller
// id.  The logit's bits become an unsigned number of the same order; -0 counts
// as +0.
__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t b = __float_as_uint(x + 0.0f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float from_ordered(uint32_t u) {
  return __uint_as_float(u & 0x80000000u ? u ^ 0x80000000u : ~u);
}
__device__ __forceinline__ uint64_t order_key(float x, int id) {
  return static_cast<uint64_t>(ordered(x)) << 32 | static_cast<uint32_t>(~id);
}
constexpr uint32_t kLowest = 0x007FFFFFu, kHighest = 0xFF800000u;  // ordered(-inf), (inf)

// What one CTA knows of its part of a row, read by the first of its cluster.
struct Part {
  float m, s, t;
  int found;
  uint64_t best[SV_MAX_TOP];
};
struct Shared {
  Part part;
  uint64_t list[2][SV_MAX_TOP];
  uint64_t cand[kCap + SV_MAX_TOP];
  float red[3][kWarps];
  int count[3];  // candidates of the tiles, in turn
};

// A tile of a row in registers: kVec loads of 16 bytes a thread.
template <class T>
struct Tile {
  static constexpr int kWidth = kBytes / sizeof(T);  // elements of a load
  static constexpr int kVec = 32 / kWidth;           // 32 elements a thread
  uint4 v[kVec];
  __device__ __forceinline__ float at(int i) const {
    const uint32_t *w = reinterpret_cast<const uint32_t *>(v);
    if constexpr (sizeof(T) == 4) return __uint_as_float(w[i]);
    const uint32_t h = w[i / 2];
    if constexpr (std::is_same<T, __nv_bfloat16>::value)
      return __uint_as_float(i & 1 ? h & 0xFFFF0000u : h << 16);
    const __half2 f = *reinterpret_cast<const __half2 *>(&h);
    return i & 1 ? __high2float(f) : __low2float(f);
  }
  // Loads vectors first, first + kThreads, ... below `end`; the elements of a row
  // of V start `lead` into its first vector.  What is outside is -inf.
  __device__ __forceinline__ void load(const T *row, int lead, int V, int first, int end) {
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      const int j = first + i * kThreads, e0 = j * kWidth - lead;
      if (j < end && e0 >= 0 && e0 + kWidth <= V) {
        v[i] = __ldcs(reinterpret_cast<const uint4 *>(row + e0));
      } else {
        alignas(16) T e[kWidth];
#pragma unroll
        for (int k = 0; k < kWidth; ++k)
          e[k] = j < end && e0 + k >= 0 && e0 + k < V ? row[e0 + k] : from_float<T>(-INFINITY);
        v[i] = *reinterpret_cast<const uint4 *>(e);
      }
    }
  }
  // The largest element of each load (a NaN stays).
  __device__ __forceinline__ void maxima(float (&most)[kVec]) const {
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      most[i] = max_nan(at(i * kWidth), at(i * kWidth + 1));
#pragma unroll
      for (int k = 2; k < kWidth; k += 2)
        most[i] = max3_nan(most[i], at(i * kWidth + k), at(i * kWidth + k + 1));
    }
  }
  __device__ __forceinline__ static int index(int i, int first, int lead) {
    return (first + i / kWidth * kThreads) * kWidth + i % kWidth - lead;
  }
};

// The `top` best of the list and the candidates, in order, by counting for each
// key the greater ones (keys differ).
__device__ __forceinline__ void rank_keys(const uint64_t *keys, int n, int top, uint64_t *out) {
  for (int i = threadIdx.x; i < n; i += kThreads) {
    const uint64_t k = keys[i];
    int r = 0;
    for (int j = 0; j < n; ++j) r += keys[j] > k;
    if (r < top) out[r] = k;
  }
}

// All threads of the cluster.
__device__ __forceinline__ void cluster_sync() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// A value at the same place in another CTA's shared memory.
template <class V>
__device__ __forceinline__ V remote(const V *p, uint32_t rank) {
  uint32_t at;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(p)), "r"(rank));
  if constexpr (sizeof(V) == 8) {
    uint64_t v;
    asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(at) : "memory");
    return v;
  } else {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
    return *reinterpret_cast<const V *>(&v);
  }
}

// One cluster a row, a part of it for each CTA.
template <class T>
__global__ void __launch_bounds__(kThreads, 2)
    log_probs_kernel(const sv_log_probs_t P, int *status) {
  using R = Tile<T>;
  __shared__ Shared sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint32_t rank, parts;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(parts));
  const int64_t row = blockIdx.x / parts;
  const T *x = static_cast<const T *>(P.logits) + row * P.stride;
  const int V = static_cast<int>(P.V), top = P.top;
  const int lead = static_cast<int>((reinterpret_cast<uintptr_t>(x) & (kBytes - 1)) / sizeof(T));
  const int vecs = (lead + V + R::kWidth - 1) / R::kWidth;
  const int begin = static_cast<int>(static_cast<int64_t>(vecs) * rank / parts);
  const int end = static_cast<int>(static_cast<int64_t>(vecs) * (rank + 1) / parts);
  const float c2 = 1.4426950408889634f / P.temperature;  // to powers of two
  pdl_wait();
  pdl_launch_dependents();

  float m = -INFINITY, s = 0.0f, t = 0.0f;  // of this thread's elements, d in log2
  int found = 0, cur = 0;                   // the list's keys and its buffer
  uint32_t lim = kLowest;                   // ordered values from here are candidates
  // Candidates that wait to be ranked.  A tile counts its own in a counter of three
  // in turn, which the next tile reads behind its barrier and the one after that
  // clears, so that one barrier a tile serves.
  int waiting = 0, turn = 0, last = -1;
  if (tid < 3) sh.count[tid] = 0;
  // Ranks the list's keys and the n candidates that wait.
  auto rank_all = [&](int n) {
    for (int i = tid; i < found; i += kThreads) sh.cand[n + i] = sh.list[cur][i];
    __syncthreads();
    n += found;
    cur ^= 1;
    rank_keys(sh.cand, n, top, sh.list[cur]);
    __syncthreads();
    waiting = 0;
    last = -1;
    found = min(n, top);
    if (found == top) lim = max(lim, static_cast<uint32_t>(sh.list[cur][top - 1] >> 32) + 1);
  };
  R tile, next;
  next.load(x, lead, V, begin + tid, end);
  for (int v0 = begin; v0 < end; v0 += kThreads * R::kVec) {
    const int first = v0 + tid;
    tile = next;
    if (v0 + kThreads * R::kVec < end) next.load(x, lead, V, first + kThreads * R::kVec, end);
    float mv[R::kVec];
    tile.maxima(mv);
    float most = mv[0];
#pragma unroll
    for (int i = 1; i < R::kVec; ++i) most = max_nan(most, mv[i]);
    const float m2 = max_nan(m, most);
    if (!(m2 <= m)) {  // larger, or a NaN
      const float d = fmaxf((m - m2) * c2, -200.0f), e = ex2(d);
      t = e * fmaf(d, s, t);
      s *= e;
      m = m2;
    }
    if (m > -INFINITY) {
      const uint64_t neg = pair2(-m, -m), c = pair2(c2, c2);
      uint64_t s2 = 0, t2 = 0;
#pragma unroll
      for (int i = 0; i < 32; i += 2) {
        float2 d = unpair2(mul2(add2(pair2(tile.at(i), tile.at(i + 1)), neg), c));
        // (2^-200 is 0 here, and 0 times it stays 0 where a logit is -inf)
        d.x = fmaxf(d.x, -200.0f);
        d.y = fmaxf(d.y, -200.0f);
        const uint64_t e = pair2(ex2(d.x), ex2(d.y));
        s2 = add2(s2, e);
        t2 = fma2(pair2(d.x, d.y), e, t2);
      }
      const float2 a = unpair2(s2), b = unpair2(t2);
      s += a.x + a.y;
      t += b.x + b.y;
    }
    if (top == 0) continue;

    // ---- alternatives ----
    const uint32_t high = ordered(most);
    int n = __syncthreads_count(high >= lim);  // and the last tile's candidates are there
    if (last >= 0) waiting += sh.count[last];
    last = -1;
    turn = turn == 2 ? 0 : turn + 1;
    if (tid == 0) sh.count[turn == 2 ? 0 : turn + 1] = 0;  // the next tile's
    if (waiting > kFlush) {
      rank_all(waiting);
      n = __syncthreads_count(high >= lim);
    }
    if (n == 0) continue;
    last = turn;
    // As many threads have a candidate as there are alternatives: their maxima
    // bound the last one from below, and what lies under it is none.  Any bound
    // that `top` maxima reach will do, so the search ends early.
    if (n > top + 16) {
      uint32_t lo = lim, hi = kHighest + 1;  // count(lo) >= top > count(hi)
      while (hi - lo > 1) {
        const uint32_t mid = lo + (hi - lo) / 2;
        n = __syncthreads_count(high >= mid);
        if (n >= top) {
          lo = mid;
          if (n <= top + 16) break;
        } else {
          hi = mid;
        }
      }
      lim = lo;
      n = kThreads;  // (as many as there may be, where the search ended on a tie)
    }
    const float limf = from_ordered(lim);
    if (high >= lim) {
#pragma unroll
      for (int i = 0; i < R::kVec; ++i) {
        if (!(mv[i] >= limf) && !isnan(mv[i])) continue;
#pragma unroll
        for (int k = 0; k < R::kWidth; ++k) {
          const float y = tile.at(i * R::kWidth + k);
          if (!(y >= limf)) continue;
          const int id = R::index(i * R::kWidth + k, first, lead);
          if (id < 0 || id >= V || first + i * kThreads >= end) continue;
          const int at = waiting + atomicAdd(&sh.count[turn], 1);
          if (at < kCap) sh.cand[at] = order_key(y, id);
        }
      }
    }
    if (waiting + n * 32 <= kCap) continue;  // there was room for all of them
    __syncthreads();
    int all = waiting + sh.count[turn];
    if (all > kCap) {
      // Too many (equal) ones: the value of the tile's last alternative, then the
      // ids of those that equal it, by halving.
      auto count = [&](auto &&want) {
        int c = 0;
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          const int id = R::index(i, first, lead);
          const bool in = id >= 0 && id < V && first + i / R::kWidth * kThreads < end;
          const uint32_t u = ordered(tile.at(i));
          c += in && u <= kHighest && want(u, id);
        }
        c = __reduce_add_sync(0xffffffffu, c);
        __syncthreads();
        if (lane == 0) sh.red[0][warp] = __int_as_float(c);
        __syncthreads();
        c = 0;
        for (int w = 0; w < kWarps; ++w) c += __float_as_int(sh.red[0][w]);
        return c;
      };
      uint32_t lo = lim, hi = kHighest + 1;  // count(lo) >= top > count(hi)
      while (hi - lo > 1) {
        const uint32_t mid = lo + (hi - lo) / 2;
        if (count([&](uint32_t u, int) { return u >= mid; }) >= top)
          lo = mid;
        else
          hi = mid;
      }
      const int more = count([&](uint32_t u, int) { return u > lo; });
      int below = -1, upto = V - 1;  // ids up to `upto` are enough, up to `below` too few
      while (upto - below > 1) {
        const int mid = below + (upto - below) / 2;
        if (more + count([&](uint32_t u, int id) { return u == lo && id <= mid; }) >= top)
          upto = mid;
        else
          below = mid;
      }
      // (what waited before stays; the tile's own take the places after it)
      __syncthreads();
      if (tid == 0) sh.count[turn] = 0;
      __syncthreads();
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        const float y = tile.at(i);
        const uint32_t u = ordered(y);
        const int id = R::index(i, first, lead);
        const bool in = id >= 0 && id < V && first + i / R::kWidth * kThreads < end;
        if (in && u <= kHighest && (u > lo || (u == lo && id <= upto)))
          sh.cand[waiting + atomicAdd(&sh.count[turn], 1)] = order_key(y, id);
      }
      __syncthreads();
      all = waiting + sh.count[turn];
    }
    rank_all(all);
  }
  if (top) {
    __syncthreads();
    if (last >= 0) waiting += sh.count[last];
    if (waiting) rank_all(waiting);
  }

  // ---- the parts of a CTA, then those of the row ----
  float mb = m;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mb = max_nan(mb, __shfl_xor_sync(0xffffffffu, mb, o));
  if (lane == 0) sh.red[0][warp] = mb;
  __syncthreads();
  mb = sh.red[0][0];
  for (int w = 1; w < kWarps; ++w) mb = max_nan(mb, sh.red[0][w]);
  {
    const float d = fmaxf((m - mb) * c2, -200.0f), e = m > -INFINITY ? ex2(d) : 0.0f;
    t = e * fmaf(d, s, t);
    s *= e;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    s += __shfl_xor_sync(0xffffffffu, s, o);
    t += __shfl_xor_sync(0xffffffffu, t, o);
  }
  if (lane == 0) {
    sh.red[1][warp] = s;
    sh.red[2][warp] = t;
  }
  __syncthreads();
  if (tid == 0) {
    s = t = 0.0f;
    for (int w = 0; w < kWarps; ++w) {
      s += sh.red[1][w];
      t += sh.red[2][w];
    }
    sh.part.m = mb;
    sh.part.s = s;
    sh.part.t = t;
    sh.part.found = found;
  }
  for (int i = tid; i < found; i += kThreads) sh.part.best[i] = sh.list[cur][i];
  if (parts > 1) cluster_sync();
  else __syncthreads();
  if (rank == 0) {
    float rm = -INFINITY, rs = 0.0f, rt = 0.0f;
    int keys = 0;
    for (uint32_t q = 0; q < parts; ++q) rm = max_nan(rm, remote(&sh.part.m, q));
    for (uint32_t q = 0; q < parts; ++q) {
      const float pm = remote(&sh.part.m, q), ps = remote(&sh.part.s, q);
      const float d = fmaxf((pm - rm) * c2, -200.0f), e = pm > -INFINITY ? ex2(d) : 0.0f;
      rt += e * fmaf(d, ps, remote(&sh.part.t, q));
      rs = fmaf(e, ps, rs);
      const int f = remote(&sh.part.found, q);
      for (int i = tid; i < f; i += kThreads) sh.cand[keys + i] = remote(&sh.part.best[i], q);
      keys += f;
    }
    const bool fine = isfinite(rm);
    const float log_s = fine ? logf(rs) : NAN, inv_t = 1.0f / P.temperature;
    if (tid == 0 && P.entropy) P.entropy[row] = log_s - 0.69314718055994531f * (rt / rs);
    for (int i = tid; i < P.n; i += kThreads) {
      const int id = P.tokens[row * P.n + i];
      float y = 0.0f;
      if (id >= 0 && id < V) {
        y = (to_float(x[id]) - rm) * inv_t - log_s;
      } else if (id != -1) {
        y = NAN;
        set_status(status, SV_ERR_TOKEN);
      }
      P.log_probs[row * P.n + i] = y;
    }
    if (top) {
      __syncthreads();
      rank_keys(sh.cand, keys, top, sh.list[0]);
      __syncthreads();
      for (int i = tid; i < top; i += kThreads) {
        const uint64_t k = sh.list[0][i];
        P.top_ids[row * top + i] = fine ? static_cast<int>(~static_cast<uint32_t>(k)) : -1;
        P.top_log_probs[row * top + i] =
            fine ? (from_ordered(static_cast<uint32_t>(k >> 32)) - rm) * inv_t - log_s : NAN;
      }
    }
  }
  if (parts > 1) cluster_sync();  // nobody reads a CTA that is gone
}

template <class T>
cudaError_t launch_typed(const sv_log_probs_t &a, int num_sms, int *status,
                         cudaStream_t stream) {
  // Parts of a row: as many as fill the GPU, of at least one tile each.
  const int64_t tiles = (a.V + kThreads * 32 - 1) / (kThreads * 32);
  int parts = 1;
  while (parts < kMaxCluster && 2 * parts <= tiles && a.rows * parts < 4 * num_sms) parts *= 2;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = parts;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.rows * parts));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = parts > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, log_probs_kernel<T>, a, status);
}

}  // namespace

int log_probs_checks(const sv_log_probs_t &a) {
  if ((a.dtype != SV_BF16 && a.dtype != SV_FP16 && a.dtype != SV_FP32) ||
      !(a.temperature > 0.0f) || !std::isfinite(a.temperature) ||
      !std::isfinite(1.4426950408889634f / a.temperature) || a.n < 0)
    return SV_ERR_ARG;
  constexpr int64_t kMost = int64_t(1) << 24;
  if (a.V < 1 || a.V > kMost || a.top < 0 || a.top > SV_MAX_TOP || a.top > a.V ||
      a.n > (1 << 16) || a.rows < 0 || a.rows > kMost)
    return SV_ERR_SHAPE;
  if (a.rows == 0) return SV_OK;
  if (!a.logits || (a.n && (!a.tokens || !a.log_probs)) ||
      (a.top && (!a.top_ids || !a.top_log_probs)))
    return SV_ERR_ARG;
  if (a.rows > 1 && a.stride < a.V) return SV_ERR_SHAPE;
  auto at = [](const void *p, size_t n) { return (reinterpret_cast<uintptr_t>(p) % n) == 0; };
  return at(a.logits, a.dtype == SV_FP32 ? 4 : 2) && at(a.tokens, 4) && at(a.log_probs, 4) &&
                 at(a.entropy, 4) && at(a.top_ids, 4) && at(a.top_log_probs, 4)
             ? SV_OK
             : SV_ERR_ALIGN;
}

cudaError_t launch_log_probs(const sv_log_probs_t &a, int num_sms, int *status,
                             cudaStream_t stream) {
  switch (a.dtype) {
    case SV_BF16: return launch_typed<__nv_bfloat16>(a, num_sms, status, stream);
    case SV_FP16: return launch_typed<__half>(a, num_sms, status, stream);
    default: return launch_typed<float>(a, num_sms, status, stream);
  }
}

}  // namespace sv
