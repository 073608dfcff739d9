// sv_log_probs.cu -- log probabilities of given tokens, entropy and the top
// alternatives of logit rows:
//
//   z = x / T, lse = log sum exp z;  z_t - lse;  H = -sum p (z - lse)
//
// With m the row's maximum and d = (x - m) / T <= 0, s = sum exp d and
// t = sum d exp d: lse - m / T = log s and H = log s - t / s.
//
// One pass: a thread keeps the maximum of what it has read, s and t, and puts them on
// a larger maximum when it meets one.  The alternatives come out of the same pass: the
// threads' maxima give a bound under which there are none, loads that hold anything
// from the bound on are kept in shared memory, and the few keys from the last bound on
// are ranked at the end.  Rows whose ties or order make too many candidates are read
// again by a form that halves its way to the exact one.  A row is read by one CTA, or,
// where rows are few, by a cluster whose parts the first CTA joins.
//
// What bounds it (times of kernels in a CUDA graph): HBM in fp32 (2000 x 128256 with 20
// alternatives 167 us, 6.1 TB/s; 320 x 128256 36 us, two CTAs on some SMs, three on
// others), instructions in 16 bits (4095 x 128003 in bf16 210 us with five alternatives,
// 5.0 TB/s; 169 without), and latencies for few rows: 5 x 128256 takes 8.8 us, 4.7
// without alternatives.  With one tile ahead in registers in place of two in shared
// memory these took 181, 37, 213, 179, 8.8 and 4.8; a CTA that goes on to the next row
// with its first tile on the way spills: 337 us for the bf16 rows.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "sv_target.cuh"
#include "sv_tmem.cuh"

namespace sv {
namespace {

constexpr int kVec = 4;             // loads of a thread in a tile
constexpr int kResident = 24;       // warps on an SM (the registers are bounded for it)
constexpr int kBytes = 16;          // of a load
constexpr int kRing = 3;            // tiles of a thread in shared memory
// Loads with candidates that a row keeps, and candidates of a tile where it is taken by
// itself: for a row of this many warps (fewer in short rows, of which more CTAs are to
// fit an SM).
template <int kWarps>
constexpr int stage_loads() { return kWarps == 8 ? 1024 : 192 + 32 * kWarps; }
constexpr int kFew = 256;           // candidates that are ranked
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
constexpr uint32_t kFinite = 0x00800000u, kHighest = 0xFF800000u;  // ordered(-FLT_MAX), (inf)

// What one CTA knows of its part of a row, read by the first of its cluster.
struct Part {
  float m, s, t;
  int found;
  uint64_t best[SV_MAX_TOP];
};
template <int kWarps>
struct Shared {
  static constexpr int kStage = stage_loads<kWarps>(), kCap = stage_loads<kWarps>();
  Part part;
  uint64_t list[2][SV_MAX_TOP];
  uint64_t few[kFew];
  union {
    struct {
      uint4 load[kStage];
      int at[kStage];
    } stage;
    uint64_t cand[kCap + SV_MAX_TOP];
  };
  float red[3][kMaxCluster];
  uint32_t bound[kWarps], first;
  int count, few_count;
};

// The loads of 16 bytes of a CTA's part of a row: `row` is 16-byte aligned, and
// its first element has the id `id0` (what lies before it and behind the last load
// of the row are its edges).
template <class T, int kWarps>
struct Span {
  static constexpr int kThreads = 32 * kWarps;
  static constexpr int kWidth = kBytes / sizeof(T);  // elements of a load
  static constexpr int kPer = kVec * kWidth;         // elements of a thread in a tile
  static constexpr int kTile = kThreads * kVec;      // of a tile
  const T *row;
  int id0, begin, end;
  __device__ __forceinline__ bool has(int load) const { return load < end; }
  // The id of element i of a thread whose first load of the tile is `first`.
  __device__ __forceinline__ int id(int i, int first) const {
    return id0 + (first + i / kWidth * kThreads) * kWidth + i % kWidth;
  }
};

template <class T>
__device__ __forceinline__ float element(const uint4 &v, int i) {
  const uint32_t *w = reinterpret_cast<const uint32_t *>(&v);
  if constexpr (sizeof(T) == 4) return __uint_as_float(w[i]);
  const uint32_t h = w[i / 2];
  if constexpr (std::is_same<T, __nv_bfloat16>::value)
    return __uint_as_float(i & 1 ? h & 0xFFFF0000u : h << 16);
  const __half2 f = *reinterpret_cast<const __half2 *>(&h);
  return i & 1 ? __high2float(f) : __low2float(f);
}

// A tile in registers.
template <class T, int kWarps>
struct Tile {
  using S = Span<T, kWarps>;
  static constexpr int kThreads = S::kThreads;
  uint4 v[kVec];
  __device__ __forceinline__ float at(int i) const {
    return element<T>(v[i / S::kWidth], i % S::kWidth);
  }
  // The tile from load v0 on; -inf behind the part.
  __device__ __forceinline__ void load(const S &s, int v0) {
    const T low = from_float<T>(-INFINITY);
    uint32_t w = 0xFF800000u;
    if constexpr (sizeof(T) == 2) w = *reinterpret_cast<const uint16_t *>(&low) * 0x10001u;
    const int first = v0 + threadIdx.x;
    const uint4 *p = reinterpret_cast<const uint4 *>(s.row) + first;
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      v[i] = make_uint4(w, w, w, w);
      if (s.has(first + i * kThreads)) v[i] = __ldcs(p + i * kThreads);
    }
  }
  // The same in two steps: the copy of the thread's loads into its own places of a ring
  // in shared memory, and the read of what it copied itself.
  __device__ __forceinline__ static void copy(const S &s, int v0, uint32_t ring) {
    const int first = v0 + threadIdx.x;
    const uint4 *p = reinterpret_cast<const uint4 *>(s.row) + first;
#pragma unroll
    for (int i = 0; i < kVec; ++i)
      if (s.has(first + i * kThreads))
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                         ring + i * kThreads * kBytes),
                     "l"(p + i * kThreads)
                     : "memory");
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
  __device__ __forceinline__ void read(const S &s, int v0, uint32_t ring) {
    const T low = from_float<T>(-INFINITY);
    uint32_t w = 0xFF800000u;
    if constexpr (sizeof(T) == 2) w = *reinterpret_cast<const uint16_t *>(&low) * 0x10001u;
    const int first = v0 + threadIdx.x;
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      v[i] = make_uint4(w, w, w, w);
      if (s.has(first + i * kThreads))
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(v[i].x), "=r"(v[i].y), "=r"(v[i].z), "=r"(v[i].w)
                     : "r"(ring + i * kThreads * kBytes)
                     : "memory");
    }
  }
  // The largest element of each load (a NaN stays).
  __device__ __forceinline__ void maxima(float (&most)[kVec]) const {
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      most[i] = max_nan(at(i * S::kWidth), at(i * S::kWidth + 1));
#pragma unroll
      for (int k = 2; k < S::kWidth; k += 2)
        most[i] = max3_nan(most[i], at(i * S::kWidth + k), at(i * S::kWidth + k + 1));
    }
  }
};

// The `top` best of n keys, in order, by counting for each the greater ones (keys
// differ).
__device__ __forceinline__ void rank_keys(const uint64_t *keys, int n, int top, uint64_t *out) {
  for (int i = threadIdx.x; i < n; i += blockDim.x) {
    const uint64_t k = keys[i];
    int r = 0;
#pragma unroll 4
    for (int j = 0; j < n; ++j) r += keys[j] > k;
    if (r < top) out[r] = k;
  }
}

// The best keys so far and the bound under which there are none.  All threads of
// the block call its functions, which agree on n and on what is kept here.
template <int kWarps>
struct Best {
  using Sh = Shared<kWarps>;
  static constexpr int kThreads = 32 * kWarps;
  int top, warps;
  int found = 0, cur = 0;   // the list's keys and its buffer
  uint32_t lim = kFinite;   // ordered values from here are candidates

  // Ranks the n candidates with the list.
  __device__ __forceinline__ void rank(int n, Sh &sh) {
    for (int i = threadIdx.x; i < found; i += kThreads) sh.cand[n + i] = sh.list[cur][i];
    __syncthreads();
    n += found;
    cur ^= 1;
    rank_keys(sh.cand, n, top, sh.list[cur]);
    if (threadIdx.x == 0) sh.count = 0;
    __syncthreads();
    found = min(n, top);
    // (what comes later and equals the last one has a larger id)
    if (found == top) lim = max(lim, static_cast<uint32_t>(sh.list[cur][top - 1] >> 32) + 1);
  }
  // Each of the warps that have a load for every lane (or the first alone) has
  // ceil(top / warps) elements, of different threads, from a bound on, so what lies
  // under it is no alternative; the bound is the least of the warps' own.  `most` is
  // the thread's largest element so far.  A warp's bound only rises, so a read without
  // a barrier is of a bound too, maybe a lower one.
  __device__ __forceinline__ void publish(float most, Sh &sh) const {
    uint32_t u = ordered(most), bound = 0;
    for (int r = (top + warps - 1) / warps; r > 0; --r) {
      bound = __reduce_max_sync(0xffffffffu, u);
      const uint32_t who = __ballot_sync(0xffffffffu, u == bound);
      if ((threadIdx.x & 31) == __ffs(who) - 1) u = 0;
    }
    if ((threadIdx.x & 31) == 0)
      *const_cast<volatile uint32_t *>(&sh.bound[threadIdx.x >> 5]) = bound;
    __syncwarp();
  }
  __device__ __forceinline__ void raise(const Sh &sh) {
    const volatile uint32_t *bounds = sh.bound;
    uint32_t bound = bounds[0];
    for (int w = 1; w < warps; ++w) bound = min(bound, bounds[w]);
    lim = max(lim, bound);
  }
};

// The best of a part whose tiles are taken one by one, however many of their
// elements equal each other or rise; `edges` keys of the row's edges (and of a part's
// first elements) lie in `few` and come last, so that the tiles are met in the order of
// their ids.
template <class T, int kWarps>
__device__ __noinline__ Best<kWarps> best_of_each(const Span<T, kWarps> s, int edges,
                                                 Best<kWarps> best, Shared<kWarps> &sh) {
  using S = Span<T, kWarps>;
  constexpr int kThreads = S::kThreads;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  __syncthreads();
  if (threadIdx.x == 0) sh.count = 0;
  for (int v0 = s.begin; v0 < s.end; v0 += S::kTile) {
    const int first = v0 + threadIdx.x;
    Tile<T, kWarps> tile;
    tile.load(s, v0);
    float most = tile.at(0);
#pragma unroll
    for (int i = 1; i < S::kPer; ++i) most = max_nan(most, tile.at(i));
    best.publish(most, sh);
    __syncthreads();
    best.raise(sh);
    __syncthreads();
    // Elements that `want` takes: how many there are, and writing them.
    auto count = [&](auto &&want) {
      int c = 0;
#pragma unroll
      for (int i = 0; i < S::kPer; ++i) {
        const uint32_t u = ordered(tile.at(i));
        c += s.has(first + i / S::kWidth * kThreads) && u <= kHighest && want(u, s.id(i, first));
      }
      c = __reduce_add_sync(0xffffffffu, c);
      __syncthreads();
      if (lane == 0) sh.red[0][warp] = __int_as_float(c);
      __syncthreads();
      c = 0;
      for (int w = 0; w < kWarps; ++w) c += __float_as_int(sh.red[0][w]);
      return c;
    };
    uint32_t lo = best.lim;
    int upto = s.id0 + s.end * S::kWidth;  // of those that equal lo
    int n = count([&](uint32_t u, int) { return u >= lo; });
    if (n == 0) continue;
    if (n > sh.kCap) {
      // the value of the tile's last alternative, then the ids of those that equal
      // it, by halving
      uint32_t hi = kHighest + 1;  // count(lo) >= top > count(hi)
      while (hi - lo > 1) {
        const uint32_t mid = lo + (hi - lo) / 2;
        if (count([&](uint32_t u, int) { return u >= mid; }) >= best.top)
          lo = mid;
        else
          hi = mid;
      }
      const int more = count([&](uint32_t u, int) { return u > lo; });
      int below = -1;  // ids up to `upto` are enough, up to `below` too few
      while (upto - below > 1) {
        const int mid = below + (upto - below) / 2;
        if (more + count([&](uint32_t u, int id) { return u == lo && id <= mid; }) >= best.top)
          upto = mid;
        else
          below = mid;
      }
    }
#pragma unroll
    for (int i = 0; i < S::kPer; ++i) {
      const uint32_t u = ordered(tile.at(i));
      const int id = s.id(i, first);
      if (s.has(first + i / S::kWidth * kThreads) && u <= kHighest &&
          (u > lo || (u == lo && id <= upto))) {
        const int j = atomicAdd(&sh.count, 1);
        if (j < sh.kCap) sh.cand[j] = order_key(tile.at(i), id);
      }
    }
    __syncthreads();
    n = min(sh.count, static_cast<int>(sh.kCap));
    __syncthreads();
    best.rank(n, sh);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < edges; i += kThreads) sh.cand[i] = sh.few[i];
  best.rank(edges, sh);
  return best;
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
template <class T, int kWarps>
__global__ void __launch_bounds__(32 * kWarps, kResident / kWarps)
    log_probs_kernel(const sv_log_probs_t P, int *status) {
  using S = Span<T, kWarps>;
  constexpr int kThreads = S::kThreads;
  static_assert(kThreads >= SV_MAX_TOP);
  __shared__ Shared<kWarps> sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint32_t rank, parts;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(parts));
  const int V = static_cast<int>(P.V), top = P.top;
  const float c2 = 1.4426950408889634f / P.temperature;  // to powers of two
  const float inv_t = 1.0f / P.temperature;
  const int64_t row = blockIdx.x / parts;
  const T *x = static_cast<const T *>(P.logits) + row * P.stride;
  S s;
  s.id0 = static_cast<int>((0 - reinterpret_cast<uintptr_t>(x)) % kBytes / sizeof(T));
  s.id0 = min(s.id0, V);
  s.row = x + s.id0;
  const int loads = (V - s.id0) / S::kWidth;
  s.begin = static_cast<int>(static_cast<int64_t>(loads) * rank / parts);
  s.end = static_cast<int>(static_cast<int64_t>(loads) * (rank + 1) / parts);
  // the edges: one element for some of the first CTA's threads
  const int tail = s.id0 + loads * S::kWidth;
  int edges = rank == 0 ? s.id0 + V - tail : 0;
  if (tid == 0) {
    sh.count = 0;
    sh.few_count = edges;
    sh.first = kFinite - 1;
  }
  pdl_wait();
  pdl_launch_dependents();

  // two tiles are on their way while one is worked on
  extern __shared__ uint4 ring_raw[];
  const uint32_t ring = smem_u32(ring_raw) + tid * kBytes;
  constexpr uint32_t kSlot = S::kTile * kBytes;
  Tile<T, kWarps> tile;
  for (int i = 0; i + 1 < kRing; ++i) tile.copy(s, s.begin + i * S::kTile, ring + i * kSlot);
  uint32_t slot = 0;
  float m = -INFINITY, sum = 0.0f, t = 0.0f;  // of this thread's elements, d in log2
  if (tid < edges) {
    const int id = tid < s.id0 ? tid : tail + tid - s.id0;
    m = to_float(x[id]);
    sum = m > -INFINITY ? 1.0f : 0.0f;
    sh.few[tid] = order_key(m, id);
  }
  // the logit of a given token: NaN outside the vocabulary
  auto given = [&](int i) {
    const int id = P.tokens[row * P.n + i];
    if (id >= 0 && id < V) return to_float(x[id]);
    if (id == -1) return 0.0f;  // none
    set_status(status, SV_ERR_TOKEN);
    return NAN;
  };
  const float early = rank == 0 && tid < P.n ? given(tid) : 0.0f;
  Best<kWarps> best;
  best.top = top;
  best.warps = max(1, min(kWarps, (s.end - s.begin) / 32));
  // Loads with candidates are kept without a barrier between the tiles, under a bound
  // that rises from time to time.
  int next_start = 0, number = 0;
  for (int v0 = s.begin; v0 < s.end; v0 += S::kTile, ++number) {
    asm volatile("cp.async.wait_group %0;" ::"n"(kRing - 2) : "memory");
    tile.read(s, v0, ring + slot * kSlot);
    // (into the place of the last tile, which this thread has read)
    tile.copy(s, v0 + (kRing - 1) * S::kTile, ring + (slot == 0 ? kRing - 1 : slot - 1) * kSlot);
    slot = slot + 1 == kRing ? 0 : slot + 1;
    float mv[kVec];
    tile.maxima(mv);
    float most = mv[0];
#pragma unroll
    for (int i = 1; i < kVec; ++i) most = max_nan(most, mv[i]);
    const float m2 = max_nan(m, most);
    if (!(m2 <= m)) {  // larger, or a NaN
      const float d = fmaxf((m - m2) * c2, -200.0f), e = ex2(d);
      t = e * fmaf(d, sum, t);
      sum *= e;
      m = m2;
    }
    if (m > -INFINITY) {
      const uint64_t neg = pair2(-m, -m), c = pair2(c2, c2);
      uint64_t s2 = 0, t2 = 0;
#pragma unroll
      for (int i = 0; i < S::kPer; i += 2) {
        float2 d = unpair2(mul2(add2(pair2(tile.at(i), tile.at(i + 1)), neg), c));
        // (2^-200 is 0 here, and 0 times it stays 0 where a logit is -inf)
        d.x = fmaxf(d.x, -200.0f);
        d.y = fmaxf(d.y, -200.0f);
        const uint64_t e = pair2(ex2(d.x), ex2(d.y));
        s2 = add2(s2, e);
        t2 = fma2(pair2(d.x, d.y), e, t2);
      }
      const float2 a = unpair2(s2), b = unpair2(t2);
      sum += a.x + a.y;
      t += b.x + b.y;
    }
    if (top) {
      if (number == next_start) {
        best.publish(m, sh);
        if (number == 0) __syncthreads();
        best.raise(sh);
        // Behind the part's first `top` elements, one that only equals the least of them
        // is no alternative.  Ties at a row's least value, as a mask makes them, are no
        // candidates so, but for those first ones (with them, rows of 128256 masked down
        // to 10 were read again: 5 rows took 26.8 us in place of 8.1, 320 rows 120 in
        // place of 32).  A warp looks there if all its threads have a candidate.
        if (number == 0 && __all_sync(0xffffffffu, ordered(most) >= best.lim) &&
            (s.end - s.begin) * S::kWidth >= top) {
          uint32_t u = kHighest;
#pragma unroll 1
          for (int i = lane; i < top; i += 32)
            u = min(u, ordered(to_float(s.row[s.begin * S::kWidth + i])));
          u = max(__reduce_min_sync(0xffffffffu, u), kFinite - 1);
          if (lane == 0) sh.first = u;
          best.lim = max(best.lim, u + 1);
        }
        next_start = number == 0 ? 1 : number < 32 ? 2 * number : number + 32;
      }
      const float lim = from_ordered(best.lim);
      if (!(most < lim)) {
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
          if (!(mv[i] >= lim) || !s.has(v0 + tid + i * kThreads)) continue;
          const int j = atomicAdd(&sh.count, 1);
          if (j < sh.kStage) {
            sh.stage.load[j] = tile.v[i];
            sh.stage.at[j] = v0 + tid + i * kThreads;
          }
        }
      }
    }
  }
  if (top) {
    best.publish(m, sh);
    __syncthreads();
    best.raise(sh);
    best.lim = max(best.lim, sh.first + 1);
    const int n = sh.count;
    if (best.lim == sh.first + 1) {
      // maybe not `top` from it on: the first ones fill up
      const bool inside = tid < min(top, (s.end - s.begin) * S::kWidth);
      const float y = inside ? to_float(s.row[s.begin * S::kWidth + tid]) : INFINITY;
      const bool fill = ordered(y) < best.lim;
      if (fill)
        sh.few[atomicAdd(&sh.few_count, 1)] = order_key(y, s.id0 + s.begin * S::kWidth + tid);
      edges += __syncthreads_count(fill);
    }
    if (n <= sh.kStage) {
      for (int i = tid; i < n * S::kWidth; i += kThreads) {
        const int j = i / S::kWidth, k = i % S::kWidth;
        const float y = to_float(reinterpret_cast<const T *>(&sh.stage.load[j])[k]);
        if (ordered(y) < best.lim) continue;
        const int at = atomicAdd(&sh.few_count, 1);
        if (at < kFew) sh.few[at] = order_key(y, s.id0 + sh.stage.at[j] * S::kWidth + k);
      }
      __syncthreads();
    }
    const int few = sh.few_count;
    if (n > sh.kStage || few > kFew) {
      best = best_of_each(s, edges, best, sh);  // some were not kept
    } else {
      rank_keys(sh.few, few, top, sh.list[0]);
      best.found = min(few, top);
    }
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
    t = e * fmaf(d, sum, t);
    sum *= e;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    sum += __shfl_xor_sync(0xffffffffu, sum, o);
    t += __shfl_xor_sync(0xffffffffu, t, o);
  }
  if (lane == 0) {
    sh.red[1][warp] = sum;
    sh.red[2][warp] = t;
  }
  __syncthreads();
  sum = t = 0.0f;
  for (int w = 0; w < kWarps; ++w) {
    sum += sh.red[1][w];
    t += sh.red[2][w];
  }
  const uint64_t *keys = sh.list[best.cur];
  if (parts > 1) {
    if (tid == 0) {
      sh.part.m = mb;
      sh.part.s = sum;
      sh.part.t = t;
      sh.part.found = best.found;
    }
    for (int i = tid; i < best.found; i += kThreads) sh.part.best[i] = keys[i];
    cluster_sync();
    if (rank == 0) {
      // a warp for each part; keys that a part lacks are 0, below every other
      for (int q = warp; q < static_cast<int>(parts); q += kWarps) {
        if (lane == 0) sh.red[0][q] = remote(&sh.part.m, q);
        if (lane == 1) sh.red[1][q] = remote(&sh.part.s, q);
        if (lane == 2) sh.red[2][q] = remote(&sh.part.t, q);
        const int f = remote(&sh.part.found, q);
        for (int i = lane; i < top; i += 32)
          sh.cand[q * top + i] = i < f ? remote(&sh.part.best[i], q) : 0;
      }
      __syncthreads();
      mb = sh.red[0][0];
      for (uint32_t q = 1; q < parts; ++q) mb = max_nan(mb, sh.red[0][q]);
      sum = t = 0.0f;
      for (uint32_t q = 0; q < parts; ++q) {
        const float pm = sh.red[0][q];
        const float d = fmaxf((pm - mb) * c2, -200.0f), e = pm > -INFINITY ? ex2(d) : 0.0f;
        t += e * fmaf(d, sh.red[1][q], sh.red[2][q]);
        sum = fmaf(e, sh.red[1][q], sum);
      }
      keys = sh.list[0];
      rank_keys(sh.cand, static_cast<int>(parts) * top, top, sh.list[0]);
      __syncthreads();
    }
    cluster_sync();  // nobody reads a CTA that is gone
  }
  if (rank == 0) {
    const bool fine = isfinite(mb);
    const float log_s = fine ? logf(sum) : NAN;
    if (tid == 0 && P.entropy) P.entropy[row] = log_s - 0.69314718055994531f * (t / sum);
    for (int i = tid; i < P.n; i += kThreads) {
      const float y = i == tid ? early : given(i);
      const bool none = P.tokens[row * P.n + i] == -1;
      P.log_probs[row * P.n + i] = none ? 0.0f : (y - mb) * inv_t - log_s;
    }
    for (int i = tid; i < top; i += kThreads) {
      const uint64_t k = keys[i];
      P.top_ids[row * top + i] = fine ? static_cast<int>(~static_cast<uint32_t>(k)) : -1;
      P.top_log_probs[row * top + i] =
          fine ? (from_ordered(static_cast<uint32_t>(k >> 32)) - mb) * inv_t - log_s : NAN;
    }
  }
}

template <class T, int kWarps>
cudaError_t launch_warps(const sv_log_probs_t &a, int parts, int *status, cudaStream_t stream) {
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = parts;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.rows * parts));
  cfg.blockDim = dim3(32 * kWarps);
  cfg.dynamicSmemBytes = kRing * Span<T, kWarps>::kTile * kBytes;
  const cudaError_t e = cudaFuncSetAttribute(log_probs_kernel<T, kWarps>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             kRing * Span<T, kWarps>::kTile * kBytes);
  if (e != cudaSuccess) return e;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = parts > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, log_probs_kernel<T, kWarps>, a, status);
}
template <class T>
cudaError_t launch_typed(const sv_log_probs_t &a, int num_sms, int *status,
                         cudaStream_t stream) {
  // Eight warps a CTA where a row has eight of their tiles (128 KB), fewer for short
  // rows, whose start and end then run beside more others': 4000 rows of 20000 in
  // bf16 took 75 us with eight warps, 55 with four, 56 with two; 16000 of 2000 156, 82
  // and 56; 4095 of 128003 226, 216 and 261, 320 of 128256 in fp32 36.5, 50 and 87 (with
  // one tile ahead, in registers).  Parts of a row only where rows leave SMs idle, as
  // clusters start slowly: 40 rows of 128256 took 16.8 us in one part, 11.3 in six; 320
  // 44 in one and 51 in two.
  constexpr int64_t kTileBytes = 256 * kVec * kBytes;
  const int64_t bytes = a.V * static_cast<int64_t>(sizeof(T));
  const int64_t most = std::min<int64_t>(2 * num_sms / a.rows, (bytes - 1) / kTileBytes + 1);
  const int parts = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(most, kMaxCluster)));
  if (parts > 1 || bytes >= 8 * kTileBytes) return launch_warps<T, 8>(a, parts, status, stream);
  if (bytes >= kTileBytes) return launch_warps<T, 4>(a, 1, status, stream);
  return launch_warps<T, 2>(a, 1, status, stream);
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
