// sv_attn_tc.cu -- attention of new tokens over the pages on the tensor
// cores (bf16, fp16): tcgen05 products with the scores, the weights and the
// output in tensor memory, K and V brought page by page by TMA.
//
//   o = sum_j softmax_j(scale q . k_j) v_j
//
// in one pass over the keys with a running maximum m and sum l of each row:
// a tile of keys gives S = Q K^T, P = 2^((S - m) scale log2 e), and
// O += P V.  m only moves when a row's maximum has grown by more than 2^8, so
// that O is rarely rescaled; l and O stay relative to the m they were summed
// with.  P is rounded to the 16-bit type for its product (half a step a weight),
// l sums it unrounded.  fp16 has few exponents below one: there P, and with it
// l and O, carry a further 2^7 (up to 2^15 of 2^16), so that a weight is lost
// only below 2^-32 of the row's largest, and not below 2^-25, of which 2^17 equal
// ones under one large weight would be missed by 0.2% of the output.
//
//  * The rows of one cache head are its new tokens times the G = Hq / Hkv
//    query heads that share it, so each K and V tile serves all of them.  An
//    item is one (sequence, cache head, block of rows): up to 128 rows
//    ("narrow": a verification round, single tokens) or 256 ("wide").
//  * Two slots (S, P and O in tensor memory, one warpgroup for the softmax)
//    work in turn, so that one slot's products run under the other's softmax.
//    Wide: a slot holds 128 of the rows and both take every K and V tile of
//    128 keys.  Narrow: both hold the same rows, slot 0 takes the even tiles
//    of 64 keys and slot 1 the odd ones, and their sums are joined at the end.
//    (Narrow is bound by the cache's bytes: with tiles of 128 keys the two
//    slots held four fifths of the ring while it should have been loading.)
//  * A persistent grid, one CTA per SM; the (item, tile) units of the whole
//    call are cut into equal runs, so ragged lengths and few sequences fill
//    all SMs alike.  An item that is cut leaves its parts' (m, l, O) in the
//    handle's scratch and a second launch joins them in a fixed order.  The
//    lengths are read on the device: no host plan, a graph replays with new
//    ones.
//  * Warps 0-3 and 4-7: softmax of the two slots, one row a thread; warp 8,
//    and warp 11 for the V of narrow tiles: TMA into a ring of 160 KB; warp 9:
//    the products; warp 10 hands out the items.
//
// What bounds it (times in this file are of kernels in a CUDA graph, but for those
// at report_pages).  Cached bytes, for few rows a head: 64 single tokens over 2048
// to 8192 in 211 us, 6.4 TB/s (210 to 222 by single calls).  Products, for many:
// 4096 tokens over 16384 in 657 us, 1.46 PFLOP/s (675 to 685 by single calls),
// where the scores' product reads 8 KB of shared memory
// in each of its 64 cycles, all that there is, beside the copies that arrive.
// Latency, for short calls and short sequences: 5 tokens over 1000 in 14.4 us
// (4 of them the second launch), and about 8 us an item of up to 512 keys (256
// single tokens over 512: 117 us).  Tried and slower: a warp of its own for
// each slot's products (834 us against 688), an item's queries fetched under
// the last one's end (669 against 653), half a wide tile's weights handed over
// at a time (665 against 663).
//
// What is masked must not count even where it is not finite: keys past the
// sequence are zeroed in V's tile, and a row whose output is not finite is
// taken again by attend_row, which multiplies only what the row sees.
#include <cudaTypedefs.h>

#include <type_traits>

#include "sv_attn.cuh"
#include "sv_tmem.cuh"

namespace sv {
namespace {

constexpr int kWideKeys = 128, kNarrowKeys = 64;  // keys of a tile
constexpr int kRows = 128;     // rows of a slot
constexpr int kThreads = 384;
// Registers a thread: 168 at launch; the softmax warpgroups take what the
// third one gives back (256 * 216 + 128 * 72 = 384 * 168).
constexpr int kSoftmaxRegs = 216, kOtherRegs = 72;
constexpr int kSoftmaxWarps = 8;
constexpr int kRingBytes = 160 * 1024;
// Pages up to this size come with both 128-byte halves of a row in one box, as
// a warp takes about 55 ns to issue one whatever it holds: 4096 tokens over 16384
// in pages of 8 and 16 take 749 and 682 us against 1123 and 766, 64 single tokens
// over 8192 209 and 207 against 260 and 209; pages of 32 and more gain nothing.
constexpr int kPairedPage = 16;
constexpr int kMaxSlots = 10;
constexpr uint64_t kCleanupLimitNs = 2000000000ull;
constexpr float kRescale = 8.0f;  // log2 of the growth of m that rescales O
// log2 of what P, l and O carry beside the weights: fp16 ends at 2^16, which
// leaves kRescale 7 and a bit; bf16 has fp32's exponents.
template <class T>
constexpr float carried() { return __is_same(T, __half) ? 7.0f : 0.0f; }
constexpr float kLn2 = 0.69314718055994531f;

template <int DPAD>
struct Shape {
  static constexpr int kSlabs = DPAD / 64;          // 128-byte columns of a tile
  // A slot of the ring: a wide tile of K or V, or a narrow tile's K and V.
  static constexpr int kSlotBytes = kWideKeys * DPAD * 2;
  static constexpr int kSlots = kRingBytes / kSlotBytes;
  static constexpr int kQBytes = kRows * DPAD * 2;
  static constexpr int kSmem = 1024 + 2 * kQBytes + kRingBytes;  // + Ctl
};

// One item of this CTA's run, as the scheduling warp hands it to the others.
struct Run {
  int n;            // tiles of it in this run; 0: no more items
  int tile0;        // its first tile
  int wide;         // 256 rows rather than 128
  int whole;        // all of the item's tiles are here
  int once;         // its cache is read by one or two items, not by many
  int part;         // where its part goes: 0 it began earlier, 1 it begins here
  int b, h, r0, rows;
  SeqGeom s;
};
constexpr int kRuns = 4;

struct Ctl {
  Run run[kRuns];
  uint64_t run_full[kRuns], run_empty[kRuns];
  uint64_t full[kMaxSlots], empty[kMaxSlots];
  uint64_t q_ready, s_full[2], p_ready[2], o_full, x_full, x_free, teardown;
  uint32_t tmem;
  int abort;
  int slow;           // a softmax warp is in attend_row: waits go on
  int issued[2], consumed;  // slots of the ring
  int start_b;
  int64_t start_off, start_per;
  int64_t scan[kThreads / 32];
  float xm[kRows], xl[kRows];
};

// A cut item's parts: which CTAs of its walk hold some, and whose rows.
constexpr int kMaxWalks = 160;
struct Desc {
  uint32_t held[kMaxWalks / 32];  // bit k: the walk's k-th CTA from here on
  int parts;                      // CTAs it may be spread over (0: no cut item)
  int b, h, r0, rows, t0;
};

// The parts of one CTA: per part m, l and O as [2 + DPAD][256 rows], so that a
// warp's rows lie side by side.  Part 0 is of an item that began in an earlier
// CTA, part 1 of one that begins here.
constexpr int kPartRows = 256;
template <int DPAD>
__host__ __device__ constexpr size_t part_floats() {
  return static_cast<size_t>(kPartRows) * (DPAD + 2);
}
constexpr size_t kDescBytes = 64 * 1024;  // start of the scratch

struct TcArgs {
  sv_attention_t a;
  float *scratch;
  int *status;
  uint64_t wait_limit_ns;
  uint64_t by_walks;  // 2^64 / walks
  uint32_t by_group;  // 2^32 / G, rounded up (0: G is 1)
  float c;       // |scale| log2 e, kept above zero
  int negate;    // scale < 0: the queries are negated
  int pow_page;  // log2 of the page size
  int side;      // cache heads walked side by side
  int walks;     // grid / side
  int paired;    // both 128-byte halves of a row come in one box
  int head2, head3;  // paired: a head's coordinates in dimensions 2 and 3
};

// `side` CTAs, for as many neighbouring cache heads, walk the same items and
// tiles at the same time, as the heads of a cached token lie side by side in
// the usual layout (256 bytes each).  The walk's units are cut into equal runs
// (any monotone rule will do, so this one takes no division), but of two units
// at least: the two slots take two narrow tiles in the time of one, and each
// run more is a part to be joined.
__device__ __forceinline__ int64_t cut_at(const TcArgs &args, int64_t total, int c) {
  if (total < 2 * args.walks) return 2 * c < total ? 2 * c : total;
  return c >= args.walks ? total
                         : static_cast<int64_t>(__umul64hi(total, args.by_walks * c));
}

// r / G for a row.
__device__ __forceinline__ int group_div(const TcArgs &args, int G, int r) {
  if (!args.by_group) return r;
  const int q = static_cast<int>(__umulhi(static_cast<uint32_t>(r), args.by_group));
  return q * G > r ? q - 1 : q;  // the reciprocal is rounded up: at most one too many
}

constexpr int kFewItems = 4;  // items of a sequence that one lane counts by itself

// Walks the items of every side-th cache head (h counts those) from a unit on.
// Divisions and long arithmetic are kept out: the first tile waits for this.
struct Items {
  const TcArgs &args;
  const sv_attention_t &a;
  int G, heads;
  SeqGeom s;
  int b, h, m, nm;
  int64_t ub;  // first unit of the current item
  int shift;   // 0: narrow, a tile is one unit; 1: wide, two
  int ntiles, tile_lo, r0, rows;

  __device__ explicit Items(const TcArgs &t)
      : args(t), a(t.a), G(t.a.Hq / t.a.Hkv), heads(t.a.Hkv / t.side) {}

  __device__ void sequence() {
    const int total = s.n * G;
    nm = total > kRows ? (total + 2 * kRows - 1) / (2 * kRows) : 1;
  }
  __device__ void item() {
    const int total = s.n * G;
    r0 = m * (2 * kRows);
    rows = nm == 1 ? total : min(2 * kRows, total - r0);
    shift = rows > kRows ? 1 : 0;
    int lo, hi, x;
    key_range(a, s, nm == 1 ? 0 : group_div(args, G, r0), lo, x);
    key_range(a, s, nm == 1 ? s.n - 1 : group_div(args, G, r0 + rows - 1), x, hi);
    const int bits = shift ? 7 : 6;
    static_assert(kWideKeys == 128 && kNarrowKeys == 64, "bits");
    tile_lo = lo >> bits;
    ntiles = max(1, ((hi + (1 << bits) - 1) >> bits) - tile_lo);
  }
  __device__ int64_t units() const { return static_cast<int64_t>(ntiles) << shift; }

  // Units of one cache head of each lane's sequence (whole warp; n may be 0).
  __device__ int64_t head_units(int lane) {
    int64_t u = 0;
    sequence();
    if (s.n > 0 && nm <= kFewItems) {
      for (m = 0; m < nm; ++m) {
        item();
        u += units();
      }
    }
    // sequences of many items: the warp takes one at a time, an item a lane
    const SeqGeom mine = s;
    unsigned many = __ballot_sync(0xffffffffu, s.n > 0 && nm > kFewItems);
    while (many) {
      const int src = __ffs(many) - 1;
      many &= many - 1;
      s.t0 = __shfl_sync(0xffffffffu, mine.t0, src);
      s.n = __shfl_sync(0xffffffffu, mine.n, src);
      s.kv = __shfl_sync(0xffffffffu, mine.kv, src);
      s.ctx = __shfl_sync(0xffffffffu, mine.ctx, src);
      sequence();
      int64_t sum = 0;
      for (m = lane; m < nm; m += 32) {
        item();
        sum += units();
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      if (lane == src) u = sum;
    }
    s = mine;
    return u;
  }
  // To the item of sequence b (s is set, `per` units a head) that holds its unit
  // `off`, which is unit u of the walk.
  __device__ void seek(int64_t per, int64_t off, int64_t u, int lane) {
    sequence();
    h = 0;
    if (off >= 16 * per) {
      h = static_cast<int>(off / per);
      off -= h * per;
    }
    for (; off >= per; ++h) off -= per;
    if (nm <= kFewItems) {
      for (m = 0; m + 1 < nm; ++m) {
        item();
        if (off < units()) break;
        off -= units();
      }
    }
    for (int m0 = 0; nm > kFewItems && m0 < nm; m0 += 32) {
      m = m0 + lane;
      int64_t mine = 0;
      if (m < nm) {
        item();
        mine = units();
      }
      int64_t incl = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
      }
      const unsigned here = __ballot_sync(0xffffffffu, off < incl);
      if (here) {
        const int src = __ffs(here) - 1;
        off -= __shfl_sync(0xffffffffu, incl - mine, src);
        m = m0 + src;
        break;
      }
      off -= __shfl_sync(0xffffffffu, incl, 31);
    }
    item();
    ub = u - off;
  }
  // The next item; its units follow the current ones.  False: none left.
  __device__ bool next() {
    ub += units();
    if (++m == nm) {
      m = 0;
      if (++h == heads) {
        h = 0;
        do {
          if (++b >= a.B) return false;
          bool bad;
          s = seq_geom(a, b, &bad);
        } while (s.n == 0);
        sequence();
      }
    }
    item();
    return true;
  }
};

// The tiles of an item in the units [u0, u1).
__device__ __forceinline__ void tile_run(int64_t ub, int shift, int ntiles, int64_t u0, int64_t u1,
                                         int &tb, int &te) {
  const int64_t lo = u0 > ub ? (u0 - ub + shift) >> shift : 0;
  const int64_t hi = u1 > ub ? (u1 - ub + shift) >> shift : 0;
  tb = static_cast<int>(lo < ntiles ? lo : ntiles);
  te = static_cast<int>(hi < ntiles ? hi : ntiles);
}

// Whether a waiting warp has to give up: its limit ran out, or another role
// gave up.  A softmax warp in attend_row holds the others up for as long as it
// takes, so the limit starts over then.
__device__ __noinline__ bool give_up(Ctl *ctl, uint64_t &since, uint64_t limit_ns, int *status) {
  const volatile int *abort = &ctl->abort, *slow = &ctl->slow;
  const uint64_t now = globaltimer();
  if (since == 0 || *slow > 0) since = now;
  const bool out = now - since >= limit_ns;
  if (!__any_sync(0xffffffffu, out || *abort)) return false;
  if ((threadIdx.x & 31) == 0) {
    *reinterpret_cast<volatile int *>(&ctl->abort) = 1;
    set_status(status, SV_ERR_TIMEOUT);
  }
  __syncwarp();
  return true;
}
// Waits on a barrier with the whole warp; false: given up.  Few instructions
// where the barrier is ready, as the warp that issues the products pays for
// each (about 5 cycles).
__device__ __forceinline__ bool wait_warp(Ctl *ctl, uint64_t *bar, uint32_t parity,
                                          uint64_t limit_ns, int *status) {
  const uint32_t at = smem_u32(bar);
  if (__all_sync(0xffffffffu, mbar_try_wait(at, parity))) return true;
  uint64_t since = 0;
  while (true) {
    for (int i = 0; i < 16; ++i)
      if (__all_sync(0xffffffffu, mbar_try_wait(at, parity))) return true;
    if (give_up(ctl, since, limit_ns, status)) return false;
  }
}

// 32 bits of a tree row from bit s on (s may be negative): the context before
// the new tokens is seen, what lies past the words is not.
__device__ __forceinline__ uint32_t tree_bits(const int32_t *row, int words, int s) {
  const int w = s >> 5;
  auto word = [&](int i) {
    return i < 0 ? 0xffffffffu : i < words ? static_cast<uint32_t>(__ldg(row + i)) : 0u;
  };
  return __funnelshift_r(word(w), word(w + 1), s & 31);
}
// Whether a row of the run's item sees a key of [k0, k1).
__device__ __forceinline__ bool item_sees(const TcArgs &args, const Run &it, int k0, int k1) {
  const sv_attention_t &a = args.a;
  const int G = a.Hq / a.Hkv;
  const int first = group_div(args, G, it.r0), last = group_div(args, G, it.r0 + it.rows - 1);
  int lo, hi, x;
  key_range(a, it.s, first, lo, x);
  key_range(a, it.s, last, x, hi);
  k0 = max(k0, lo);
  k1 = min(k1, hi);
  if (k0 >= k1) return false;
  if (!a.tree_mask || k0 < it.s.ctx) return true;
  for (int i = first; i <= last; ++i) {
    const int32_t *row = a.tree_mask + static_cast<int64_t>(it.s.t0 + i) * a.tree_words;
    for (int k = k0; k < k1; ++k)
      if (tree_sees(row, a.tree_words, k - it.s.ctx)) return true;
  }
  return false;
}
// Reports pages outside the cache among those of a run's tiles t .. last, the ones that
// this lane brings (keys key_in .. key_in + page_keys - 1 of a tile of `keys`).  Only
// where a row sees a key of them, as tiles and pages reach beyond what is seen:
// below a window, and to new tokens that no row of a tree has its bit for.  Asked
// after a run that met such a page: in the loop over the tiles it cost a chunk of
// 4096 tokens 684 us against 677 and a round of 5 tokens 14.8 against 14.4 (single
// calls; here 680 and 14.5), and a scan of whole runs 64 windows of 4000 over freed
// pages of 8 179 us against 172.
__device__ __forceinline__ void report_pages(const TcArgs &args, const Run &it, int t, int last,
                                             int keys, int key_in, int page_keys) {
  const sv_attention_t &a = args.a;
  const int32_t *pages = a.page_table + it.b * a.table_stride;
  for (; t <= last; ++t) {
    const int key = (it.tile0 + t) * keys + key_in;
    if (static_cast<uint32_t>(pages[key >> args.pow_page]) >= a.num_pages &&
        item_sees(args, it, key, key + page_keys)) {
      set_status(args.status, SV_ERR_CACHE);
      return;
    }
  }
}
// Bits i of [lo, hi) of a group of 32 keys.
__device__ __forceinline__ uint32_t range_bits(int lo, int hi) {
  const uint32_t below = hi >= 32 ? 0xffffffffu : hi <= 0 ? 0u : (1u << hi) - 1u;
  const uint32_t under = lo >= 32 ? 0xffffffffu : lo <= 0 ? 0u : (1u << lo) - 1u;
  return below & ~under;
}

template <class T>
__device__ __forceinline__ uint32_t pack2(float lo, float hi);
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&v);
}
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&v);
}

__device__ __forceinline__ bool fast_output(const sv_attention_t &a) {
  return (reinterpret_cast<uintptr_t>(a.out) & 15u) == 0 && ((a.o_token | a.o_head) & 7) == 0;
}
// Stores N elements of a row of the output from d0 on; `fast`: 16-byte aligned
// rows.  D is a multiple of 8.
template <class T, int N = 32>
__device__ __forceinline__ void store_row(const sv_attention_t &a, T *o, int d0, const float *x,
                                          bool fast) {
  static_assert(N % 8 == 0, "16-byte stores");
#pragma unroll
  for (int v = 0; v < N; v += 8) {
    if (d0 + v >= a.D) break;
    if (fast) {
      uint4 q;
      q.x = pack2<T>(x[v], x[v + 1]);
      q.y = pack2<T>(x[v + 2], x[v + 3]);
      q.z = pack2<T>(x[v + 4], x[v + 5]);
      q.w = pack2<T>(x[v + 6], x[v + 7]);
      *reinterpret_cast<uint4 *>(o + d0 + v) = q;
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) o[d0 + v + e] = from_float<T>(x[v + e]);
    }
  }
}

template <class T, int DPAD>
__global__ void __launch_bounds__(kThreads, 1)
    attention_tc_kernel(const __grid_constant__ CUtensorMap tmK,
                        const __grid_constant__ CUtensorMap tmV,
                        const __grid_constant__ TcArgs args) {
  using Sh = Shape<DPAD>;
  constexpr bool kBf16 = sizeof(T) == 2 && !__is_same(T, __half);
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t *smem = smem_raw + (base - raw);
  Ctl *ctl = reinterpret_cast<Ctl *>(smem + 2 * Sh::kQBytes + kRingBytes);
  const uint32_t ring = base + 2 * Sh::kQBytes;
  const sv_attention_t &a = args.a;
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // uniform to the compiler
  Desc *desc = reinterpret_cast<Desc *>(args.scratch) + blockIdx.x;
  float *parts = args.scratch + kDescBytes / 4;

  if (tid == 0) {
    for (int i = 0; i < Sh::kSlots; ++i) {
      mbar_init(smem_u32(&ctl->full[i]), 2);
      mbar_init(smem_u32(&ctl->empty[i]), 1);
    }
    for (int i = 0; i < kRuns; ++i) {
      mbar_init(smem_u32(&ctl->run_full[i]), 1);
      mbar_init(smem_u32(&ctl->run_empty[i]), kSoftmaxWarps + 3);
    }
    mbar_init(smem_u32(&ctl->q_ready), kSoftmaxWarps);
    for (int w = 0; w < 2; ++w) {
      mbar_init(smem_u32(&ctl->s_full[w]), 1);
      mbar_init(smem_u32(&ctl->p_ready[w]), kSoftmaxWarps / 2);
    }
    mbar_init(smem_u32(&ctl->o_full), 1);
    mbar_init(smem_u32(&ctl->x_full), kSoftmaxWarps / 2);
    mbar_init(smem_u32(&ctl->x_free), kSoftmaxWarps / 2);
    mbar_init(smem_u32(&ctl->teardown), 1);
    ctl->abort = ctl->slow = ctl->issued[0] = ctl->issued[1] = ctl->consumed = 0;
    ctl->start_b = -1;
    mbar_fence_init();
  }
  if (warp == 8 && lane == 0) {
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  if (warp == 9) {
    tmem_alloc(smem_u32(&ctl->tmem), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, ctl->tmem, 0);
  pdl_wait();
  pdl_launch_dependents();

  // ---- this CTA's run of units ----
  // With up to 32 sequences the warp that hands out the items finds it alone;
  // with more the block does.
  const int walk = blockIdx.x / args.side;
  Items it(args);
  // units of sequence b (one a lane), and of one head of it
  auto sequence_units = [&](int b, int64_t &per) {
    bool bad = false;
    it.s = SeqGeom{0, 0, 0, 0};
    if (b < a.B) it.s = seq_geom(a, b, &bad);
    if (bad && blockIdx.x == 0) set_status(args.status, SV_ERR_CACHE);
    per = it.head_units(lane);
    return per * it.heads;
  };
  auto scan32 = [&](int64_t x) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    return x;
  };
  int64_t total = 0, u0 = 0, u1 = 0;
  if (a.B > 32) {
    int64_t before = 0, per;
    for (int pass = 0; pass < 2; ++pass) {  // the total, then where u0 lies
      for (int b0 = 0; b0 < a.B; b0 += kThreads) {
        const int64_t u = sequence_units(b0 + tid, per);
        const int64_t incl = scan32(u);
        __syncthreads();  // the last sums have been read
        if (lane == 31) ctl->scan[warp] = incl;
        __syncthreads();
        int64_t pre = before;
        for (int i = 0; i < kThreads / 32; ++i) {
          if (i < warp) pre += ctl->scan[i];
          before += ctl->scan[i];
        }
        if (pass == 1 && u > 0 && u0 < u1 && u0 >= pre + incl - u && u0 < pre + incl) {
          ctl->start_b = b0 + tid;
          ctl->start_off = u0 - (pre + incl - u);
          ctl->start_per = per;
        }
      }
      if (pass == 0) {
        total = before;
        before = 0;
        u0 = cut_at(args, total, walk);
        u1 = cut_at(args, total, walk + 1);
      }
    }
    __syncthreads();
  }
  // The next item for a role's warp; false: none left, or the call is given up.
  int runs = 0;
  auto take = [&]() {
    const int i = runs % kRuns;
    if (!wait_warp(ctl, &ctl->run_full[i], (runs / kRuns) & 1, args.wait_limit_ns, args.status))
      return false;
    ++runs;
    return ctl->run[i].n > 0;
  };
  auto give_back = [&]() {
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&ctl->run_empty[(runs - 1) % kRuns]));
  };

  if (warp < kSoftmaxWarps) {
    // ---------------- softmax and output ----------------
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    const int w = warp >> 2;
    const int row = tid & 127;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + lanes + w * 128, tO = tmem + lanes + 256 + w * 128;
    const bool out_fast = fast_output(a);
    const int G = a.Hq / a.Hkv;
    int items = 0, cnt = 0, narrow = 0;
    bool ok = true;
    while (ok && take()) {
      const Run &it = ctl->run[(runs - 1) % kRuns];
      const int n = it.n;
      const bool wide = it.wide;
      // ---- this thread's row ----
      const int r = wide ? w * kRows + row : row;
      const bool valid = r < it.rows;
      const int tok = valid ? group_div(args, G, it.r0 + r) : 0;
      const int head = it.h * G + (it.r0 + r) - tok * G;
      const int64_t t = it.s.t0 + tok;
      int lo = 0, hi = 0;
      const int32_t *tree = nullptr;
      if (valid) {
        key_range(a, it.s, tok, lo, hi);
        if (a.tree_mask) tree = a.tree_mask + t * a.tree_words;
      }
      if (wide || w == 0) {
        const T *q = static_cast<const T *>(a.q) + t * a.q_token + head * a.q_head;
        uint8_t *dst = smem + (wide ? w : 0) * Sh::kQBytes + row * 128;
#pragma unroll
        for (int v = 0; v < DPAD / 8; ++v) {
          uint4 x = make_uint4(0, 0, 0, 0);
          if (valid && 8 * v < a.D) x = *reinterpret_cast<const uint4 *>(q + 8 * v);
          if (args.negate) {
            x.x ^= 0x80008000u;
            x.y ^= 0x80008000u;
            x.z ^= 0x80008000u;
            x.w ^= 0x80008000u;
          }
          *reinterpret_cast<uint4 *>(dst + (v / 8) * (kRows * 128) +
                                     (((v % 8) ^ (row & 7)) << 4)) = x;
        }
        fence_proxy_async_smem();
      }
      tc_fence_before();  // the last item's reads of O come before its products
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&ctl->q_ready));

      const bool live = __any_sync(0xffffffffu, valid);
      const int steps = wide ? n : (n + 1 - w) / 2;
      float m = -INFINITY, l = 0.0f;
      // One tile of NK keys for this warp's rows.
      auto tile = [&](auto nk, int k0, bool first) {
        constexpr int NK = decltype(nk)::value;
        uint32_t sr[NK];
#pragma unroll
        for (int g = 0; g < NK / 32; ++g) tmem_ld32(tS + 32 * g, sr + 32 * g);
        tmem_ld_wait();
#pragma unroll
        for (int g = 0; g < NK / 32; ++g) tmem_reg_fence32(sr + 32 * g);
        float *x = reinterpret_cast<float *>(sr);
        const bool whole =
            !valid || (lo <= k0 && hi >= k0 + NK && (!tree || k0 + NK <= it.s.ctx));
        if (!__all_sync(0xffffffffu, whole)) {
#pragma unroll
          for (int g = 0; g < NK / 32; ++g) {
            uint32_t keep = range_bits(lo - k0 - 32 * g, hi - k0 - 32 * g);
            if (tree) keep &= tree_bits(tree, a.tree_words, k0 + 32 * g - it.s.ctx);
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (!(keep & (1u << i))) x[32 * g + i] = -INFINITY;
          }
        }
        float top;
        {
          float t4[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) t4[i] = max3(x[i], x[i + 4], x[i + 8]);
#pragma unroll
          for (int g = 12; g + 8 <= NK; g += 8)
#pragma unroll
            for (int i = 0; i < 4; ++i) t4[i] = max3(t4[i], x[g + i], x[g + 4 + i]);
          constexpr int rest = 12 + (NK - 12) / 8 * 8;
#pragma unroll
          for (int i = rest; i < NK; ++i) t4[i & 3] = fmaxf(t4[i & 3], x[i]);
          top = fmaxf(max3(t4[0], t4[1], t4[2]), t4[3]);
        }
        const bool grow = m == -INFINITY ? top > -INFINITY : (top - m) * args.c > kRescale;
        if (__any_sync(0xffffffffu, grow)) {
          const float to = grow ? top : m;
          const float f = grow ? (m == -INFINITY ? 0.0f : ex2((m - to) * args.c)) : 1.0f;
          m = to;
          l *= f;
          if (!first) {
            // the products of the last step are complete: they precede the
            // scores of this one
#pragma unroll
            for (int g = 0; g < DPAD / 16; ++g) {
              uint32_t o[16];
              tmem_ld16(tO + 16 * g, o);
              tmem_ld_wait();
              tmem_reg_fence(o);
#pragma unroll
              for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
              tmem_st16(tO + 16 * g, o);
            }
          }
        }
        const float off = m == -INFINITY ? 0.0f : -m * args.c + carried<T>();
        const uint64_t c2 = pair2(args.c, args.c), off2 = pair2(off, off);
        uint64_t ls[2] = {0, 0};
#pragma unroll
        for (int g = 0; g < NK / 64; ++g) {
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            const int j = 64 * g + 2 * i;
            const float2 y = unpair2(fma2(pair2(x[j], x[j + 1]), c2, off2));
            const float p0 = ex2(y.x), p1 = ex2(y.y);
            ls[i & 1] = add2(ls[i & 1], pair2(p0, p1));
            sr[32 * g + i] = pack2<T>(p0, p1);
          }
          tmem_st32(tS + 32 * g, sr + 32 * g);
        }
        const float2 sum2 = unpair2(add2(ls[0], ls[1]));
        l += sum2.x + sum2.y;
        tmem_st_wait();
        tc_fence_before();
      };
      const int keys = wide ? kWideKeys : kNarrowKeys;
      for (int st = 0; st < steps; ++st) {
        const int k0 = (it.tile0 + (wide ? st : 2 * st + w)) * keys;
        if (!wait_warp(ctl, &ctl->s_full[w], cnt & 1, args.wait_limit_ns, args.status)) {
          ok = false;
          break;
        }
        ++cnt;
        tc_fence_after();
        if (live) {
          if (wide)
            tile(std::integral_constant<int, kWideKeys>{}, k0, st == 0);
          else
            tile(std::integral_constant<int, kNarrowKeys>{}, k0, st == 0);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&ctl->p_ready[w]));
      }
      if (!ok) break;
      if (!wait_warp(ctl, &ctl->o_full, items & 1, args.wait_limit_ns, args.status)) {
        ok = false;
        break;
      }
      ++items;
      tc_fence_after();

      // A NaN score is no maximum, so it may have left m at -inf; as the largest
      // of all it is not taken for "saw nothing" where parts are joined.
      if (l != l) m = INFINITY;

      // ---- the item's result, or this CTA's part of it ----
      float f0 = 1.0f, f1 = 0.0f;
      const bool join = !wide && n > 1;
      if (!wide) {
        // slot 1 hands its m and l to slot 0, which reads both outputs
        if (w == 1) {
          if (narrow > 0 && !(ok = wait_warp(ctl, &ctl->x_free, (narrow - 1) & 1,
                                             args.wait_limit_ns, args.status)))
            break;
          ctl->xm[row] = m;
          ctl->xl[row] = l;
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&ctl->x_full));
        } else {
          if (!(ok = wait_warp(ctl, &ctl->x_full, narrow & 1, args.wait_limit_ns, args.status)))
            break;
          const float m1 = ctl->xm[row], l1 = ctl->xl[row];
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&ctl->x_free));
          if (join) {
            const float to = fmaxf(m, m1);
            f0 = m == -INFINITY ? 0.0f : ex2((m - to) * args.c);
            f1 = m1 == -INFINITY ? 0.0f : ex2((m1 - to) * args.c);
            l = l * f0 + l1 * f1;
            m = to;
          }
        }
        ++narrow;
      }
      if ((wide || w == 0) && live) {
        const bool all = it.whole;
        float *part =
            parts + (static_cast<size_t>(blockIdx.x) * 2 + it.part) * part_floats<DPAD>();
        const float inv = l != 0.0f ? 1.0f / l : 0.0f;
        T *o = static_cast<T *>(a.out) + t * a.o_token + head * a.o_head;
        bool fine = true;
        // (written out once: code that runs once an item is not unrolled further)
#pragma unroll 1
        for (int g = 0; g < DPAD / 32; ++g) {
          uint32_t y[32], z[32];
          tmem_ld32(tO + 32 * g, y);
          if (join) tmem_ld32(tO + 128 + 32 * g, z);
          tmem_ld_wait();
          tmem_reg_fence32(y);
          tmem_reg_fence32(z);
          float *x = reinterpret_cast<float *>(y);
          if (join) {
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              // a slot that saw nothing has nothing to add
              x[i] = f0 != 0.0f ? x[i] * f0 : 0.0f;
              if (f1 != 0.0f) x[i] = fmaf(__uint_as_float(z[i]), f1, x[i]);
            }
          }
          if (all) {
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              x[i] = l != 0.0f ? x[i] * inv : 0.0f;
              fine &= fabsf(x[i]) < INFINITY;
            }
            if (valid) store_row<T>(a, o, 32 * g, x, out_fast);
          } else if (valid) {
#pragma unroll
            for (int i = 0; i < 32; ++i) part[(2 + 32 * g + i) * kPartRows + r] = x[i];
          }
        }
        if (valid) {
          if (all) {
            if (a.lse)
              a.lse[t * a.Hq + head] =
                  l != 0.0f ? m * (args.c * kLn2) + (logf(l) - carried<T>() * kLn2) : -INFINITY;
          } else {
            part[r] = m;
            part[kPartRows + r] = l;
          }
        }
        unsigned again = __ballot_sync(0xffffffffu, all && valid && !fine);
        if (again) {
          if (lane == 0) atomicAdd(&ctl->slow, 1);
          __syncwarp();
          while (again) {
            const int src = __ffs(again) - 1;
            again &= again - 1;
            attend_row<T>(a, it.s, it.b, __shfl_sync(0xffffffffu, tok, src),
                          __shfl_sync(0xffffffffu, head, src), lane, args.status);
          }
          __syncwarp();
          if (lane == 0) atomicSub(&ctl->slow, 1);
        }
      }
      give_back();
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp == 10) {
      // ---------------- items ----------------
      if (lane == 0) desc->parts = 0;
      bool more = false;
      if (a.B > 32) {
        it.b = ctl->start_b;
        more = it.b >= 0;
        if (more) {
          bool bad;
          it.s = seq_geom(a, it.b, &bad);
          it.seek(ctl->start_per, ctl->start_off, u0, lane);
        }
      } else {
        int64_t per;
        const int64_t u = sequence_units(lane, per), incl = scan32(u);
        total = __shfl_sync(0xffffffffu, incl, 31);
        u0 = cut_at(args, total, walk);
        u1 = cut_at(args, total, walk + 1);
        const unsigned here = __ballot_sync(0xffffffffu, u0 < u1 && u0 < incl);
        more = here != 0;
        if (more) {
          const int src = __ffs(here) - 1;
          it.b = src;
          it.s.t0 = __shfl_sync(0xffffffffu, it.s.t0, src);
          it.s.n = __shfl_sync(0xffffffffu, it.s.n, src);
          it.s.kv = __shfl_sync(0xffffffffu, it.s.kv, src);
          it.s.ctx = __shfl_sync(0xffffffffu, it.s.ctx, src);
          it.seek(__shfl_sync(0xffffffffu, per, src),
                  u0 - __shfl_sync(0xffffffffu, incl - u, src), u0, lane);
        }
      }
      while (true) {
        Run r{};
        int tb, te;
        for (; more && it.ub < u1; more = it.next()) {
          tile_run(it.ub, it.shift, it.ntiles, u0, u1, tb, te);
          if (te > tb) {
            r.n = te - tb;
            r.tile0 = it.tile_lo + tb;
            r.wide = it.shift;
            r.whole = tb == 0 && te == it.ntiles;
            r.once = it.nm <= 2;
            r.part = tb > 0 ? 0 : 1;
            r.b = it.b;
            r.h = it.h * args.side + blockIdx.x % args.side;
            r.r0 = it.r0;
            r.rows = it.rows;
            r.s = it.s;
            break;
          }
        }
        const int i = runs % kRuns;
        if (!wait_warp(ctl, &ctl->run_empty[i], ((runs / kRuns) & 1) ^ 1, args.wait_limit_ns,
                       args.status))
          break;
        if (lane == 0) {
          ctl->run[i] = r;
          mbar_arrive(smem_u32(&ctl->run_full[i]));
        }
        __syncwarp();
        ++runs;
        if (r.n == 0) break;
        // the others are at work: what the join needs, and the next item
        if (!r.whole && r.part == 1) {
          // the CTAs of the walk from here on that hold tiles of it
          const int64_t ue = it.ub + it.units();
          int n = 0;
          for (int k0 = 0;; k0 += 32) {
            const int c = walk + k0 + lane;
            const int64_t c0 = cut_at(args, total, c);
            int kb, ke;
            tile_run(it.ub, it.shift, it.ntiles, c0, cut_at(args, total, c + 1), kb, ke);
            const unsigned held = __ballot_sync(0xffffffffu, c < args.walks && kb < ke);
            if (lane == 0) desc->held[k0 / 32] = held;
            if (held) n = k0 + 32 - __clz(held);
            // (the last lane's next CTA is the next round's first)
            if (!__all_sync(0xffffffffu, c + 1 < args.walks && c0 < ue)) break;
          }
          if (lane == 0) {
            desc->b = r.b;
            desc->h = r.h;
            desc->r0 = r.r0;
            desc->rows = r.rows;
            desc->t0 = r.s.t0;
            desc->parts = n;
          }
        }
        more = it.next();
      }
    } else if (warp == 8 || warp == 11) {
      // ---------------- TMA ----------------
      // Warp 8 brings K, warp 11 a narrow tile's V (64 single tokens over 8192 in
      // pages of 8: 208 us against 249 by one warp; heads of 64 in pages of 16: 145
      // against 166).  A wide tile has twice the time: its V comes by warp 8 too
      // (a chunk 1% slower by two).
      const int v = warp == 8 ? 0 : 1;
      const int page_keys = min(64, a.page_size);
      const bool paired = Sh::kSlabs > 1 && args.paired;
      const uint32_t box_bytes =
          static_cast<uint32_t>(page_keys) * (paired ? 128u * Sh::kSlabs : 128u);
      int slot = 0, issued = 0;
      uint32_t phase = 0;
      bool ok = true;
      // Both warps wait for every slot and arrive at every slot, their own or not:
      // it is full only after both, so neither is ever a whole round of the ring
      // behind, where a wait by parity would take one round for another.
      auto slot_free = [&]() {
        return ok = wait_warp(ctl, &ctl->empty[slot], phase ^ 1, args.wait_limit_ns, args.status);
      };
      auto next_slot = [&]() {
        ++issued;
        if (++slot == Sh::kSlots) {
          slot = 0;
          phase ^= 1;
        }
      };
      while (ok && take()) {
        const Run &it = ctl->run[(runs - 1) % kRuns];
        const int n = it.n, tile0 = it.tile0, kv = it.s.kv, head = it.h;
        const bool wide = it.wide;
        const bool brings = !(wide && v);  // a wide tile's V comes by warp 8
        // K and V that are not read again need not stay in L2: 64 single tokens
        // over 8192 in 247 us against 253, eight trees of 65 in 62 against 68; a
        // prompt's chunk, which comes back to them, in 723 against 653
        const uint64_t policy = it.once ? policy_evict_first() : policy_evict_normal();
        const int keys = wide ? kWideKeys : kNarrowKeys;
        const int32_t *pages = a.page_table + it.b * a.table_stride;
        // lane i brings box i of a tile: box i / slabs of its keys, slab i %
        // slabs (at most 32 boxes, as a page holds 8 keys or more); paired: all
        // slabs of box i
        const int each = paired ? 1 : Sh::kSlabs;
        const int slab = lane % each, key_in = lane / each * page_keys;
        const uint32_t offset =
            static_cast<uint32_t>(slab * keys * 128 + key_in * (paired ? 128 * Sh::kSlabs : 128));
        const int head2 = head * args.head2, head3 = head * args.head3;
        auto page_of = [&](int t) {
          const int key = (tile0 + t) * keys + key_in;
          return brings && t < n && key_in < keys && key < kv ? pages[key >> args.pow_page] : 0;
        };
        int page = page_of(0);
        // tiles with a page that is not there (which is loaded as zeros): the first
        // and the last, for the lane
        int miss0 = n, miss1 = -1;
        for (int t = 0; t < n && ok; ++t) {
          const int next = page_of(t + 1);
          const int k0 = (tile0 + t) * keys;
          const bool mine = key_in < keys && k0 + key_in < kv;
          const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, mine)) * box_bytes;
          if (mine && static_cast<uint32_t>(page) >= a.num_pages) {
            miss0 = min(miss0, t);
            miss1 = t;
          }
          const int in_page = (k0 + key_in) & (a.page_size - 1);
          for (int x = 0; x < (wide ? 2 : 1); ++x) {
            if (!slot_free()) break;
            const uint32_t full = smem_u32(&ctl->full[slot]);
            const bool second = wide ? x == 1 : v == 1;  // V, not K
            const CUtensorMap *map = second ? &tmV : &tmK;
            if (lane == 0) {
              if (brings)
                mbar_arrive_expect_tx(full, bytes);
              else
                mbar_arrive(full);
            }
            __syncwarp();
            const uint32_t at =
                ring + slot * Sh::kSlotBytes + offset + (wide || !v ? 0 : Sh::kSlotBytes / 2);
            if (mine && brings) {
              if (paired)
                tma_load_5d(at, map, 0, 0, head2, head3 + (in_page >> 3), page, full, policy);
              else
                tma_load_4d(at, map, slab * 64, head, in_page, page, full, policy);
            }
            __syncwarp();
            next_slot();
          }
          page = next;
        }
        if (miss0 <= miss1) report_pages(args, it, miss0, miss1, keys, key_in, page_keys);
        give_back();
      }
      if (lane == 0) ctl->issued[v] = issued;
    } else if (warp == 9) {
      // ---------------- products ----------------
      constexpr uint32_t idesc_o = idesc_16(kBf16, kRows, DPAD, true);
      int slot = 0, consumed = 0;
      uint32_t phase = 0, q_phase = 0, p_phase = 0;
      bool ok = true;
      // the next slot of the ring, once it is full; -1: given up
      auto next_slot = [&]() {
        if (!wait_warp(ctl, &ctl->full[slot], phase, args.wait_limit_ns, args.status)) return -1;
        const int s = slot;
        ++consumed;
        if (++slot == Sh::kSlots) {
          slot = 0;
          phase ^= 1;
        }
        return s;
      };
      // Both of a slot's weights flip together with p_phase's bits.
      auto wait_p = [&](int w) {
        const bool r = wait_warp(ctl, &ctl->p_ready[w], (p_phase >> w) & 1, args.wait_limit_ns,
                                 args.status);
        p_phase ^= 1u << w;
        tc_fence_after();
        return r;
      };
      // Bytes between the groups of eight keys of a tile, and between its slabs
      // (of `keys` keys); in the layout of paired boxes a group's slabs are
      // neighbours.
      const bool paired = Sh::kSlabs > 1 && args.paired;
      const uint32_t group_bytes = paired ? 1024 * Sh::kSlabs : 1024;
      auto slab_bytes = [&](int keys) { return static_cast<uint32_t>(paired ? 1024 : keys * 128); };
      const uint64_t q0 = sw128_desc(base);
      const uint64_t k_base =
          sw128_desc(ring) + (static_cast<uint64_t>((group_bytes - 1024) >> 4) << 32);
      constexpr uint32_t kSlot16 = Sh::kSlotBytes >> 4, kQ16 = Sh::kQBytes >> 4;
      // S of slot w: `keys` keys from ring slot s on; then commits s_full and,
      // if `last`, frees the slot
      auto scores = [&](int w, uint64_t q, int s, auto keys, bool last) {
        const uint32_t slab16 = slab_bytes(keys) >> 4;
        constexpr uint32_t idesc = idesc_16(kBf16, kRows, keys, false);
        const uint64_t k = k_base + static_cast<uint32_t>(s) * kSlot16;
        if (elect_one()) {
#pragma unroll
          for (int e = 0; e < DPAD / 16; ++e)
            umma_16(tmem + w * 128, q + (e / 4) * (kRows * 128 >> 4) + 2 * (e % 4),
                    k + (e / 4) * slab16 + 2 * (e % 4), idesc, e > 0);
          umma_commit(smem_u32(&ctl->s_full[w]));
          if (last) umma_commit(smem_u32(&ctl->empty[s]));
        }
        __syncwarp();
      };
      // O of slot w += P V, V at `at` in the ring, 16 keys a product
      auto outputs = [&](int w, uint32_t at, int s, auto keys, bool more, bool last) {
        const uint64_t v = sw128_desc_mn(at, slab_bytes(keys), group_bytes);
        if (elect_one()) {
#pragma unroll
          for (int e = 0; e < keys / 16; ++e)
            umma_16_ta(tmem + 256 + w * 128, tmem + w * 128 + e * 8,
                       v + e * (2 * group_bytes >> 4), idesc_o, more || e > 0);
          if (last) umma_commit(smem_u32(&ctl->empty[s]));
        }
        __syncwarp();
      };
      // Rows of V past the sequence hold anything: they get weight zero, which
      // has to give zero.
      auto zero_tail = [&](uint32_t at, int live, int keys) {
        uint8_t *v = smem + (at - base);
        for (int x = max(live, 0) * 8 + lane; x < keys * 8; x += 32) {
          const int key = x >> 3;
          uint8_t *at_key = v + (key >> 3) * group_bytes + (key & 7) * 128 + (x & 7) * 16;
#pragma unroll
          for (int slab = 0; slab < Sh::kSlabs; ++slab)
            *reinterpret_cast<uint4 *>(at_key + slab * slab_bytes(keys)) = make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async_smem();
        __syncwarp();
      };
      constexpr std::integral_constant<int, kWideKeys> wide_keys{};
      constexpr std::integral_constant<int, kNarrowKeys> narrow_keys{};
      while (ok && take()) {
        const Run &it = ctl->run[(runs - 1) % kRuns];
        const int n = __shfl_sync(0xffffffffu, it.n, 0);
        const int live = __shfl_sync(0xffffffffu, it.s.kv, 0) -
                         __shfl_sync(0xffffffffu, it.tile0, 0) * (it.wide ? kWideKeys
                                                                          : kNarrowKeys);
        if (!(ok = wait_warp(ctl, &ctl->q_ready, q_phase, args.wait_limit_ns, args.status))) break;
        q_phase ^= 1;
        int s = next_slot();
        ok = s >= 0;
        if (!ok) break;
        tc_fence_after();
        if (__shfl_sync(0xffffffffu, it.wide, 0)) {
          scores(0, q0, s, wide_keys, false);
          scores(1, q0 + kQ16, s, wide_keys, true);
          for (int t = 0; t < n; ++t) {
            const int v = next_slot();
            ok = v >= 0;
            if (!ok) break;
            const uint32_t at = ring + v * Sh::kSlotBytes;
            if (live < (t + 1) * kWideKeys) zero_tail(at, live - t * kWideKeys, kWideKeys);
            if (!(ok = wait_p(0))) break;
            outputs(0, at, v, wide_keys, t > 0, false);
            if (t + 1 < n) {
              s = next_slot();
              ok = s >= 0;
              if (!ok) break;
              tc_fence_after();
              scores(0, q0, s, wide_keys, false);
            }
            if (!(ok = wait_p(1))) break;
            outputs(1, at, v, wide_keys, t > 0, true);
            if (t + 1 < n) scores(1, q0 + kQ16, s, wide_keys, true);
          }
        } else {
          scores(0, q0, s, narrow_keys, false);
          int s1 = s;
          if (n > 1) {
            s1 = next_slot();
            ok = s1 >= 0;
            if (!ok) break;
            tc_fence_after();
            scores(1, q0, s1, narrow_keys, false);
          }
          for (int t = 0; t < n; ++t) {
            const int w = t & 1, v = s;
            const uint32_t at = ring + v * Sh::kSlotBytes + Sh::kSlotBytes / 2;
            if (live < (t + 1) * kNarrowKeys) zero_tail(at, live - t * kNarrowKeys, kNarrowKeys);
            if (!(ok = wait_p(w))) break;
            outputs(w, at, v, narrow_keys, t > 1, true);
            s = s1;
            if (t + 2 < n) {
              s1 = next_slot();
              ok = s1 >= 0;
            if (!ok) break;
              tc_fence_after();
              scores(w, q0, s1, narrow_keys, false);
            }
          }
        }
        if (!ok) break;
        if (elect_one()) umma_commit(smem_u32(&ctl->o_full));
        give_back();
      }
      if (lane == 0) ctl->consumed = consumed;
      if (elect_one()) {
        umma_commit(smem_u32(&ctl->teardown));
        const int never = 0;
        mbar_wait(smem_u32(&ctl->teardown), 0u, kCleanupLimitNs, &never);
      }
      __syncwarp();
    }
  }

  // ---------------- teardown ----------------
  tc_fence_before();
  __syncthreads();
  if (warp == 8 && lane == 0) {
    // only after an abort can copies still be in flight (and a slot may then
    // have its K or its V alone, for which one limit is waited)
    const int never = 0;
    const int issued = max(ctl->issued[0], ctl->issued[1]);
    for (int p = ctl->consumed; p < issued; ++p)
      if (!mbar_wait(smem_u32(&ctl->full[p % Sh::kSlots]),
                     static_cast<uint32_t>((p / Sh::kSlots) & 1), kCleanupLimitNs, &never))
        break;
  }
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Joins the parts of the items that were cut, in their order (a part of 256 rows
// is 133 KB, so this is a pass over at most 40 MB in L2; alone and with cold
// caches 5.5 us for 64 single tokens, 12 for eight trees of 65).  A warp takes 32
// rows, one a lane, and eight elements of the head; block (c, y) works on the
// item that begins in CTA c.
constexpr int kJoinWarps = 8, kJoinElems = 8, kJoinParts = 4;
template <class T, int DPAD>
__global__ void __launch_bounds__(32 * kJoinWarps)
    attention_join_kernel(const __grid_constant__ TcArgs args) {
  const sv_attention_t &a = args.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_wait();
  pdl_launch_dependents();
  const Desc &d = reinterpret_cast<const Desc *>(args.scratch)[blockIdx.x];
  const int count = d.parts;
  if (count == 0) return;
  const int rows = d.rows, G = a.Hq / a.Hkv;
  const size_t pitch = 2 * part_floats<DPAD>() * args.side;  // from CTA to CTA of the walk
  const float *parts = args.scratch + kDescBytes / 4 +
                       blockIdx.x * (2 * part_floats<DPAD>());
  auto part_of = [&](int k) { return parts + k * pitch + (k > 0 ? 0 : part_floats<DPAD>()); };
  uint32_t held[kMaxWalks / 32];
#pragma unroll
  for (int i = 0; i < kMaxWalks / 32; ++i) held[i] = 32 * i < count ? d.held[i] : 0u;
  const int b = d.b, h = d.h, r0 = d.r0, t0 = d.t0;
  constexpr int kGroups = DPAD / kJoinElems;
  const int tasks = (rows + 31) / 32 * kGroups;
  for (int i = blockIdx.y * kJoinWarps + warp; i < tasks; i += gridDim.y * kJoinWarps) {
    const int r = i / kGroups * 32 + lane, d0 = i % kGroups * kJoinElems;
    if (d0 >= a.D) continue;
    const bool valid = r < rows;
    const int row = valid ? r : 0;
    float top = -INFINITY, sum = 0.0f, acc[kJoinElems] = {};
    for (int k0 = 0; k0 < count; k0 += kJoinParts) {
      // all of the round's loads first: the parts were written by other SMs
      float m[kJoinParts], l[kJoinParts], x[kJoinParts][kJoinElems];
      uint32_t word = held[0];
#pragma unroll
      for (int i = 1; i < kMaxWalks / 32; ++i)
        if (k0 >= 32 * i) word = held[i];
      word >>= k0 & 31;
#pragma unroll
      for (int j = 0; j < kJoinParts; ++j) {
        const float *p = part_of(min(k0 + j, count - 1)) + row;
        m[j] = __ldcg(p);
        l[j] = __ldcg(p + kPartRows);
#pragma unroll
        for (int e = 0; e < kJoinElems; ++e) x[j][e] = __ldcg(p + (2 + d0 + e) * kPartRows);
      }
      float to = top;
#pragma unroll
      for (int j = 0; j < kJoinParts; ++j) {
        if (!((word >> j) & 1u)) m[j] = -INFINITY;  // none there
        to = fmaxf(to, m[j]);
      }
      const float keep = top == -INFINITY ? 0.0f : ex2((top - to) * args.c);
      sum *= keep;
#pragma unroll
      for (int e = 0; e < kJoinElems; ++e) acc[e] = keep != 0.0f ? acc[e] * keep : 0.0f;
      top = to;
#pragma unroll
      for (int j = 0; j < kJoinParts; ++j) {
        // a part that saw nothing adds nothing
        const float f = m[j] == -INFINITY ? 0.0f : ex2((m[j] - top) * args.c);
        sum = f != 0.0f ? fmaf(l[j], f, sum) : sum;
#pragma unroll
        for (int e = 0; e < kJoinElems; ++e)
          acc[e] = f != 0.0f ? fmaf(x[j][e], f, acc[e]) : acc[e];
      }
    }
    const int tok = valid ? group_div(args, G, r0 + r) : 0;
    const int head = h * G + r0 + r - tok * G;
    const int64_t t = t0 + tok;
    bool fine = true;
    if (valid) {
      const float inv = sum != 0.0f ? 1.0f / sum : 0.0f;
#pragma unroll
      for (int e = 0; e < kJoinElems; ++e) {
        acc[e] = sum != 0.0f ? acc[e] * inv : 0.0f;
        fine &= fabsf(acc[e]) < INFINITY;
      }
      if (fine) {
        store_row<T, kJoinElems>(a, static_cast<T *>(a.out) + t * a.o_token + head * a.o_head,
                                 d0, acc, fast_output(a));
        if (a.lse && d0 == 0)
          a.lse[t * a.Hq + head] =
              sum != 0.0f ? top * (args.c * kLn2) + (logf(sum) - carried<T>() * kLn2) : -INFINITY;
      }
    }
    // Other warps, at any time, have the row's other elements: this one takes
    // its own again and no more.
    unsigned again = __ballot_sync(0xffffffffu, !fine);
    if (again) {
      bool bad;
      const SeqGeom s = seq_geom(a, b, &bad);
      while (again) {
        const int src = __ffs(again) - 1;
        again &= again - 1;
        attend_row<T>(a, s, b, __shfl_sync(0xffffffffu, tok, src),
                      __shfl_sync(0xffffffffu, head, src), lane, args.status, d0,
                      d0 + kJoinElems);
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void *p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  }();
  return fn;
}

// The cache as a tensor map.  A box is 64 columns (128 bytes) of up to 64
// tokens of one page and head, or, paired, both halves of their rows: columns,
// tokens of a group of eight, halves, groups, page, where heads share a
// dimension with the halves (head2 = 2: a token's heads lie side by side) or
// with the groups (head3: a head's tokens lie side by side).
bool encode_cache(CUtensorMap *map, const TcArgs &args, const void *base, int64_t page,
                  int64_t token, int64_t head) {
  const sv_attention_t &a = args.a;
  const cuuint32_t keys = a.page_size < 64 ? a.page_size : 64;
  auto bytes = [](int64_t elements) { return static_cast<cuuint64_t>(elements) * 2; };
  const cuuint64_t heads = static_cast<cuuint64_t>(a.Hkv);
  const cuuint64_t groups = static_cast<cuuint64_t>(a.page_size / 8);
  const cuuint64_t pages = static_cast<cuuint64_t>(a.num_pages);
  const cuuint64_t dims4[4] = {static_cast<cuuint64_t>(a.D), heads,
                               static_cast<cuuint64_t>(a.page_size), pages};
  const cuuint64_t strides4[3] = {bytes(head), bytes(token), bytes(page)};
  const cuuint32_t box4[4] = {64, 1, keys, 1};
  const cuuint64_t dims5[5] = {64, 8, args.head2 ? 2 * heads : 2,
                               args.head3 ? heads * groups : groups, pages};
  const cuuint64_t strides5[4] = {bytes(token), bytes(64), bytes(8 * token), bytes(page)};
  const cuuint32_t box5[5] = {64, 8, 2, keys / 8, 1};
  const cuuint32_t estr[5] = {1, 1, 1, 1, 1};
  const bool five = args.paired != 0;
  return encode_fn()(map,
                     a.dtype == SV_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                        : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                     five ? 5 : 4, const_cast<void *>(base), five ? dims5 : dims4,
                     five ? strides5 : strides4, five ? box5 : box4, estr,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                     CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <class T, int DPAD>
int launch_typed(const spec_target &h, const TcArgs &args, const CUtensorMap &tmK,
                 const CUtensorMap &tmV, cudaStream_t stream) {
  constexpr int smem = Shape<DPAD>::kSmem + static_cast<int>(sizeof(Ctl));
  static_assert(smem <= 232448, "shared memory of one SM");
  if (cudaFuncSetAttribute(attention_tc_kernel<T, DPAD>,
                           cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
    return SV_ERR_CUDA;
  const int grid = h.num_sms;
  if (kDescBytes + sizeof(float) * part_floats<DPAD>() * 2 * grid > h.scratch_bytes ||
      sizeof(Desc) * grid > kDescBytes || args.walks > kMaxWalks)
    return SV_ERR_CUDA;
  if (launch_chained(attention_tc_kernel<T, DPAD>, dim3(grid), dim3(kThreads), smem, stream, tmK,
                     tmV, args) != cudaSuccess)
    return SV_ERR_CUDA;
  // an item's rows, on average: sixteen warps for each 32 of them
  const int64_t rows = (static_cast<int64_t>(args.a.T) * (args.a.Hq / args.a.Hkv) + args.a.B - 1) /
                       args.a.B;
  const int blocks = rows > 128 ? 8 : rows > 64 ? 4 : 2;
  return launch_chained(attention_join_kernel<T, DPAD>, dim3(grid, blocks),
                        dim3(32 * kJoinWarps), 0, stream, args) == cudaSuccess
             ? SV_OK
             : SV_ERR_CUDA;
}

}  // namespace

int launch_attention_tc(const spec_target &h, const sv_attention_t &a, cudaStream_t stream) {
  auto ok = [](const void *p, int64_t s0, int64_t s1, int64_t s2) {
    return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && ((s0 | s1 | s2) & 7) == 0;
  };
  // TMA takes positive strides below 2^40 bytes
  auto span = [](int64_t s) { return s > 0 && s < (int64_t(1) << 38); };
  if ((a.dtype != SV_BF16 && a.dtype != SV_FP16) || a.D % 8 != 0 || a.D > 128 ||
      a.page_size < 8 || (a.page_size & (a.page_size - 1)) != 0 ||
      !ok(a.q, a.q_token, a.q_head, 0) || !ok(a.k_cache, a.kc_page, a.kc_token, a.kc_head) ||
      !ok(a.v_cache, a.vc_page, a.vc_token, a.vc_head) || !span(a.kc_page) ||
      !span(a.kc_token) || !span(a.kc_head) || !span(a.vc_page) || !span(a.vc_token) ||
      !span(a.vc_head))
    return kNotTaken;
  CUtensorMap tmK, tmV;
  if (!encode_fn()) return SV_ERR_CUDA;
  TcArgs args{};
  args.a = a;
  if (a.D == 128 && a.page_size <= kPairedPage) {
    auto side_by_side = [&](int64_t head) { return head == a.D; };
    auto in_turn = [&](int64_t token, int64_t head) { return head == token * a.page_size; };
    if (a.Hkv == 1) {
      args.paired = 1;
    } else if (side_by_side(a.kc_head) && side_by_side(a.vc_head)) {
      args.paired = 1;
      args.head2 = 2;
    } else if (in_turn(a.kc_token, a.kc_head) && in_turn(a.vc_token, a.vc_head)) {
      args.paired = 1;
      args.head3 = a.page_size / 8;
    }
  }
  if (!encode_cache(&tmK, args, a.k_cache, a.kc_page, a.kc_token, a.kc_head) ||
      !encode_cache(&tmV, args, a.v_cache, a.vc_page, a.vc_token, a.vc_head))
    return kNotTaken;
  args.scratch = h.scratch;
  args.status = h.status;
  args.wait_limit_ns = h.wait_limit_ns;
  // a scale of zero becomes one too small to matter, so that -inf stays -inf
  const float c = fabsf(a.scale) * 1.4426950408889634f;
  args.c = c > 1e-37f ? c : 1e-37f;
  args.negate = a.scale < 0.0f;
  while ((1 << args.pow_page) < a.page_size) ++args.pow_page;
  args.side = 1;
  while (args.side < 8 && a.Hkv % (2 * args.side) == 0 && h.num_sms % (2 * args.side) == 0)
    args.side *= 2;
  args.walks = h.num_sms / args.side;
  args.by_walks = args.walks > 1 ? ~uint64_t(0) / args.walks : 0;
  const uint64_t G = a.Hq / a.Hkv;
  args.by_group = G > 1 ? static_cast<uint32_t>(((uint64_t(1) << 32) + G - 1) / G) : 0;
  if (a.dtype == SV_BF16)
    return a.D <= 64 ? launch_typed<__nv_bfloat16, 64>(h, args, tmK, tmV, stream)
                     : launch_typed<__nv_bfloat16, 128>(h, args, tmK, tmV, stream);
  return a.D <= 64 ? launch_typed<__half, 64>(h, args, tmK, tmV, stream)
                   : launch_typed<__half, 128>(h, args, tmK, tmV, stream);
}

}  // namespace sv
