// sv_linear_pair.cu -- products with an epilogue for many rows of x: pairs of
// CTAs on two SMs share a tile of 256 rows of x and up to 256 rows of the
// weight (tcgen05 cta_group::2).
//
//  * Each CTA of a pair loads its 128 rows of x and half of the weight's rows of
//    the tile, so a K block of 64 costs an SM 32 KB for 256 x 128 x 64 products.
//    Gated: the one CTA loads rows of the gate's weight and the other the same
//    rows of the second one, so that both factors of an element lie in one row
//    of tensor memory.
//  * The pairs are persistent; a tile's epilogue (warps 0-7) runs beside the next
//    tile's products, in the other half of tensor memory.
//  * Fewer tiles than pairs: a cluster of two or four pairs shares a tile, each pair
//    takes a part of K, and each finishes some of the columns: the others' sums of
//    these come through distributed shared memory and are added in the order of K.
//  * Warp 8: TMA of its CTA; warp 9: products, in the first CTA of the pair alone.
//  * The columns of a tile are chosen so that the tiles fill whole waves.
//
// What bounds it (times of kernels in a CUDA graph): many rows the tensor cores (4096 x
// 14336 x 4096 gated 480 us, 2.0 PFLOP/s, their pipe 97% active; 4096 x 4096 x 14336
// 264 us, 1.82, in four waves of 224 columns; under the power cap of long runs 1.77 and
// 1.58).  Few tiles: about 8 us of start, first load, exchange and epilogue, and x, whose
// rows all tiles read at once: 205 x 8192 x 8192 takes 32 us (the weight's bytes 21), 43
// if every load of x is of the same rows, 29 if the weight's are.  Other places in K for
// each tile's start: 5 to 25% slower.  A short K: the epilogue.
#include <algorithm>

#include "sv_linear_tc.cuh"

namespace sv {
namespace {

constexpr int kEpiWarps = 8, kLoadWarp = 8, kMmaWarp = 9;
constexpr int kThreads = 32 * 10;
constexpr int kLanes = 128;      // rows of x of a CTA
constexpr int kStage = (kLanes + 128) * 128;
constexpr int kMaxStages = 7;

struct Args {
  LinearParams p;
  int *status;
  uint64_t limit_ns;
  int bn;                      // columns of a tile: rows of the weight(s)
  int row_tiles, col_tiles, group;
  int split;                   // pairs that share a tile, each a part of K
  int kblocks, stages;
  int bf16;
  int wide;  // 16-byte accesses of the output's and the residual's rows
};

struct Ctl {
  uint64_t full[kMaxStages], empty[kMaxStages];
  uint64_t tfull[2], tempty[2];
  uint64_t teardown, parts, idle;
  uint32_t tmem;
  int abort;
};

constexpr int kSmemBytes = 1024 + kMaxStages * kStage + static_cast<int>(sizeof(Ctl));
static_assert(kSmemBytes <= 232448, "shared memory of one SM");

// ---- the pair's forms of the tensor-core instructions -----------------------
__device__ __forceinline__ void alloc_pair(uint32_t dst_smem, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst_smem),
               "r"(ncols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void dealloc_pair(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols)
               : "memory");
}
__device__ __forceinline__ void umma_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Arrives on the barrier at this offset in both CTAs of the pair (`mask`) when the
// products issued so far have completed.
__device__ __forceinline__ void commit_pair(uint32_t bar, uint16_t mask) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 "
      "[%0], %1;" ::"r"(bar),
      "h"(mask)
      : "memory");
}
// A load into this CTA that completes on a barrier of either.
__device__ __forceinline__ void load_pair(uint32_t dst, const CUtensorMap *m, int32_t c0,
                                          int32_t c1, uint32_t bar, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes.cta_group::2"
      ".L2::cache_hint [%0], [%1, {%2, %3}], [%4], %5;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(c0), "r"(c1), "r"(bar), "l"(policy)
      : "memory");
}

// ---- epilogue ---------------------------------------------------------------
// Four lanes hold a row each, of four pieces of 16 bytes; afterwards lane q of the four
// holds piece q of each of their rows (and the other way round).
__device__ __forceinline__ void swap_pieces(uint4 &send0, uint4 &send1, bool upper, int lanes) {
  // the upper lane gives its first piece for the lower one's second
  uint4 t = upper ? send0 : send1;
  t.x = __shfl_xor_sync(0xffffffffu, t.x, lanes);
  t.y = __shfl_xor_sync(0xffffffffu, t.y, lanes);
  t.z = __shfl_xor_sync(0xffffffffu, t.z, lanes);
  t.w = __shfl_xor_sync(0xffffffffu, t.w, lanes);
  if (upper)
    send0 = t;
  else
    send1 = t;
}
__device__ __forceinline__ void turn_pieces(uint4 (&p)[4]) {
  const bool odd = threadIdx.x & 1, high = threadIdx.x & 2;
  swap_pieces(p[0], p[1], odd, 1);
  swap_pieces(p[2], p[3], odd, 1);
  swap_pieces(p[0], p[2], high, 2);
  swap_pieces(p[1], p[3], high, 2);
}
// 32 consecutive elements of a row that is 16-byte aligned.
__device__ __forceinline__ void load_row32(const void *p, int64_t at, int dtype, float *v) {
  if (dtype == SV_FP32) {
    const uint4 *q = reinterpret_cast<const uint4 *>(static_cast<const float *>(p) + at);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint4 u = q[i];
      v[4 * i] = __uint_as_float(u.x), v[4 * i + 1] = __uint_as_float(u.y);
      v[4 * i + 2] = __uint_as_float(u.z), v[4 * i + 3] = __uint_as_float(u.w);
    }
  } else {
    const uint4 *q = reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p) + at);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint4 u = q[i];
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float2 f;
        if (dtype == SV_BF16)
          f = make_float2(__uint_as_float(w[j] << 16), __uint_as_float(w[j] & 0xFFFF0000u));
        else
          f = __half22float2(*reinterpret_cast<const __half2 *>(&w[j]));
        v[8 * i + 2 * j] = f.x;
        v[8 * i + 2 * j + 1] = f.y;
      }
    }
  }
}
// 32 consecutive elements of a row a lane, the first `rows` lanes' inside, all 16-byte
// aligned.  Four lanes store 64 bytes of a row together: with each lane on its own row a
// store meets 32 lines, which bounds the epilogue of a short K (2616 x 13840 x 112: 31.4
// us against 38.7; loads of the residual gain nothing so, as L1 holds their lines).
__device__ __forceinline__ void store_row32(void *p, int64_t at, int64_t stride, int rows,
                                            int dtype, const float *v) {
  const int size = dtype == SV_FP32 ? 4 : 2;
  char *base = static_cast<char *>(p) + at * size;
  uint4 w[4];
  auto put = [&](char *to, int64_t row_bytes) {
    const int lane = threadIdx.x & 31, first = lane & ~3;
    char *q = to + first * row_bytes + (lane & 3) * 16;
#pragma unroll
    for (int j = 0; j < 4; ++j, q += row_bytes)
      if (first + j < rows) *reinterpret_cast<uint4 *>(q) = w[j];
  };
  if (dtype == SV_FP32) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int i = 0; i < 16; ++i)
        reinterpret_cast<uint32_t *>(w)[i] = __float_as_uint(v[16 * h + i]);
      turn_pieces(w);
      put(base + 64 * h, stride * 4);
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    uint32_t u;
    if (dtype == SV_BF16) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      u = *reinterpret_cast<const uint32_t *>(&h);
    } else {
      const __half2 h = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
      u = *reinterpret_cast<const uint32_t *>(&h);
    }
    reinterpret_cast<uint32_t *>(w)[i] = u;
  }
  turn_pieces(w);
  put(base, stride * 2);
}
// One element of each of 32 rows, `live` of them inside.
__device__ __forceinline__ void load_rows32(const void *p, int64_t at, int64_t stride, int live,
                                            int dtype, float *v) {
  uint32_t w[32];
  if (dtype == SV_FP32) {
    const uint32_t *q = static_cast<const uint32_t *>(p) + at;
#pragma unroll
    for (int r = 0; r < 32; ++r, q += stride) w[r] = r < live ? *q : 0;
  } else {
    const uint16_t *q = static_cast<const uint16_t *>(p) + at;
#pragma unroll
    for (int r = 0; r < 32; ++r, q += stride) w[r] = r < live ? *q : 0;
  }
#pragma unroll
  for (int r = 0; r < 32; ++r)
    v[r] = dtype == SV_FP32   ? __uint_as_float(w[r])
           : dtype == SV_BF16 ? __uint_as_float(w[r] << 16)
                              : __half2float(__ushort_as_half(static_cast<unsigned short>(w[r])));
}
__device__ __forceinline__ void store_rows32(void *p, int64_t at, int64_t stride, int live,
                                             int dtype, const float *v) {
  if (dtype == SV_FP32) {
    float *q = static_cast<float *>(p) + at;
#pragma unroll
    for (int r = 0; r < 32; ++r, q += stride)
      if (r < live) *q = v[r];
  } else {
    uint16_t *q = static_cast<uint16_t *>(p) + at;
#pragma unroll
    for (int r = 0; r < 32; ++r, q += stride)
      if (r < live)
        *q = dtype == SV_BF16 ? __bfloat16_as_ushort(__float2bfloat16_rn(v[r]))
                              : __half_as_ushort(__float2half_rn(v[r]));
  }
}
__device__ __forceinline__ void activate32(float *v, int act) {
  if (act == SV_ACT_NONE) return;
#pragma unroll
  for (int i = 0; i < 32; i += 8) {
    const Eight r = activate8({make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]),
                               make_float4(v[i + 4], v[i + 5], v[i + 6], v[i + 7])},
                              act);
    v[i] = r.a.x, v[i + 1] = r.a.y, v[i + 2] = r.a.z, v[i + 3] = r.a.w;
    v[i + 4] = r.b.x, v[i + 5] = r.b.y, v[i + 6] = r.b.z, v[i + 7] = r.b.w;
  }
}
// The biases of 32 columns, one a lane, of which the lanes hand each other theirs.
__device__ __forceinline__ float load_bias(const void *p, int64_t n, int in, int dtype) {
  const int lane = threadIdx.x & 31;
  return p && lane < in ? load_any(p, n + lane, dtype) : 0.0f;
}
__device__ __forceinline__ void add_bias(float (&y)[32], float b) {
#pragma unroll
  for (int i = 0; i < 32; ++i) y[i] += __shfl_sync(0xffffffffu, b, i);
}

// Tiles in the order of the pairs: bands of `group` row tiles, within a band
// column by column, so that the tiles that run at once share rows and columns.
__device__ __forceinline__ void place(const Args &a, int tile, int &tr, int &tc) {
  const int band = tile / (a.group * a.col_tiles), in = tile - band * a.group * a.col_tiles;
  const int rows = min(a.group, a.row_tiles - band * a.group);
  tr = band * a.group + in % rows;
  tc = in / rows;
}

// 32 columns of a row a thread, from their sums to the output: y of x w^T (or of the
// gate's), u of the second factor.  `in` columns from n on are inside; m0: the warp's
// first row; piece: its 32 x 32 floats of shared memory.
template <bool kGated>
__device__ __forceinline__ void finish(const Args &args, int64_t m0, float *piece, int64_t n,
                                       int in, float (&y)[32], float (&u)[32], float b, float bu) {
  const LinearParams &p = args.p;
  const int lane = threadIdx.x & 31;
  if (p.bias) add_bias(y, b);
  activate32(y, p.act);
  if constexpr (kGated) {
    if (p.bias_u) add_bias(u, bu);
#pragma unroll
    for (int i = 0; i < 32; ++i) y[i] *= u[i];
  }
  if (args.wide && in == 32) {
    const int rows = static_cast<int>(max(min(static_cast<int64_t>(32), p.M - m0),
                                          static_cast<int64_t>(0)));
    if (p.res && lane < rows) {
      load_row32(p.res, (m0 + lane) * p.rs + n, p.out_dtype, u);
#pragma unroll
      for (int i = 0; i < 32; ++i) y[i] += u[i];
    }
    __syncwarp();  // (the residual may be the output itself)
    store_row32(p.out, m0 * p.os + n, p.os, rows, p.out_dtype, y);
  } else {
    // Through shared memory, a row at a time with a lane for each column: rows of an
    // odd stride, by single elements of 32 rows at once, took 54 us of 205 x 8190 x
    // 8192 without an activation, and 32 so.
#pragma unroll
    for (int i = 0; i < 32; ++i) piece[lane * 32 + (i ^ lane)] = y[i];
    const int live = lane < in ? static_cast<int>(min(static_cast<int64_t>(32), p.M - m0)) : 0;
    if (p.res) load_rows32(p.res, m0 * p.rs + n + lane, p.rs, live, p.out_dtype, u);
    __syncwarp();
#pragma unroll
    for (int r = 0; r < 32; ++r) y[r] = piece[r * 32 + (lane ^ r)];
    if (p.res) {
#pragma unroll
      for (int r = 0; r < 32; ++r) y[r] += u[r];
    }
    store_rows32(p.out, m0 * p.os + n + lane, p.os, live, p.out_dtype, y);
  }
  __syncwarp();
}

template <bool kGated>
__global__ void __launch_bounds__(kThreads, 1)
    linear_pair_kernel(const __grid_constant__ CUtensorMap tmX,
                       const __grid_constant__ CUtensorMap tmW,
                       const __grid_constant__ CUtensorMap tmU, const __grid_constant__ Args args) {
  const LinearParams &p = args.p;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t *smem = smem_raw + (base - raw);
  Ctl *ctl = reinterpret_cast<Ctl *>(smem + kMaxStages * kStage);
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const int crank = static_cast<int>(lin_cluster_rank());
  const int rank = crank & 1, part = crank >> 1;  // in the pair; the pair in the cluster
  const LinAbort ab{args.status, args.limit_ns, &ctl->abort};

  if (tid == 0) {
    for (int i = 0; i < args.stages; ++i) {
      mbar_init(smem_u32(&ctl->full[i]), 1);
      mbar_init(smem_u32(&ctl->empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&ctl->tfull[i]), 1);
      mbar_init(smem_u32(&ctl->tempty[i]), 2 * kEpiWarps);
    }
    mbar_init(smem_u32(&ctl->teardown), 1);
    mbar_init(smem_u32(&ctl->parts), 1);
    mbar_init(smem_u32(&ctl->idle), kEpiWarps * (args.split > 1 ? args.split - 1 : 1));
    ctl->abort = 0;
    mbar_fence_init();
  }
  if (warp == kLoadWarp && lane == 0) {
    tma_prefetch_desc(&tmX);
    tma_prefetch_desc(&tmW);
    if (kGated) tma_prefetch_desc(&tmU);
  }
  if (warp == kMmaWarp) alloc_pair(smem_u32(&ctl->tmem), 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, ctl->tmem, 0);
  lin_cluster_sync();  // the barriers of all CTAs are set up
  pdl_wait();
  pdl_launch_dependents();

  const int first = blockIdx.x / (2 * args.split), step = gridDim.x / (2 * args.split);
  const int tiles = args.row_tiles * args.col_tiles;
  const int half = args.bn / 2;                   // weight rows that a CTA loads
  const int cols = kGated ? half : args.bn;       // output columns of a tile
  const int kb0 = static_cast<int>(static_cast<int64_t>(args.kblocks) * part / args.split);
  const int kb1 = static_cast<int>(static_cast<int64_t>(args.kblocks) * (part + 1) / args.split);
  // an epilogue warp's lanes of tensor memory and rows of the tile
  const uint32_t tacc = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
  float *piece = reinterpret_cast<float *>(smem + (kMaxStages - 1) * kStage) + (warp & 7) * 1024;
  bool ok = true;

  if (warp < kEpiWarps) {
    // ---------------- epilogue ----------------
    const uint32_t tempty0 = lin_remote(smem_u32(&ctl->tempty[0]), crank & ~1);
    const int row = (warp & 3) * 32 + lane;
    // Pair q of the cluster finishes the tile's columns [q own, (q + 1) own).
    const int own = cols / args.split;
    const int width = kGated ? 2 * own : own;  // columns of a part
    const float4 *in_parts = reinterpret_cast<const float4 *>(smem);
    uint32_t it = 0;
    for (int tile = first; tile < tiles && ok; tile += step, ++it) {
      int tr, tc;
      place(args, tile, tr, tc);
      const uint32_t slot = it & 1;
      if (!(ok = lin_wait(smem_u32(&ctl->tfull[slot]), it >> 1 & 1, ab))) break;
      tc_fence_after();
      if (args.split > 1) {
        // The other pairs' sums of the columns that this one finishes come into its
        // ring, which by now is idle, as [pair][column / 4][row][column % 4] (gated: of
        // both factors).  A cluster takes one tile, so this happens once.
        const uint32_t bar = smem_u32(&ctl->parts), idle = smem_u32(&ctl->idle);
        if (tid == 0) mbar_arrive_expect_tx(bar, (args.split - 1) * width * kLanes * 4);
        for (int d = 1; d < args.split; ++d)
          if (lane == 0)
            lin_arrive_remote(lin_remote(idle, 2 * ((part + d) % args.split) + rank));
        __syncwarp();
        if (!(ok = lin_wait<true>(idle, 0, ab))) break;
        for (int d = 1; d < args.split; ++d) {
          const int q = (part + d) % args.split;
          const int at = part < q ? part : part - 1;  // this pair's place among q's parts
          const uint32_t to = lin_remote(base + (at * width * kLanes + row * 4) * 4, 2 * q + rank);
          const uint32_t to_bar = lin_remote(bar, 2 * q + rank);
          for (int v = (warp >> 2) * 32; v < width; v += 64) {
            const int c = v < own ? q * own + v : half + q * own + v - own;
            uint32_t x[32];
            tmem_ld32(tacc + c, x);
            tmem_ld_wait();
            tmem_reg_fence32(x);
#pragma unroll
            for (int e = 0; e < 32; e += 4)
              lin_store_remote(to + (v + e) * kLanes * 4, x + e, to_bar);
          }
        }
        __syncwarp();
        if (!(ok = lin_wait<true>(bar, 0, ab))) break;
      }
      const int64_t m0 = static_cast<int64_t>(tr) * 256 + rank * kLanes + (warp & 3) * 32;
      for (int v = (warp >> 2) * 32; v < own; v += 64) {
        const int c = part * own + v;  // column of the tile
        const int64_t n = static_cast<int64_t>(tc) * cols + c;
        const int in = static_cast<int>(min(p.N - n, static_cast<int64_t>(min(32, cols - c))));
        if (in <= 0) break;
        const float b = load_bias(p.bias, n, in, p.dtype);
        const float bu = kGated ? load_bias(p.bias_u, n, in, p.dtype) : 0.0f;
        uint32_t x[2][32];
        tmem_ld32(tacc + slot * 256 + c, x[0]);
        if (kGated) tmem_ld32(tacc + slot * 256 + half + c, x[1]);
        tmem_ld_wait();
        float y[2][32];
#pragma unroll
        for (int g = 0; g < (kGated ? 2 : 1); ++g) {
          tmem_reg_fence32(x[g]);
          if (args.split == 1) {
#pragma unroll
            for (int e = 0; e < 32; ++e) y[g][e] = __uint_as_float(x[g][e]);
          } else {
            // the sums in the order of K
#pragma unroll
            for (int e = 0; e < 32; ++e) y[g][e] = 0.0f;
            for (int q = 0; q < args.split; ++q) {
              if (q == part) {
#pragma unroll
                for (int e = 0; e < 32; ++e) y[g][e] += __uint_as_float(x[g][e]);
              } else {
                const float4 *f =
                    in_parts + ((q < part ? q : q - 1) * width + g * own + v) / 4 * kLanes + row;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                  const float4 a = f[e * kLanes];
                  y[g][4 * e] += a.x, y[g][4 * e + 1] += a.y;
                  y[g][4 * e + 2] += a.z, y[g][4 * e + 3] += a.w;
                }
              }
            }
          }
        }
        finish<kGated>(args, m0, piece, n, in, y[0], y[1], b, bu);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) lin_arrive_remote(tempty0 + slot * 8);
      __syncwarp();
    }
  } else if (warp == kLoadWarp) {
    // ---------------- TMA ----------------
    // A weight that all its tiles read at about the same time leaves L2 first (3% of
    // 205 to 2048 rows; more rows read it again later).
    const uint64_t policy = policy_evict_normal();
    const uint64_t policy_w = args.row_tiles <= args.group ? policy_evict_first() : policy;
    const CUtensorMap *tmB = kGated && rank ? &tmU : &tmW;
    const uint32_t full0 = lin_remote(smem_u32(&ctl->full[0]), crank & ~1);
    int stage = 0;
    uint32_t phase = 0;
    for (int tile = first; tile < tiles && ok; tile += step) {
      int tr, tc;
      place(args, tile, tr, tc);
      const int m0 = tr * 256 + rank * kLanes;
      const int n0 = kGated ? tc * half : tc * args.bn + rank * half;
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!(ok = lin_wait(smem_u32(&ctl->empty[stage]), phase ^ 1u, ab))) break;
        if (lane == 0) {
          // the first CTA's barrier counts the bytes of both
          if (rank == 0)
            mbar_arrive_expect_tx(smem_u32(&ctl->full[stage]), 2 * (kLanes + half) * 128);
          const uint32_t at = base + stage * kStage, full = full0 + stage * 8;
          load_pair(at, &tmX, kb * kLinBlk, m0, full, policy);
          load_pair(at + kLanes * 128, tmB, kb * kLinBlk, n0, full, policy_w);
        }
        __syncwarp();
        if (++stage == args.stages) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
  } else if (rank == 0) {
    // ---------------- products ----------------
    const uint32_t idesc = idesc_16(args.bf16, 256, args.bn, false);
    const uint16_t mask = static_cast<uint16_t>(3u << (crank & ~1));
    int stage = 0;
    uint32_t phase = 0, it = 0;
    for (int tile = first; tile < tiles && ok; tile += step, ++it) {
      const uint32_t slot = it & 1;
      if (!(ok = lin_wait<true>(smem_u32(&ctl->tempty[slot]), (it >> 1 & 1) ^ 1u, ab))) break;
      tc_fence_after();
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!(ok = lin_wait<true>(smem_u32(&ctl->full[stage]), phase, ab))) break;
        tc_fence_after();
        if (elect_one()) {
          const uint32_t at = base + stage * kStage;
          const uint64_t ad = sw128_desc(at), bd = sw128_desc(at + kLanes * 128);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            umma_pair(tmem + slot * 256, ad + 2u * k, bd + 2u * k, idesc, kb > kb0 || k > 0);
          commit_pair(smem_u32(&ctl->empty[stage]), mask);
          if (kb == kb1 - 1) commit_pair(smem_u32(&ctl->tfull[slot]), mask);
        }
        __syncwarp();
        if (++stage == args.stages) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    if (elect_one()) commit_pair(smem_u32(&ctl->teardown), mask);
    __syncwarp();
  }

  // ---------------- teardown ----------------
  if (warp == kLoadWarp) {
    const int never = 0;
    // the products are done: their commit arrives in both CTAs
    if (lane == 0) mbar_wait(smem_u32(&ctl->teardown), 0u, kLinCleanupNs, &never);
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  lin_leave(&ctl->abort, 2 * args.split);
  if (warp == kMmaWarp) {
    tc_fence_after();
    dealloc_pair(tmem, 512);
  }
}

template <bool kGated>
int launch(const spec_target &h, const LinearParams &P, cudaStream_t stream) {
  if (!lin_encode_fn()) return SV_ERR_CUDA;
  Args args{};
  args.p = P;
  args.status = h.status;
  args.limit_ns = h.wait_limit_ns;
  args.bf16 = P.dtype == SV_BF16;
  args.kblocks = static_cast<int>((P.K + kLinBlk - 1) / kLinBlk);
  const int64_t row_tiles = (P.M + 255) / 256;
  // Columns of a tile, and pairs that share one: by the time of a K block, which is
  // that of its products (two cycles a column) or of its loads (about 40 bytes a
  // cycle), the waves of tiles, and what a tile takes besides.
  int64_t best = INT64_MAX, col_tiles = 0;
  for (int split = 1; split <= 4; split *= 2) {
    const int64_t clusters = split == 1 ? h.num_sms / 2 : h.clusters[2 * split];
    if (split > args.kblocks) break;
    for (int bn = 256; bn >= 64; bn -= 32) {
      const int cols = kGated ? bn / 2 : bn;
      if (cols % (32 * split) != 0) continue;  // the epilogue takes 32 columns at a time
      const int64_t ct = (P.N + cols - 1) / cols, tiles = row_tiles * ct;
      if (split > 1 && tiles > clusters) continue;  // a cluster takes one tile
      const int64_t block = std::max(2 * bn, (kLanes + bn / 2) * 128 / 40);
      const int64_t time = (tiles + clusters - 1) / clusters *
                               ((args.kblocks + split - 1) / split * block + 16 * bn) +
                           (split > 1 ? 4000 : 0);
      if (time < best) {
        best = time;
        args.bn = bn;
        args.split = split;
        col_tiles = ct;
      }
    }
  }
  if (row_tiles * col_tiles > (1 << 30)) return SV_ERR_SHAPE;
  args.row_tiles = static_cast<int>(row_tiles);
  args.col_tiles = static_cast<int>(col_tiles);
  // Row tiles of a band: eight, and up to sixteen where their rows of x (36 MB) stay in
  // L2 while the weight passes, which then comes from HBM once a band (under the power
  // cap, with an epilogue of 10 us more, 4096 x 14336 x 4096 gated took 557 us with
  // sixteen, 580 with eight; 8192 x 8192 x 8192 693 and 680).
  const int64_t fit = (int64_t(36) << 20) / (512 * P.K);
  args.group = static_cast<int>(std::min(row_tiles, std::clamp<int64_t>(fit, 8, 16)));
  const int es = P.out_dtype == SV_FP32 ? 4 : 2;
  auto wide = [](const void *p, int64_t stride_bytes, int64_t rows) {
    return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && (rows <= 1 || stride_bytes % 16 == 0);
  };
  args.wide = wide(P.out, P.os * es, P.M) && wide(P.res, P.rs * es, P.M);
  // (rows that leave through shared memory take the last stage's; a cluster's ring is
  // idle by then)
  args.stages =
      (args.wide && P.N % 32 == 0) || args.split > 1 ? kMaxStages : kMaxStages - 1;
  CUtensorMap x, w, u;
  if (!lin_encode(&x, P.x, P.xs, P.K, P.M, kLanes) ||
      !lin_encode(&w, P.w, P.ws, P.K, P.N, args.bn / 2) ||
      !lin_encode(&u, kGated ? P.wu : P.w, kGated ? P.wus : P.ws, P.K, P.N, args.bn / 2))
    return SV_ERR_CUDA;
  cudaError_t e = cudaFuncSetAttribute(linear_pair_kernel<kGated>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
  if (e != cudaSuccess) return SV_ERR_CUDA;
  const int64_t tiles = row_tiles * col_tiles;
  const int64_t pairs = args.split > 1 ? tiles * args.split
                                       : std::min<int64_t>(tiles, h.num_sms / 2);
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2 * args.split;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(2 * pairs));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  e = cudaLaunchKernelEx(&cfg, linear_pair_kernel<kGated>, x, w, u, args);
  return e == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}

}  // namespace

int launch_linear_pair(const spec_target &h, const LinearParams &P, cudaStream_t stream) {
  return P.wu ? launch<true>(h, P, stream) : launch<false>(h, P, stream);
}

}  // namespace sv
