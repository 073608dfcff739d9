// sv_matmul8.cu -- 8-bit product with one fp32 scale per row and 128 columns
// of A and per 128 x 128 block of W:
//
//   out[m, n] = sum_b as[m, b] ws[n / 128, b] sum_{k in b} A8[m, k] W8[n, k]
//
// The tensor cores (tcgen05 kind::f8f6f4) sum one block of 128 columns into a
// slot of tensor memory; the epilogue warps read the slot, scale it and add
// it to fp32 registers, while the next blocks are multiplied into other
// slots.  The scales can be any fp32 number, which the hardware's own block
// scales (powers of two) cannot.
//
//  * Few rows (up to 96): the weight's rows are the 128 lanes of a tile and
//    A's rows its columns, so W is streamed once and nothing is padded to
//    128.  More rows: A's rows are the lanes and a tile is 128 x 256 (or 128),
//    so a thread's scale is one number for its columns.
//  * Fewer tiles than SMs: a cluster of up to eight CTAs shares a tile, each
//    takes a part of K, and the parts are added through distributed shared
//    memory in the order of K (repeatable, no scratch, no second launch).
//  * Warps 0-7: scale and add (two warpgroups, half of the columns each);
//    warp 8: TMA; warp 9: products; warps 10, 11: the columns' scales.
//
// Times in this file are of kernels in a CUDA graph.  What bounds it (4096 x 14336 x
// 4096, 206 us, 2.33 PFLOP/s; 220 to 230 by single calls): a block of 128 x
// 256 x 128 takes the tensor cores 512 cycles and the whole loop about 1000.
// The products alone run in 127 us.  With the loads it is 190: a load takes
// 1.6 us from its slot's being freed to its use, and the four blocks of 48 KB
// that fit in shared memory are in flight for that long.  With the adding it
// is 189: tensor memory holds two blocks, and a block's products, hand-over
// and reading follow one another.  So the second limit stays when the first is
// lifted: pairs of CTAs that share W's blocks (six of 32 KB in flight) took 214
// us, and handing over half a block's columns at a time 270.
#include <cudaTypedefs.h>

#include "sv_target.cuh"
#include "sv_tmem.cuh"

namespace sv {
namespace {

constexpr int kAddWarps = 8;
constexpr int kThreads = 32 * kAddWarps + 128;
// Registers a thread: 168 at launch; the adding warps take what the others give
// back (256 * 216 + 128 * 72 = 256 * 224 + 128 * 56 = 384 * 168).
template <int kCols>
constexpr int add_regs() { return kCols == 256 ? 224 : 216; }
template <int kCols>
constexpr int other_regs() { return kCols == 256 ? 56 : 72; }
constexpr int kLoadWarp = kAddWarps, kMmaWarp = kAddWarps + 1, kScaleWarp = kAddWarps + 2;
constexpr int kLanes = 128;      // rows of a tile
constexpr int kBlk = 128;        // K elements (bytes) of a block
constexpr int kRingBytes = 192 * 1024;
constexpr int kMaxStages = 8;
constexpr int kScaleSlots = 8;
constexpr int kMaxSplit = 8;
constexpr uint64_t kCleanupLimitNs = 2000000000ull;

struct Args {
  MatmulParams p;
  int *status;
  uint64_t wait_limit_ns;
  int bn;                 // columns of a tile
  int tiles, lane_tiles;  // tiles; of these along the lanes' rows (fastest)
  int split;              // CTAs of a tile
  int stages, stage_bytes;
  int fast;               // 16-byte stores of the output's rows
  int fast_scales;        // 16-byte loads of four scales of a row
};

struct Ctl {
  float scale[kScaleSlots][256];
  uint64_t full[kMaxStages], empty[kMaxStages];
  uint64_t tfull[8], tempty[8];
  uint64_t sfull[kScaleSlots], sempty[kScaleSlots];
  uint64_t teardown;
  uint32_t tmem;
  int abort, issued, consumed;
};

__device__ __noinline__ bool give_up(Ctl *ctl, uint64_t &since, const Args &a) {
  const volatile int *abort = &ctl->abort;
  const uint64_t now = globaltimer();
  if (since == 0) since = now;
  if (!__any_sync(0xffffffffu, now - since >= a.wait_limit_ns || *abort)) return false;
  if ((threadIdx.x & 31) == 0) {
    *reinterpret_cast<volatile int *>(&ctl->abort) = 1;
    set_status(a.status, SV_ERR_TIMEOUT);
  }
  __syncwarp();
  return true;
}
// Waits on a barrier with the whole warp; false: the limit ran out, or another
// role gave up.
__device__ __forceinline__ bool wait_warp(Ctl *ctl, uint64_t *bar, uint32_t parity,
                                          const Args &a) {
  const uint32_t at = smem_u32(bar);
  if (__all_sync(0xffffffffu, mbar_try_wait(at, parity))) return true;
  uint64_t since = 0;
  while (true) {
    for (int i = 0; i < 16; ++i)
      if (__all_sync(0xffffffffu, mbar_try_wait(at, parity))) return true;
    if (give_up(ctl, since, a)) return false;
  }
}

// All threads of the cluster.
__device__ __forceinline__ void cluster_sync() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// The address of another CTA's shared memory in the cluster, and a store there.
__device__ __forceinline__ uint32_t remote_smem(uint32_t smem_addr, uint32_t rank) {
  uint32_t at;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_addr), "r"(rank));
  return at;
}
__device__ __forceinline__ void store_remote(uint32_t at, float x) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(at), "f"(x) : "memory");
}

template <int kChunk>
__device__ __forceinline__ void read_columns(uint32_t at, uint32_t *x) {
  if constexpr (kChunk == 32)
    tmem_ld32(at, x);
  else
    tmem_ld16(at, *reinterpret_cast<uint32_t(*)[16]>(x));
}
template <int kChunk>
__device__ __forceinline__ void columns_arrived(uint32_t *x) {
  tmem_ld_wait();
  if constexpr (kChunk == 32)
    tmem_reg_fence32(x);
  else
    tmem_reg_fence(*reinterpret_cast<uint32_t(*)[16]>(x));
}

__device__ __forceinline__ void store_one(const MatmulParams &p, int64_t at, float x) {
  if (p.out_dtype == SV_BF16)
    static_cast<__nv_bfloat16 *>(p.out)[at] = __float2bfloat16_rn(x);
  else if (p.out_dtype == SV_FP16)
    static_cast<__half *>(p.out)[at] = __float2half_rn(x);
  else
    static_cast<float *>(p.out)[at] = x;
}
// Eight consecutive elements of a row (n of them inside).
__device__ __forceinline__ void store_eight(const MatmulParams &p, int64_t at, const float *x,
                                            int n, bool fast) {
  if (fast && n >= 8) {
    if (p.out_dtype == SV_FP32) {
      float4 *o = reinterpret_cast<float4 *>(static_cast<float *>(p.out) + at);
      o[0] = make_float4(x[0], x[1], x[2], x[3]);
      o[1] = make_float4(x[4], x[5], x[6], x[7]);
    } else {
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (p.out_dtype == SV_BF16) {
          const __nv_bfloat162 v = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
          w[i] = *reinterpret_cast<const uint32_t *>(&v);
        } else {
          const __half2 v = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
          w[i] = *reinterpret_cast<const uint32_t *>(&v);
        }
      }
      *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p.out) + at) =
          make_uint4(w[0], w[1], w[2], w[3]);
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i < n) store_one(p, at + i, x[i]);
}

// kSwap: lanes are W's rows, columns A's (bn <= kCols of them); otherwise
// lanes are A's rows, columns W's (bn == kCols).
template <int kCols, bool kSwap>
__global__ void __launch_bounds__(kThreads, 1)
    matmul8_kernel(const __grid_constant__ CUtensorMap tmLane,
                   const __grid_constant__ CUtensorMap tmCol, const __grid_constant__ Args args) {
  constexpr int kParts = kAddWarps / 4;
  constexpr int kMine = kCols / kParts < 16 ? 16 : kCols / kParts;  // columns of a thread
  constexpr int kSlots = 512 / kCols < 8 ? 512 / kCols : 8;  // blocks in tensor memory
  const MatmulParams &p = args.p;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t *smem = smem_raw + (base - raw);
  Ctl *ctl = reinterpret_cast<Ctl *>(smem + kRingBytes);
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // uniform to the compiler

  if (tid == 0) {
    for (int i = 0; i < args.stages; ++i) {
      mbar_init(smem_u32(&ctl->full[i]), 1);
      mbar_init(smem_u32(&ctl->empty[i]), 1);
    }
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(smem_u32(&ctl->tfull[i]), 1);
      mbar_init(smem_u32(&ctl->tempty[i]), kAddWarps);
    }
    for (int i = 0; i < kScaleSlots; ++i) {
      mbar_init(smem_u32(&ctl->sfull[i]), 1);
      mbar_init(smem_u32(&ctl->sempty[i]), kAddWarps);
    }
    mbar_init(smem_u32(&ctl->teardown), 1);
    ctl->abort = ctl->issued = ctl->consumed = 0;
    mbar_fence_init();
  }
  if (warp == kLoadWarp && lane == 0) {
    tma_prefetch_desc(&tmLane);
    tma_prefetch_desc(&tmCol);
  }
  if (warp == kMmaWarp) {
    tmem_alloc(smem_u32(&ctl->tmem), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, ctl->tmem, 0);
  pdl_wait();
  pdl_launch_dependents();

  const int rank = args.split > 1 ? static_cast<int>(cluster_rank()) : 0;
  const int first = blockIdx.x / args.split, step = gridDim.x / args.split;
  const int kb0 = p.kb * rank / args.split, kb1 = p.kb * (rank + 1) / args.split;

  if (warp < kAddWarps) {
    // ---------------- scale, add, store ----------------
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(add_regs<kCols>()));
    const int own = (warp >> 2) * kMine, row = tid & 127;  // first column, lane
    const uint32_t tacc =
        tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + own;
    int slot = 0, sslot = 0;
    uint32_t tphase = 0, sphase = 0;
    bool ok = true;
    for (int tile = first; tile < args.tiles && ok; tile += step) {
      const int l0 = tile % args.lane_tiles * kLanes;
      const int c0 = tile / args.lane_tiles * args.bn + own;
      uint64_t acc[kMine / 2];  // two columns each
#pragma unroll
      for (int i = 0; i < kMine / 2; ++i) acc[i] = 0;
      const bool work = own < args.bn;
      // lanes = A's rows: one scale a row and one a 128-column block of W
      const bool in = l0 + row < p.M;
      const float *as = p.as + static_cast<int64_t>(in ? l0 + row : 0) * p.kb;
      const float *ws = p.ws + static_cast<int64_t>(c0 < p.N ? c0 / kBlk : 0) * p.kb;
      // scales of four blocks at a time, the next four on their way (one 16-byte
      // load for a row's four: 32 rows are 32 lines, whatever is read of them)
      float sc[4] = {}, as_next[4] = {}, ws_next[4] = {};
      auto fetch = [&](int kb) {
        if (args.fast_scales) {
          const float4 v = __ldg(reinterpret_cast<const float4 *>(as + kb));
          const float4 w = __ldg(reinterpret_cast<const float4 *>(ws + kb));
          as_next[0] = v.x, as_next[1] = v.y, as_next[2] = v.z, as_next[3] = v.w;
          ws_next[0] = w.x, ws_next[1] = w.y, ws_next[2] = w.z, ws_next[3] = w.w;
        } else {
#pragma unroll
          for (int t = 0; t < 4; ++t)
            if (kb + t < kb1) {
              as_next[t] = __ldg(as + kb + t);
              ws_next[t] = __ldg(ws + kb + t);
            }
        }
      };
      if (!kSwap && kb0 < kb1) fetch(kb0);
      for (int kb = kb0; kb < kb1; ++kb) {
        float s = 0.0f;
        if constexpr (!kSwap) {
          const int t = (kb - kb0) & 3;
          if (t == 0) {
#pragma unroll
            for (int i = 0; i < 4; ++i) sc[i] = as_next[i] * ws_next[i];
            if (kb + 4 < kb1) fetch(kb + 4);
          }
          s = t < 2 ? (t == 0 ? sc[0] : sc[1]) : (t == 2 ? sc[2] : sc[3]);
        } else {
          if (!(ok = wait_warp(ctl, &ctl->sfull[sslot], sphase, args))) break;
        }
        if (!(ok = wait_warp(ctl, &ctl->tfull[slot], tphase, args))) break;
        tc_fence_after();
        // the slot is free once its last columns have been read
        auto free_slot = [&]() {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&ctl->tempty[slot]));
        };
        const uint64_t s2 = pair2(s, s);
        if (work) {
          // the next columns are read while these are scaled and added
          constexpr int kChunk = kMine < 32 ? 16 : 32, kChunks = kMine / kChunk;
          uint32_t x[kChunks > 1 ? 2 : 1][kChunk];
          read_columns<kChunk>(tacc + slot * kCols, x[0]);
#pragma unroll
          for (int g = 0; g < kChunks; ++g) {
            uint32_t *y = x[g & 1];
            columns_arrived<kChunk>(y);
            if (g + 1 < kChunks)
              read_columns<kChunk>(tacc + slot * kCols + (g + 1) * kChunk, x[(g + 1) & 1]);
            else
              free_slot();
#pragma unroll
            for (int i = 0; i < kChunk; i += 4) {
              uint64_t s01 = s2, s23 = s2;
              if constexpr (kSwap) {
                const ulonglong2 sc = *reinterpret_cast<const ulonglong2 *>(
                    &ctl->scale[sslot][own + g * kChunk + i]);
                s01 = sc.x;
                s23 = sc.y;
              }
              const int j = (g * kChunk + i) / 2;
              acc[j] = fma2(pair2(__uint_as_float(y[i]), __uint_as_float(y[i + 1])), s01, acc[j]);
              acc[j + 1] = fma2(pair2(__uint_as_float(y[i + 2]), __uint_as_float(y[i + 3])), s23,
                                acc[j + 1]);
            }
          }
        } else {
          free_slot();
        }
        if constexpr (kSwap) {
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&ctl->sempty[sslot]));
        }
        if (++slot == kSlots) {
          slot = 0;
          tphase ^= 1u;
        }
        if (++sslot == kScaleSlots) {
          sslot = 0;
          sphase ^= 1u;
        }
      }
      float x[kMine];
#pragma unroll
      for (int i = 0; i < kMine / 2; ++i) {
        const float2 v = unpair2(acc[i]);
        x[2 * i] = v.x;
        x[2 * i + 1] = v.y;
      }
      const int cols = min(args.bn, (kSwap ? p.M : p.N) - (c0 - own));  // of the tile
      if (args.split > 1) {
        // CTA q of the cluster sums the columns [q * per, (q + 1) * per)
        const int per = (args.bn + 8 * args.split - 1) / (8 * args.split) * 8;
        cluster_sync();  // every CTA is done with its ring
        if (ok && work) {
#pragma unroll
          for (int i = 0; i < kMine; i += 8) {
            const int c = own + i;  // eight columns go to one CTA: per is a multiple of 8
            if (c < cols) {
              const int q = c / per;
              const uint32_t at = remote_smem(
                  base + static_cast<uint32_t>(((rank * per + c - q * per) * kLanes + row) * 4), q);
#pragma unroll
              for (int e = 0; e < 8; ++e) store_remote(at + e * kLanes * 4, x[i + e]);
            }
          }
        }
        cluster_sync();
        const float *in_parts = reinterpret_cast<const float *>(smem);
        const int n = min(per, cols - rank * per);
        for (int v = 8 * (warp >> 2); v < n; v += 8 * kParts) {
          float y[8] = {};
          for (int q = 0; q < args.split; ++q)
#pragma unroll
            for (int e = 0; e < 8; ++e)
              if (v + e < n) y[e] += in_parts[(q * per + v + e) * kLanes + row];
          const int c = c0 - own + rank * per + v;
          if (l0 + row < (kSwap ? p.N : p.M) && !*const_cast<volatile int *>(&ctl->abort)) {
            if constexpr (kSwap) {
#pragma unroll
              for (int e = 0; e < 8; ++e)
                if (v + e < n) store_one(p, (c + e) * p.os + l0 + row, y[e]);
            } else {
              store_eight(p, (l0 + row) * p.os + c, y, n - v, args.fast);
            }
          }
        }
      } else if (ok && work && l0 + row < (kSwap ? p.N : p.M)) {
        if constexpr (kSwap) {
#pragma unroll
          for (int i = 0; i < kMine; ++i)
            if (own + i < cols) store_one(p, (c0 + i) * p.os + l0 + row, x[i]);
        } else {
#pragma unroll
          for (int i = 0; i < kMine; i += 8)
            if (own + i < cols)
              store_eight(p, (l0 + row) * p.os + c0 + i, x + i, cols - own - i,
                          args.fast);
        }
      }
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(other_regs<kCols>()));
    if (warp == kLoadWarp) {
      // ---------------- TMA ----------------
      const uint64_t policy = policy_evict_normal();
      const uint32_t tx = static_cast<uint32_t>((kLanes + args.bn) * kBlk);
      int stage = 0, issued = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int tile = first; tile < args.tiles && ok; tile += step) {
        const int l0 = tile % args.lane_tiles * kLanes, c0 = tile / args.lane_tiles * args.bn;
        for (int kb = kb0; kb < kb1; ++kb) {
          if (!(ok = wait_warp(ctl, &ctl->empty[stage], phase ^ 1u, args))) break;
          if (lane == 0) {
            const uint32_t at = base + stage * args.stage_bytes;
            const uint32_t full = smem_u32(&ctl->full[stage]);
            mbar_arrive_expect_tx(full, tx);
            tma_load_2d(at, &tmLane, kb * kBlk, l0, full, policy);
            tma_load_2d(at + kLanes * kBlk, &tmCol, kb * kBlk, c0, full, policy);
            ctl->issued = ++issued;
          }
          __syncwarp();
          if (++stage == args.stages) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
    } else if (warp == kMmaWarp) {
      // ---------------- products ----------------
      const uint32_t idesc = idesc_e4m3(kLanes, args.bn);
      int stage = 0, slot = 0, consumed = 0;
      uint32_t phase = 0, tphase = 0;
      bool ok = true;
      for (int tile = first; tile < args.tiles && ok; tile += step) {
        for (int kb = kb0; kb < kb1; ++kb) {
          if (!(ok = wait_warp(ctl, &ctl->full[stage], phase, args))) break;
          if (lane == 0) ctl->consumed = ++consumed;
          const uint32_t at = base + stage * args.stage_bytes;
          const uint64_t ad = sw128_desc(at), bd = sw128_desc(at + kLanes * kBlk);
          if (!(ok = wait_warp(ctl, &ctl->tempty[slot], tphase ^ 1u, args))) break;
          tc_fence_after();
          if (elect_one()) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              umma_f8(tmem + slot * kCols, ad + 2u * k, bd + 2u * k, idesc, k > 0);
            umma_commit(smem_u32(&ctl->empty[stage]));
            umma_commit(smem_u32(&ctl->tfull[slot]));
          }
          __syncwarp();
          if (++stage == args.stages) {
            stage = 0;
            phase ^= 1u;
          }
          if (++slot == kSlots) {
            slot = 0;
            tphase ^= 1u;
          }
        }
      }
      if (elect_one()) {
        umma_commit(smem_u32(&ctl->teardown));
        const int never = 0;
        mbar_wait(smem_u32(&ctl->teardown), 0u, kCleanupLimitNs, &never);
      }
      __syncwarp();
    } else if (kSwap) {
      // ---------------- the columns' scales: the last two warps in turn --------
      // four blocks at a time, so that one wait for memory serves four
      int i0 = 0;  // first block of the group in this CTA's run
      bool ok = true;
      for (int tile = first; tile < args.tiles && ok; tile += step) {
        const int lt = tile % args.lane_tiles, c0 = tile / args.lane_tiles * args.bn;
        const float *ws = p.ws + static_cast<int64_t>(lt) * p.kb;
        for (int kb = kb0; kb < kb1 && ok; kb += 4) {
          const int n = min(4, kb1 - kb), i = i0;
          i0 += n;
          if (((kb - kb0) >> 2 & 1) != warp - kScaleWarp) continue;
          constexpr int kE = kCols / 32;
          float v[kE][4], w[4];
#pragma unroll
          for (int t = 0; t < 4; ++t) w[t] = t < n ? __ldg(ws + kb + t) : 0.0f;
#pragma unroll
          for (int e = 0; e < kE; ++e) {
            const int c = c0 + lane + 32 * e;
            const bool in = lane + 32 * e < args.bn && c < p.M;
            const float *as = p.as + static_cast<int64_t>(in ? c : 0) * p.kb + kb;
#pragma unroll
            for (int t = 0; t < 4; ++t) v[e][t] = in && t < n ? __ldg(as + t) : 0.0f;
          }
#pragma unroll
          for (int t = 0; t < 4; ++t) {
            if (t >= n) break;
            const int s = (i + t) % kScaleSlots;
            if (!(ok = wait_warp(ctl, &ctl->sempty[s], (((i + t) / kScaleSlots) & 1) ^ 1, args)))
              break;
#pragma unroll
            for (int e = 0; e < kE; ++e) ctl->scale[s][lane + 32 * e] = v[e][t] * w[t];
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&ctl->sfull[s]));
          }
        }
      }
    }
    if (args.split > 1) {
      cluster_sync();
      cluster_sync();
    }
  }

  // ---------------- teardown ----------------
  tc_fence_before();
  __syncthreads();
  if (warp == kLoadWarp && lane == 0) {
    // only after an abort can copies still be in flight
    const int never = 0;
    for (int i = ctl->consumed; i < ctl->issued; ++i)
      mbar_wait(smem_u32(&ctl->full[i % args.stages]),
                static_cast<uint32_t>((i / args.stages) & 1), kCleanupLimitNs, &never);
  }
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
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

// E4M3 rows [rows, K]: box of `box` rows of 128 bytes.
bool encode_rows(CUtensorMap *map, const void *base, int64_t K, int64_t rows, int box) {
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(K), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(K)};
  const cuuint32_t boxes[2] = {kBlk, static_cast<cuuint32_t>(box)};
  const cuuint32_t estr[2] = {1, 1};
  return encode_fn()(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(base), dims,
                     strides, boxes, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                     CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

constexpr int kSmemBytes = 1024 + kRingBytes + static_cast<int>(sizeof(Ctl));
static_assert(kSmemBytes <= 232448, "shared memory of one SM");

void configure(cudaLaunchConfig_t &cfg, cudaLaunchAttribute (&attr)[2], int split, int grid,
               cudaStream_t stream) {
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = split;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
}

template <int kCols, bool kSwap>
cudaError_t launch(const Args &args, const CUtensorMap &lane, const CUtensorMap &col, int grid,
                   cudaStream_t stream) {
  const cudaError_t e = cudaFuncSetAttribute(
      matmul8_kernel<kCols, kSwap>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr[2];
  configure(cfg, attr, args.split, grid, stream);
  return cudaLaunchKernelEx(&cfg, matmul8_kernel<kCols, kSwap>, lane, col, args);
}

}  // namespace

// How many clusters of each size the GPU holds at once: its SMs come in groups
// that a cluster cannot span, so this is less than SMs / size.
cudaError_t plan_matmul_fp8(spec_target &h) {
  cudaError_t e = cudaFuncSetAttribute(matmul8_kernel<64, true>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
  for (int split = 1; split <= kMaxSplit && e == cudaSuccess; ++split) {
    cudaLaunchConfig_t cfg;
    cudaLaunchAttribute attr[2];
    configure(cfg, attr, split, split, nullptr);
    cfg.numAttrs = 1;
    e = cudaOccupancyMaxActiveClusters(&h.clusters[split], matmul8_kernel<64, true>, &cfg);
  }
  return e;
}

int launch_matmul_fp8(const spec_target &h, const MatmulParams &P, cudaStream_t stream) {
  if (!encode_fn()) return SV_ERR_CUDA;
  Args args{};
  args.p = P;
  args.status = h.status;
  args.wait_limit_ns = h.wait_limit_ns;
  // Up to 96 rows W's rows are the lanes: 96 x 8192 x 8192 in 17.7 us against
  // 18.1 the other way, 128 in 18.9 against 18.5.
  const bool swap = P.M <= 96;
  const int rows = swap ? P.N : P.M, other = swap ? P.M : P.N;
  const int lane_tiles = (rows + kLanes - 1) / kLanes;
  // A tile's columns and the CTAs that share it, by the time that its blocks
  // take (a block of 256 columns about 1000 cycles, of 128 about 600): the
  // largest cluster of which all tiles' run at once, else one CTA a tile and
  // whole waves.
  int64_t tiles = 0, best = INT64_MAX;
  for (const int bn : {swap ? (P.M + 15) / 16 * 16 : 256, 128}) {
    const int64_t n = static_cast<int64_t>(lane_tiles) * ((other + bn - 1) / bn);
    int split = 1;
    for (int s = 2; s <= kMaxSplit && s <= P.kb; ++s)
      if (n <= h.clusters[s]) split = s;
    const int64_t waves = split > 1 ? 1 : (n + h.num_sms - 1) / h.num_sms;
    const int64_t time = waves * ((P.kb + split - 1) / split) * (bn > 128 ? 10 : 6);
    if (time < best) {
      best = time;
      tiles = n;
      args.bn = bn;
      args.split = split;
    }
    if (swap) break;
  }
  if (tiles > INT32_MAX) return SV_ERR_SHAPE;
  args.lane_tiles = lane_tiles;
  args.tiles = static_cast<int>(tiles);
  const int grid = args.split > 1 ? args.split * args.tiles
                                  : (args.tiles < h.num_sms ? args.tiles : h.num_sms);
  args.stage_bytes = ((kLanes + args.bn) * kBlk + 1023) / 1024 * 1024;
  args.stages = kRingBytes / args.stage_bytes;
  if (args.stages > kMaxStages) args.stages = kMaxStages;
  const int es = P.out_dtype == SV_FP32 ? 4 : 2;
  args.fast = (reinterpret_cast<uintptr_t>(P.out) & 15u) == 0 && P.os * es % 16 == 0;
  args.fast_scales = P.kb % 4 == 0 && args.split == 1 &&
                     ((reinterpret_cast<uintptr_t>(P.as) | reinterpret_cast<uintptr_t>(P.ws)) &
                      15u) == 0;
  CUtensorMap lane, col;
  if (!encode_rows(&lane, swap ? P.w : P.a, P.K, rows, kLanes) ||
      !encode_rows(&col, swap ? P.a : P.w, P.K, other, args.bn))
    return SV_ERR_CUDA;
  cudaError_t e;
  if (!swap)
    e = args.bn == 256 ? launch<256, false>(args, lane, col, grid, stream)
                       : launch<128, false>(args, lane, col, grid, stream);
  else if (args.bn <= 32)
    e = launch<32, true>(args, lane, col, grid, stream);
  else if (args.bn <= 64)
    e = launch<64, true>(args, lane, col, grid, stream);
  else
    e = launch<128, true>(args, lane, col, grid, stream);
  return e == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}

}  // namespace sv
