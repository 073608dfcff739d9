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
//  * Few rows (up to 256): the weight's rows are the 128 lanes of a tile and
//    A's rows its columns, so W is streamed once and nothing is padded to
//    128.  More rows: A's rows are the lanes and a tile is 128 x 256, so a
//    thread's scale is one number for 128 columns.
//  * Fewer tiles than SMs: a cluster of up to eight CTAs shares a tile, each
//    takes a part of K, and the parts are added through distributed shared
//    memory in the order of K (repeatable, no scratch, no second launch).
//  * Warps 0-7: scale and add (two warpgroups, half of the columns each);
//    warp 8: TMA; warp 9: products; warps 10, 11: the columns' scales.
#include <cudaTypedefs.h>

#include "sv_target.cuh"
#include "sv_tmem.cuh"

namespace sv {
namespace {

constexpr int kThreads = 384;
constexpr int kAddWarps = 8;
constexpr int kAddRegs = 216, kOtherRegs = 72;  // see the attention's kernel
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

__device__ __forceinline__ bool wait_warp(Ctl *ctl, uint64_t *bar, uint32_t parity,
                                          const Args &a) {
  const bool ok = mbar_wait(smem_u32(bar), parity, a.wait_limit_ns, &ctl->abort);
  if (__all_sync(0xffffffffu, ok)) return true;
  if ((threadIdx.x & 31) == 0) {
    *reinterpret_cast<volatile int *>(&ctl->abort) = 1;
    set_status(a.status, SV_ERR_TIMEOUT);
  }
  __syncwarp();
  return false;
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
__device__ __forceinline__ void store_remote(uint32_t smem_addr, uint32_t rank, float x) {
  uint32_t at;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_addr), "r"(rank));
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(at), "f"(x) : "memory");
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
  constexpr int kHalf = kCols / 2;                       // columns of a thread
  constexpr int kSlots = 512 / kCols < 8 ? 512 / kCols : 8;  // blocks in tensor memory
  const MatmulParams &p = args.p;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t *smem = smem_raw + (base - raw);
  Ctl *ctl = reinterpret_cast<Ctl *>(smem + kRingBytes);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

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
  if (warp == 8 && lane == 0) {
    tma_prefetch_desc(&tmLane);
    tma_prefetch_desc(&tmCol);
  }
  if (warp == 9) {
    tmem_alloc(smem_u32(&ctl->tmem), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl->tmem;
  pdl_wait();
  pdl_launch_dependents();

  const int rank = args.split > 1 ? static_cast<int>(cluster_rank()) : 0;
  const int first = blockIdx.x / args.split, step = gridDim.x / args.split;
  const int kb0 = p.kb * rank / args.split, kb1 = p.kb * (rank + 1) / args.split;

  if (warp < kAddWarps) {
    // ---------------- scale, add, store ----------------
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kAddRegs));
    const int half = warp >> 2, row = tid & 127;
    const uint32_t tacc =
        tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + half * kHalf;
    int slot = 0, sslot = 0;
    uint32_t tphase = 0, sphase = 0;
    bool ok = true;
    for (int tile = first; tile < args.tiles && ok; tile += step) {
      const int l0 = tile % args.lane_tiles * kLanes;
      const int c0 = tile / args.lane_tiles * args.bn + half * kHalf;
      float2 acc[kHalf / 2];
#pragma unroll
      for (int i = 0; i < kHalf / 2; ++i) acc[i] = make_float2(0.0f, 0.0f);
      const bool work = !kSwap || half * kHalf < args.bn;
      // lanes = A's rows: one scale a row and one a 128-column block of W
      const bool in = l0 + row < p.M;
      const float *as = p.as + static_cast<int64_t>(in ? l0 + row : 0) * p.kb;
      const float *ws = p.ws + static_cast<int64_t>(c0 < p.N ? c0 / kBlk : 0) * p.kb;
      float s_next = 0.0f;
      if constexpr (!kSwap) s_next = kb0 < kb1 ? __ldg(as + kb0) * __ldg(ws + kb0) : 0.0f;
      for (int kb = kb0; kb < kb1; ++kb) {
        float s = 0.0f;
        if constexpr (!kSwap) {
          s = s_next;
          if (kb + 1 < kb1) s_next = __ldg(as + kb + 1) * __ldg(ws + kb + 1);
        } else {
          if (!(ok = wait_warp(ctl, &ctl->sfull[sslot], sphase, args))) break;
        }
        if (!(ok = wait_warp(ctl, &ctl->tfull[slot], tphase, args))) break;
        tc_fence_after();
        if (work) {
          constexpr int kChunk = kHalf < 32 ? 16 : 32;
#pragma unroll
          for (int g = 0; g < kHalf / kChunk; ++g) {
            uint32_t x[kChunk];
            if constexpr (kChunk == 32) {
              tmem_ld32(tacc + slot * kCols + g * kChunk, x);
              tmem_ld_wait();
              tmem_reg_fence32(x);
            } else {
              tmem_ld16(tacc + slot * kCols + g * kChunk, x);
              tmem_ld_wait();
              tmem_reg_fence(x);
            }
#pragma unroll
            for (int i = 0; i < kChunk; i += 4) {
              float4 sc = make_float4(s, s, s, s);
              if constexpr (kSwap)
                sc = *reinterpret_cast<const float4 *>(
                    &ctl->scale[sslot][half * kHalf + g * kChunk + i]);
              const int j = (g * kChunk + i) / 2;
              acc[j] = fma2(make_float2(__uint_as_float(x[i]), __uint_as_float(x[i + 1])),
                            make_float2(sc.x, sc.y), acc[j]);
              acc[j + 1] = fma2(make_float2(__uint_as_float(x[i + 2]), __uint_as_float(x[i + 3])),
                                make_float2(sc.z, sc.w), acc[j + 1]);
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(smem_u32(&ctl->tempty[slot]));
          if (kSwap) mbar_arrive(smem_u32(&ctl->sempty[sslot]));
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
      const float *x = reinterpret_cast<const float *>(acc);
      const int cols = min(args.bn, (kSwap ? p.M : p.N) - (c0 - half * kHalf));  // of the tile
      if (args.split > 1) {
        // CTA q of the cluster sums the columns [q * per, (q + 1) * per)
        const int per = (args.bn + 8 * args.split - 1) / (8 * args.split) * 8;
        cluster_sync();  // every CTA is done with its ring
        if (ok && work) {
#pragma unroll
          for (int i = 0; i < kHalf; ++i) {
            const int c = half * kHalf + i;
            if (c < cols) {
              const int q = c / per;
              store_remote(base + static_cast<uint32_t>(((rank * per + c - q * per) * kLanes + row)
                                                        * 4),
                           q, x[i]);
            }
          }
        }
        cluster_sync();
        const float *in_parts = reinterpret_cast<const float *>(smem);
        const int n = min(per, cols - rank * per);
        for (int v = 8 * half; v < n; v += 16) {
          float y[8] = {};
          for (int q = 0; q < args.split; ++q)
#pragma unroll
            for (int e = 0; e < 8; ++e)
              if (v + e < n) y[e] += in_parts[(q * per + v + e) * kLanes + row];
          const int c = c0 - half * kHalf + rank * per + v;
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
          for (int i = 0; i < kHalf; ++i)
            if (half * kHalf + i < cols) store_one(p, (c0 + i) * p.os + l0 + row, x[i]);
        } else {
#pragma unroll
          for (int i = 0; i < kHalf; i += 8)
            if (half * kHalf + i < cols)
              store_eight(p, (l0 + row) * p.os + c0 + i, x + i, cols - half * kHalf - i,
                          args.fast);
        }
      }
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp == 8) {
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
    } else if (warp == 9) {
      // ---------------- products ----------------
      const uint32_t idesc = idesc_e4m3(kLanes, args.bn);
      int stage = 0, slot = 0, consumed = 0;
      uint32_t phase = 0, tphase = 0;
      bool ok = true;
      for (int tile = first; tile < args.tiles && ok; tile += step) {
        for (int kb = kb0; kb < kb1; ++kb) {
          if (!(ok = wait_warp(ctl, &ctl->tempty[slot], tphase ^ 1u, args))) break;
          if (!(ok = wait_warp(ctl, &ctl->full[stage], phase, args))) break;
          if (lane == 0) ctl->consumed = ++consumed;
          tc_fence_after();
          const uint32_t at = base + stage * args.stage_bytes;
          const uint64_t ad = sw128_desc(at), bd = sw128_desc(at + kLanes * kBlk);
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
      // ---------------- the columns' scales: warps 10 and 11 in turn --------
      int i = 0;  // block of this CTA's run
      bool ok = true;
      for (int tile = first; tile < args.tiles && ok; tile += step) {
        const int lt = tile % args.lane_tiles, c0 = tile / args.lane_tiles * args.bn;
        const float *ws = p.ws + static_cast<int64_t>(lt) * p.kb;
        for (int kb = kb0; kb < kb1; ++kb, ++i) {
          if ((i & 1) != warp - 10) continue;
          float v[kCols / 32];
          const float w = __ldg(ws + kb);
#pragma unroll
          for (int e = 0; e < kCols / 32; ++e) {
            const int c = c0 + lane + 32 * e;
            v[e] = lane + 32 * e < args.bn && c < p.M
                       ? __ldg(p.as + static_cast<int64_t>(c) * p.kb + kb) * w
                       : 0.0f;
          }
          const int s = i % kScaleSlots;
          if (!(ok = wait_warp(ctl, &ctl->sempty[s], ((i / kScaleSlots) & 1) ^ 1, args))) break;
#pragma unroll
          for (int e = 0; e < kCols / 32; ++e) ctl->scale[s][lane + 32 * e] = v[e];
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&ctl->sfull[s]));
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
  if (warp == 8 && lane == 0) {
    // only after an abort can copies still be in flight
    const int never = 0;
    for (int i = ctl->consumed; i < ctl->issued; ++i)
      mbar_wait(smem_u32(&ctl->full[i % args.stages]),
                static_cast<uint32_t>((i / args.stages) & 1), kCleanupLimitNs, &never);
  }
  __syncthreads();
  if (warp == 9) {
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
  const bool swap = P.M <= 256;
  const int rows = swap ? P.N : P.M, other = swap ? P.M : P.N;
  const int lane_tiles = (rows + kLanes - 1) / kLanes;
  args.bn = swap ? (P.M + 15) / 16 * 16 : 256;
  if (!swap && static_cast<int64_t>(lane_tiles) * ((other + 255) / 256) < h.num_sms) args.bn = 128;
  const int64_t tiles = static_cast<int64_t>(lane_tiles) * ((other + args.bn - 1) / args.bn);
  if (tiles > INT32_MAX) return SV_ERR_SHAPE;
  args.lane_tiles = lane_tiles;
  args.tiles = static_cast<int>(tiles);
  args.split = 1;
  // the largest cluster of which all tiles' run at once
  for (int s = 2; s <= kMaxSplit && s <= P.kb; ++s)
    if (tiles <= h.clusters[s]) args.split = s;
  const int grid = args.split > 1 ? args.split * args.tiles
                                  : (args.tiles < h.num_sms ? args.tiles : h.num_sms);
  args.stage_bytes = ((kLanes + args.bn) * kBlk + 1023) / 1024 * 1024;
  args.stages = kRingBytes / args.stage_bytes;
  if (args.stages > kMaxStages) args.stages = kMaxStages;
  const int es = P.out_dtype == SV_FP32 ? 4 : 2;
  args.fast = (reinterpret_cast<uintptr_t>(P.out) & 15u) == 0 && P.os * es % 16 == 0;
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
  else if (args.bn <= 128)
    e = launch<128, true>(args, lane, col, grid, stream);
  else
    e = launch<256, true>(args, lane, col, grid, stream);
  return e == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}

}  // namespace sv
