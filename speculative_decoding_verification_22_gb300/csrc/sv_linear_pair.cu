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
//  * Warp 8: TMA of its CTA; warp 9: products, in the first CTA of the pair alone.
//  * The columns of a tile are chosen so that the tiles fill whole waves.
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
  int kblocks, stages;
  int bf16, fast;              // fast: 16-byte accesses of the output's rows
  int fast_res, fast_bias;
};

struct Ctl {
  uint64_t full[kMaxStages], empty[kMaxStages];
  uint64_t tfull[2], tempty[2];
  uint64_t teardown;
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
// Arrives on the barrier at this offset in both CTAs when the products issued so
// far have completed.
__device__ __forceinline__ void commit_pair(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 "
      "[%0], %1;" ::"r"(bar),
      "h"(static_cast<uint16_t>(3))
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
// Values of 32 consecutive elements, zero beyond n of them.
__device__ __forceinline__ void load_row32(const void *p, int64_t at, int n, int dtype, bool fast,
                                           float *v) {
  if (fast && n >= 32) {
    if (dtype == SV_FP32) {
      const float4 *q = reinterpret_cast<const float4 *>(static_cast<const float *>(p) + at);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float4 f = q[i];
        v[4 * i] = f.x, v[4 * i + 1] = f.y, v[4 * i + 2] = f.z, v[4 * i + 3] = f.w;
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
            f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&w[j]));
          else
            f = __half22float2(*reinterpret_cast<const __half2 *>(&w[j]));
          v[8 * i + 2 * j] = f.x;
          v[8 * i + 2 * j + 1] = f.y;
        }
      }
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = i < n ? load_any(p, at + i, dtype) : 0.0f;
}
__device__ __forceinline__ void store_row32(void *p, int64_t at, int n, int dtype, bool fast,
                                            const float *v) {
  if (fast && n >= 32) {
    if (dtype == SV_FP32) {
      float4 *q = reinterpret_cast<float4 *>(static_cast<float *>(p) + at);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        q[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
    } else {
      uint4 *q = reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p) + at);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float a = v[8 * i + 2 * j], b = v[8 * i + 2 * j + 1];
          if (dtype == SV_BF16) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
            w[j] = *reinterpret_cast<const uint32_t *>(&h);
          } else {
            const __half2 h = __floats2half2_rn(a, b);
            w[j] = *reinterpret_cast<const uint32_t *>(&h);
          }
        }
        q[i] = make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 32; ++i)
    if (i < n) store_any(p, at + i, v[i], dtype);
}
template <int kAct>
__device__ __forceinline__ void activate32(float *v) {
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = activate<kAct>(v[i]);
}
__device__ __forceinline__ void activate32(float *v, int act) {
  switch (act) {
    case SV_ACT_RELU: activate32<SV_ACT_RELU>(v); break;
    case SV_ACT_GELU: activate32<SV_ACT_GELU>(v); break;
    case SV_ACT_GELU_TANH: activate32<SV_ACT_GELU_TANH>(v); break;
    case SV_ACT_SILU: activate32<SV_ACT_SILU>(v); break;
    default: break;
  }
}

// Tiles in the order of the pairs: bands of `group` row tiles, within a band
// column by column, so that the tiles that run at once share rows and columns.
__device__ __forceinline__ void place(const Args &a, int tile, int &tr, int &tc) {
  const int band = tile / (a.group * a.col_tiles), in = tile - band * a.group * a.col_tiles;
  const int rows = min(a.group, a.row_tiles - band * a.group);
  tr = band * a.group + in % rows;
  tc = in / rows;
}

template <bool kGated>
__global__ void __launch_bounds__(kThreads, 1) __cluster_dims__(2, 1, 1)
    linear_pair_kernel(const __grid_constant__ CUtensorMap tmX,
                       const __grid_constant__ CUtensorMap tmW,
                       const __grid_constant__ CUtensorMap tmU, const __grid_constant__ Args args) {
  const LinearParams &p = args.p;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  Ctl *ctl = reinterpret_cast<Ctl *>(smem_raw + (base - raw) + kMaxStages * kStage);
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const int rank = static_cast<int>(lin_cluster_rank());
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
  lin_cluster_sync();  // the barriers of both CTAs are set up
  pdl_wait();
  pdl_launch_dependents();

  const int first = blockIdx.x / 2, step = gridDim.x / 2;
  const int tiles = args.row_tiles * args.col_tiles;
  const int half = args.bn / 2;                   // weight rows that a CTA loads
  const int cols = kGated ? half : args.bn;       // output columns of a tile

  if (warp < kEpiWarps) {
    // ---------------- epilogue ----------------
    const int row = (warp & 3) * 32 + lane;
    const uint32_t tacc = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const uint32_t tempty0 = lin_remote(smem_u32(&ctl->tempty[0]), 0);
    uint32_t it = 0;
    bool ok = true;
    for (int tile = first; tile < tiles && ok; tile += step, ++it) {
      int tr, tc;
      place(args, tile, tr, tc);
      const uint32_t slot = it & 1;
      if (!(ok = lin_wait(smem_u32(&ctl->tfull[slot]), it >> 1 & 1, ab))) break;
      tc_fence_after();
      const int64_t m = static_cast<int64_t>(tr) * 256 + rank * kLanes + row;
      const bool live = m < p.M;
      for (int c = (warp >> 2) * 32; c < cols; c += 64) {
        const int64_t n = static_cast<int64_t>(tc) * cols + c;
        const int in = static_cast<int>(min(p.N - n, static_cast<int64_t>(min(32, cols - c))));
        if (in <= 0) break;
        uint32_t x[32], u[kGated ? 32 : 1];
        tmem_ld32(tacc + slot * 256 + c, x);
        if (kGated) tmem_ld32(tacc + slot * 256 + half + c, u);
        float b[32];
        if (p.bias) load_row32(p.bias, n, in, p.dtype, args.fast_bias, b);
        tmem_ld_wait();
        tmem_reg_fence32(x);
        if (kGated) tmem_reg_fence32(u);
        float y[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) y[i] = __uint_as_float(x[i]);
        if (p.bias) {
#pragma unroll
          for (int i = 0; i < 32; ++i) y[i] += b[i];
        }
        activate32(y, p.act);
        if (kGated) {
          if (p.bias_u) {
            load_row32(p.bias_u, n, in, p.dtype, args.fast_bias, b);
#pragma unroll
            for (int i = 0; i < 32; ++i) y[i] *= __uint_as_float(u[i]) + b[i];
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) y[i] *= __uint_as_float(u[i]);
          }
        }
        if (live) {
          if (p.res) {
            load_row32(p.res, m * p.rs + n, in, p.out_dtype, args.fast_res, b);
#pragma unroll
            for (int i = 0; i < 32; ++i) y[i] += b[i];
          }
          store_row32(p.out, m * p.os + n, in, p.out_dtype, args.fast, y);
        }
        __syncwarp();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) lin_arrive_remote(tempty0 + slot * 8);
      __syncwarp();
    }
  } else if (warp == kLoadWarp) {
    // ---------------- TMA ----------------
    const uint64_t policy = policy_evict_normal();
    const CUtensorMap *tmB = kGated && rank ? &tmU : &tmW;
    const uint32_t full0 = lin_remote(smem_u32(&ctl->full[0]), 0);
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int tile = first; tile < tiles && ok; tile += step) {
      int tr, tc;
      place(args, tile, tr, tc);
      const int m0 = tr * 256 + rank * kLanes;
      const int n0 = kGated ? tc * half : tc * args.bn + rank * half;
      for (int kb = 0; kb < args.kblocks; ++kb) {
        if (!(ok = lin_wait(smem_u32(&ctl->empty[stage]), phase ^ 1u, ab))) break;
        if (lane == 0) {
          // the first CTA's barrier counts the bytes of both
          if (rank == 0)
            mbar_arrive_expect_tx(smem_u32(&ctl->full[stage]), 2 * (kLanes + half) * 128);
          const uint32_t at = base + stage * kStage, full = full0 + stage * 8;
          load_pair(at, &tmX, kb * kLinBlk, m0, full, policy);
          load_pair(at + kLanes * 128, tmB, kb * kLinBlk, n0, full, policy);
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
    int stage = 0;
    uint32_t phase = 0, it = 0;
    bool ok = true;
    for (int tile = first; tile < tiles && ok; tile += step, ++it) {
      const uint32_t slot = it & 1;
      if (!(ok = lin_wait<true>(smem_u32(&ctl->tempty[slot]), (it >> 1 & 1) ^ 1u, ab))) break;
      tc_fence_after();
      for (int kb = 0; kb < args.kblocks; ++kb) {
        if (!(ok = lin_wait<true>(smem_u32(&ctl->full[stage]), phase, ab))) break;
        tc_fence_after();
        if (elect_one()) {
          const uint32_t at = base + stage * kStage;
          const uint64_t ad = sw128_desc(at), bd = sw128_desc(at + kLanes * 128);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            umma_pair(tmem + slot * 256, ad + 2u * k, bd + 2u * k, idesc, kb > 0 || k > 0);
          commit_pair(smem_u32(&ctl->empty[stage]));
          if (kb == args.kblocks - 1) commit_pair(smem_u32(&ctl->tfull[slot]));
        }
        __syncwarp();
        if (++stage == args.stages) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    if (elect_one()) commit_pair(smem_u32(&ctl->teardown));
    __syncwarp();
  }

  // ---------------- teardown ----------------
  // The products are done (their commit arrives in both CTAs); a copy can be in
  // flight only after a role gave up, and then on a barrier of the other CTA: it
  // is given a millisecond, a thousand times what it takes.
  if (warp == kLoadWarp) {
    const int never = 0;
    if (lane == 0) {
      mbar_wait(smem_u32(&ctl->teardown), 0u, kLinCleanupNs, &never);
      if (*const_cast<volatile int *>(&ctl->abort)) {
        const uint64_t t0 = globaltimer();
        while (globaltimer() - t0 < 1000000) {
        }
      }
    }
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  lin_cluster_sync();
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
  args.stages = kMaxStages;
  const int pairs = h.num_sms / 2;
  const int64_t row_tiles = (P.M + 255) / 256;
  // Columns of a tile: whole waves of tiles, each of the time of its columns (and
  // of 16 more for what a tile takes by itself).
  int64_t best = INT64_MAX, col_tiles = 0;
  for (int bn = 256; bn >= 64; bn -= 32) {
    const int cols = kGated ? bn / 2 : bn;
    const int64_t ct = (P.N + cols - 1) / cols;
    const int64_t time = (row_tiles * ct + pairs - 1) / pairs * (bn + 16);
    if (time < best) {
      best = time;
      args.bn = bn;
      col_tiles = ct;
    }
  }
  if (row_tiles * col_tiles > (1 << 30)) return SV_ERR_SHAPE;
  args.row_tiles = static_cast<int>(row_tiles);
  args.col_tiles = static_cast<int>(col_tiles);
  args.group = static_cast<int>(row_tiles < 8 ? row_tiles : 8);
  const int es = P.out_dtype == SV_FP32 ? 4 : 2;
  auto wide = [](const void *p, int64_t stride_bytes, int64_t rows) {
    return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && (rows <= 1 || stride_bytes % 16 == 0);
  };
  args.fast = wide(P.out, P.os * es, P.M);
  args.fast_res = wide(P.res, P.rs * es, P.M);
  args.fast_bias = wide(P.bias, 0, 1) && wide(P.bias_u, 0, 1);
  CUtensorMap x, w, u;
  if (!lin_encode(&x, P.x, P.xs, P.K, P.M, kLanes) ||
      !lin_encode(&w, P.w, P.ws, P.K, P.N, args.bn / 2) ||
      !lin_encode(&u, kGated ? P.wu : P.w, kGated ? P.wus : P.ws, P.K, P.N, args.bn / 2))
    return SV_ERR_CUDA;
  cudaError_t e = cudaFuncSetAttribute(linear_pair_kernel<kGated>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
  if (e != cudaSuccess) return SV_ERR_CUDA;
  const int64_t tiles = row_tiles * col_tiles;
  const int grid = 2 * static_cast<int>(tiles < pairs ? tiles : pairs);
  e = launch_chained(linear_pair_kernel<kGated>, dim3(grid), dim3(kThreads), kSmemBytes, stream, x,
                     w, u, args);
  return e == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}

}  // namespace

int launch_linear_pair(const spec_target &h, const LinearParams &P, cudaStream_t stream) {
  return P.wu ? launch<true>(h, P, stream) : launch<false>(h, P, stream);
}

}  // namespace sv
