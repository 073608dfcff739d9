// sv_linear_few.cu -- products with an epilogue for few rows of x (up to 128):
// the weight is streamed once through the tensor cores.
//
//  * The weight's rows are the 128 lanes of a tile, x's rows its columns
//    (padded to 16), so nothing but the weight costs bytes.  Gated: 64 rows of
//    each of the two weights, so that one tile holds both factors of 64
//    columns of the output.
//  * A cluster of up to eight CTAs shares a tile, each takes a part of K; the
//    parts meet in distributed shared memory, where each CTA adds some of the
//    columns in the order of K (repeatable, no scratch, no second launch) and
//    stores them.  The adding of a tile runs beside the next one's products.
//  * Warps 0-7 (0-15 from 33 rows on): sums and epilogue; then one each for TMA and
//    for the products.
//
// What bounds it (times of kernels in a CUDA graph): the bytes of the weight and about
// 4 us of start, first load and exchange.  5 x 4096 x 4096 takes 9.3 us (its bytes
// 5.0), 5 x 14336 x 4096 gated 39.4 (34.6), 20 x 28672 x 8192 gated 140.8 (138.7).  With
// many rows x's blocks, which every tile reads again from L2, and the epilogue count
// too: 64 x 4096 x 4096 10.4, 128 with a residual 12.6.  The epilogue's code is short
// because a tile that is a CTA's only one waits for it: with each activation and type
// unrolled over a thread's elements the last case took 21.  Parts of sums that went by
// plain remote stores and one release each took 105 us for the 5-row gated weight at
// eight CTAs a tile, 51 as stores that count their bytes; taking K from another place in
// each tile, so that not all read the same rows of x, made the first case 10% slower.
#include "sv_linear_tc.cuh"

namespace sv {
namespace {

// Warps of the epilogue: more of them for wider tiles (128 x 16384 x 64 takes 9.5 us
// with sixteen, 12.5 with eight), fewer for narrow ones, whose columns are few (5 x 4096 x
// 4096 9.0 us with eight, 9.3 with sixteen; 32 x 16384 x 64 5.6 and 5.0, but 32 x 1024 x
// 4096 6.0 and 6.3).
template <int kCols>
constexpr int epi_warps() { return kCols <= 32 ? 8 : 16; }
template <int kCols>
constexpr int threads() { return 32 * (epi_warps<kCols>() + 2); }
constexpr int kLanes = 128;
constexpr int kMaxSplit = 8;
constexpr int kMaxStages = 12;

struct Args {
  LinearParams p;
  int *status;
  uint64_t limit_ns;
  int bn, tiles, split, kblocks, stages;
  int bufs;  // for parts of sums: 1 or 2
  int per;   // columns whose parts a CTA adds, a multiple of four
  int bf16;
};

struct Ctl {
  uint64_t full[kMaxStages], empty[kMaxStages];
  uint64_t tfull[2], tempty[2];
  uint64_t xfull[2], xempty[2];
  uint64_t teardown;
  uint32_t tmem;
  int abort, issued, consumed;
};

// K blocks of a stage
template <int kCols>
constexpr int stage_blocks() { return kCols == 64 ? 2 : 1; }
template <int kCols>
constexpr int stage_bytes() { return stage_blocks<kCols>() * (kLanes + kCols) * 128; }

template <int kCols, bool kGated>
__global__ void __launch_bounds__(threads<kCols>(), 1)
    linear_few_kernel(const __grid_constant__ CUtensorMap tmW,
                      const __grid_constant__ CUtensorMap tmU,
                      const __grid_constant__ CUtensorMap tmX, const __grid_constant__ Args args) {
  constexpr int kEpiWarps = epi_warps<kCols>(), kLoadWarp = kEpiWarps, kMmaWarp = kEpiWarps + 1;
  constexpr int kKb = stage_blocks<kCols>(), kStage = stage_bytes<kCols>();
  constexpr int kRows = kGated ? 64 : 128;  // columns of the output in a tile
  const LinearParams &p = args.p;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t *smem = smem_raw + (base - raw);
  float *parts = reinterpret_cast<float *>(smem + args.stages * kStage);
  const int M = static_cast<int>(p.M);
  const int per = args.per;  // columns that a CTA adds
  Ctl *ctl = reinterpret_cast<Ctl *>(smem + args.stages * kStage + args.bufs * args.split * per * kLanes * 4);
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const LinAbort ab{args.status, args.limit_ns, &ctl->abort};

  if (tid == 0) {
    for (int i = 0; i < args.stages; ++i) {
      mbar_init(smem_u32(&ctl->full[i]), 1);
      mbar_init(smem_u32(&ctl->empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&ctl->tfull[i]), 1);
      mbar_init(smem_u32(&ctl->tempty[i]), kEpiWarps);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&ctl->xfull[i]), 1);
      mbar_init(smem_u32(&ctl->xempty[i]), kEpiWarps * args.split);
    }
    mbar_init(smem_u32(&ctl->teardown), 1);
    ctl->abort = ctl->issued = ctl->consumed = 0;
    mbar_fence_init();
  }
  const int rank = args.split > 1 ? static_cast<int>(lin_cluster_rank()) : 0;
  const int first = blockIdx.x / args.split, step = gridDim.x / args.split;
  const int kb0 = static_cast<int>(static_cast<int64_t>(args.kblocks) * rank / args.split);
  const int kb1 = static_cast<int>(static_cast<int64_t>(args.kblocks) * (rank + 1) / args.split);
  if (warp == kLoadWarp && lane == 0) {
    // The first blocks of the weight come into L2 while what precedes this kernel
    // ends (L2 is where all writes meet, so it does not matter who wrote them).
    for (int kb = kb0; kb < min(kb1, kb0 + args.stages * kKb); ++kb) {
      lin_prefetch(&tmW, kb * kLinBlk, first * kRows);
      if (kGated) lin_prefetch(&tmU, kb * kLinBlk, first * kRows);
    }
    tma_prefetch_desc(&tmX);
  }
  if (warp == kMmaWarp) {
    tmem_alloc(smem_u32(&ctl->tmem), 2 * kCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, ctl->tmem, 0);
  if (args.split > 1) lin_cluster_sync();  // the barriers of all CTAs are set up
  pdl_wait();
  pdl_launch_dependents();

  if (warp < kEpiWarps) {
    // ---------------- sums and epilogue ----------------
    const int row = tid & 127;  // lane of tensor memory
    const uint32_t tacc = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    uint32_t it = 0;
    bool ok = true;
    for (int tile = first; tile < args.tiles && ok; tile += step, ++it) {
      const uint32_t slot = it & 1, phase = it >> 1 & 1;
      if (!(ok = lin_wait(smem_u32(&ctl->tfull[slot]), phase, ab))) break;
      tc_fence_after();
      // The parts of the sum go to a buffer (two in turn where there is room), as
      // [part][column / 4][lane][column % 4].  Column c goes to CTA c / per.
      const uint32_t xslot = args.bufs == 2 ? slot : 0, xphase = args.bufs == 2 ? phase : it & 1;
      if (!(ok = lin_wait<true>(smem_u32(&ctl->xempty[xslot]), xphase ^ 1u, ab))) break;
      float *const buf = parts + xslot * args.split * per * kLanes;
      const uint32_t bar = smem_u32(&ctl->xfull[xslot]);
      const int mine = min(per, M - rank * per);
      const int fours = mine > 0 ? (mine + 3) / 4 : 0;
      if (tid == 0) mbar_arrive_expect_tx(bar, fours * args.split * kLanes * 16);
      const uint32_t own = smem_u32(buf + rank * per * kLanes + row * 4);
      {
        // each four warps take a share of the chunks of 16 columns
        constexpr int kShares = kEpiWarps / 4;
        const int chunks = (M + 15) / 16, share = warp >> 2;
        const int c_end = min(chunks * (share + 1) / kShares * 16, M);
        int c = chunks * share / kShares * 16, q = c / per, left = per - (c - q * per);
        uint32_t at = lin_remote(own, q) + (per - left) * kLanes * 4, to = lin_remote(bar, q);
#pragma unroll 1
        for (; c < c_end; c += 16) {
          uint32_t x[16];
          tmem_ld16(tacc + slot * kCols + c, x);
          tmem_ld_wait();
          tmem_reg_fence(x);
#pragma unroll
          for (int e = 0; e < 16; e += 4) {
            if (c + e >= M) break;
            if (left == 0) {
              left = per;
              at = lin_remote(own, ++q);
              to = lin_remote(bar, q);
            }
            lin_store_remote(at, x + e, to);
            at += kLanes * 16;
            left -= 4;
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&ctl->tempty[slot]));
      __syncwarp();
      // A thread finishes column n of the output, four rows of x at a time, one in
      // kStep; what it adds to 16 of them is loaded while their parts arrive.
      constexpr int kStep = 32 * kEpiWarps / kRows, kFours = 4;
      const int r = row % kRows;
      const int64_t n = static_cast<int64_t>(tile) * kRows + r;
      const bool in = n < p.N;
      const float b = in && p.bias ? load_any(p.bias, n, p.dtype) : 0.0f;
      const float bu = kGated && in && p.bias_u ? load_any(p.bias_u, n, p.dtype) : 0.0f;
      const bool wide_out = p.out_dtype == SV_FP32, bf_out = p.out_dtype == SV_BF16;
      const int shift = wide_out ? 2 : 1;
      const int f_first = tid / kRows;
      const int64_t m_first = rank * per + 4 * f_first;
      const int64_t os = p.os << shift, rs = p.rs << shift;  // in bytes
      char *out = static_cast<char *>(p.out) + ((m_first * p.os + n) << shift);
      const char *from = static_cast<const char *>(p.res) + ((m_first * p.rs + n) << shift);
      uint32_t res[4 * kFours];  // as they lie in memory
      auto load_res = [&](int f0) {
        const int rows = mine - 4 * f0;
#pragma unroll
        for (int i = 0; i < kFours; ++i) {
          const char *at = from + 4 * i * kStep * rs;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            res[4 * i + e] = 0;
            if (4 * i * kStep + e < rows)
              res[4 * i + e] = wide_out ? *reinterpret_cast<const uint32_t *>(at)
                                        : *reinterpret_cast<const uint16_t *>(at);
            at += rs;
          }
        }
        from += 4 * kFours * kStep * rs;
      };
      auto widen = [&](uint32_t x) {
        if (wide_out) return __uint_as_float(x);
        return bf_out ? __uint_as_float(x << 16)
                      : __half2float(__ushort_as_half(static_cast<unsigned short>(x)));
      };
      if (p.res && in) load_res(f_first);
      if (!(ok = lin_wait<true>(bar, xphase, ab))) break;
      const float4 *in_parts = reinterpret_cast<const float4 *>(buf) + r;
      for (int f0 = f_first; f0 < fours && in; f0 += kFours * kStep) {
#pragma unroll
        for (int i = 0; i < kFours; ++i) {
          const int f = f0 + i * kStep, rows = mine - 4 * f;
          if (rows <= 0) break;
          float y[4] = {}, u[4] = {};
          const float4 *part = in_parts + f * kLanes;
          for (int s = 0; s < args.split; ++s, part += per / 4 * kLanes) {
            const float4 a = part[0];
            y[0] += a.x, y[1] += a.y, y[2] += a.z, y[3] += a.w;
            if (kGated) {
              const float4 c = part[64];
              u[0] += c.x, u[1] += c.y, u[2] += c.z, u[3] += c.w;
            }
          }
          const float4 a4 = activate4(make_float4(y[0] + b, y[1] + b, y[2] + b, y[3] + b), p.act);
          y[0] = a4.x, y[1] = a4.y, y[2] = a4.z, y[3] = a4.w;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if (kGated) y[e] *= u[e] + bu;
            if (p.res) y[e] += widen(res[4 * i + e]);
          }
          char *at = out;
          if (wide_out) {
#pragma unroll
            for (int e = 0; e < 4; ++e, at += os)
              if (e < rows) *reinterpret_cast<float *>(at) = y[e];
          } else {
            uint32_t two[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              if (bf_out) {
                const __nv_bfloat162 h = __floats2bfloat162_rn(y[2 * e], y[2 * e + 1]);
                two[e] = *reinterpret_cast<const uint32_t *>(&h);
              } else {
                const __half2 h = __floats2half2_rn(y[2 * e], y[2 * e + 1]);
                two[e] = *reinterpret_cast<const uint32_t *>(&h);
              }
            }
#pragma unroll
            for (int e = 0; e < 4; ++e, at += os)
              if (e < rows)
                *reinterpret_cast<uint16_t *>(at) =
                    static_cast<uint16_t>(e & 1 ? two[e / 2] >> 16 : two[e / 2]);
          }
          out += 4 * kStep * os;
        }
        if (p.res && f0 + kFours * kStep < fours) load_res(f0 + kFours * kStep);
      }
      __syncwarp();
      if (lane < args.split) lin_arrive_remote(lin_remote(smem_u32(&ctl->xempty[xslot]), lane));
      __syncwarp();
    }
  } else if (warp == kLoadWarp) {
    // ---------------- TMA ----------------
    const uint64_t first_out = policy_evict_first(), keep = policy_evict_normal();
    int stage = 0, issued = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int tile = first; tile < args.tiles && ok; tile += step) {
      for (int kb = kb0; kb < kb1; kb += kKb) {
        if (!(ok = lin_wait(smem_u32(&ctl->empty[stage]), phase ^ 1u, ab))) break;
        if (lane == 0) {
          const uint32_t full = smem_u32(&ctl->full[stage]);
          const int blocks = min(kKb, kb1 - kb);
          mbar_arrive_expect_tx(full, blocks * (kLanes + args.bn) * 128);
          for (int j = 0; j < blocks; ++j) {
            const uint32_t at = base + stage * kStage + j * (kLanes + kCols) * 128;
            const int k = (kb + j) * kLinBlk;
            tma_load_2d(at, &tmW, k, tile * kRows, full, first_out);
            if (kGated) tma_load_2d(at + 64 * 128, &tmU, k, tile * kRows, full, first_out);
            tma_load_2d(at + kLanes * 128, &tmX, k, 0, full, keep);
          }
          ctl->issued = ++issued;
        }
        __syncwarp();
        if (++stage == args.stages) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
  } else {
    // ---------------- products ----------------
    const uint32_t idesc = idesc_16(args.bf16, kLanes, args.bn, false);
    int stage = 0, consumed = 0;
    uint32_t phase = 0, it = 0;
    bool ok = true;
    for (int tile = first; tile < args.tiles && ok; tile += step, ++it) {
      const uint32_t slot = it & 1;
      if (!(ok = lin_wait(smem_u32(&ctl->tempty[slot]), (it >> 1 & 1) ^ 1u, ab))) break;
      tc_fence_after();
      for (int kb = kb0; kb < kb1; kb += kKb) {
        if (!(ok = lin_wait(smem_u32(&ctl->full[stage]), phase, ab))) break;
        if (lane == 0) ctl->consumed = ++consumed;
        tc_fence_after();
        if (elect_one()) {
          const int blocks = min(kKb, kb1 - kb);
          for (int j = 0; j < blocks; ++j) {
            const uint32_t at = base + stage * kStage + j * (kLanes + kCols) * 128;
            const uint64_t ad = sw128_desc(at), bd = sw128_desc(at + kLanes * 128);
#pragma unroll
            for (int k = 0; k < 4; ++k)
              umma_16(tmem + slot * kCols, ad + 2u * k, bd + 2u * k, idesc,
                      kb > kb0 || j > 0 || k > 0);
          }
          umma_commit(smem_u32(&ctl->empty[stage]));
          if (kb + kKb >= kb1) umma_commit(smem_u32(&ctl->tfull[slot]));
        }
        __syncwarp();
        if (++stage == args.stages) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    if (elect_one()) {
      umma_commit(smem_u32(&ctl->teardown));
      const int never = 0;
      mbar_wait(smem_u32(&ctl->teardown), 0u, kLinCleanupNs, &never);
    }
    __syncwarp();
  }

  // ---------------- teardown ----------------
  tc_fence_before();
  __syncthreads();
  if (warp == kLoadWarp && lane == 0) {
    // only after an abort can copies still be in flight
    const int never = 0;
    for (int i = ctl->consumed; i < ctl->issued; ++i)
      mbar_wait(smem_u32(&ctl->full[i % args.stages]),
                static_cast<uint32_t>((i / args.stages) & 1), kLinCleanupNs, &never);
  }
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 2 * kCols);
  }
  if (args.split > 1) lin_leave(&ctl->abort, args.split);
}

template <int kCols, bool kGated>
int launch(const spec_target &h, const LinearParams &P, cudaStream_t stream) {
  constexpr int kRows = kGated ? 64 : 128;
  if (!lin_encode_fn()) return SV_ERR_CUDA;
  Args args{};
  args.p = P;
  args.status = h.status;
  args.limit_ns = h.wait_limit_ns;
  args.bf16 = P.dtype == SV_BF16;
  args.bn = static_cast<int>((P.M + 15) / 16 * 16);
  args.tiles = static_cast<int>((P.N + kRows - 1) / kRows);
  args.kblocks = static_cast<int>((P.K + kLinBlk - 1) / kLinBlk);
  // CTAs of a tile, by the K blocks that the longest-working one takes, and two more a
  // tile for its exchange: waves of tiles over the clusters of a size that run at once
  // (the product in 8 bits asked for these: one CTA an SM, as here).
  int64_t best = INT64_MAX;
  int clusters = 1;
  for (int s = 1; s <= kMaxSplit && s <= args.kblocks; ++s) {
    const int most = s == 1 ? h.num_sms : h.clusters[s];
    if (most < 1) continue;
    const int c = args.tiles < most ? args.tiles : most;
    const int64_t time =
        static_cast<int64_t>((args.tiles + c - 1) / c) * ((args.kblocks + s - 1) / s + 2);
    if (time < best) {
      best = time;
      args.split = s;
      clusters = c;
    }
  }
  const int per = ((static_cast<int>(P.M) + args.split - 1) / args.split + 3) / 4 * 4;
  args.per = per;
  args.bufs = P.M <= 32 ? 2 : 1;
  const int fixed =
      1024 + args.bufs * args.split * per * kLanes * 4 + static_cast<int>(sizeof(Ctl));
  // Where a CTA's part of the weight is short, half the ring leaves shared memory to the
  // next kernel of a stream, which starts and reads ahead while this one ends: the norm
  // behind a product (gated projections, product and norm of 5 x 4096 in bf16, F 4096, take
  // 26.4 us in place of 27.9), but not this kernel again, as the registers hold one CTA an
  // SM (5 x 4096 x 4096 9.05 us against 9.21; 5 x 1024 x 4096 5.95 against 5.72). From 17
  // rows on x's blocks and the parts of sums take half of that half, and the whole ring is
  // better (32 x 4096 x 4096: 9.6 us against 10.3, 32 x 6144 x 4096 11.9 against 13.9,
  // layers of 32 rows 28.4 against 29.7); so it is for most long parts (16 x 5120 x 8192
  // 16.9 us against 18.3, 5 x 4096 x 14336 21.0 against 21.7, 5 x 14336 x 4096, gated, 39.0
  // against 38.2).
  const int64_t part = static_cast<int64_t>(args.tiles) * args.kblocks * kLanes * 128 /
                       (static_cast<int64_t>(clusters) * args.split);
  const int room = P.M <= 16 && part <= 512 * 1024 ? h.smem_optin / 2 - 1024 : h.smem_optin;
  args.stages = (room - fixed) / stage_bytes<kCols>();
  if (args.stages > kMaxStages) args.stages = kMaxStages;
  if (args.stages < 2) return SV_ERR_CUDA;
  const int smem = fixed + args.stages * stage_bytes<kCols>();
  CUtensorMap w, u, x;
  if (!lin_encode(&w, P.w, P.ws, P.K, P.N, kRows) ||
      !lin_encode(&u, kGated ? P.wu : P.w, kGated ? P.wus : P.ws, P.K, P.N, kRows) ||
      !lin_encode(&x, P.x, P.xs, P.K, P.M, args.bn))
    return SV_ERR_CUDA;
  cudaError_t e = cudaFuncSetAttribute(linear_few_kernel<kCols, kGated>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, h.smem_optin);
  if (e != cudaSuccess) return SV_ERR_CUDA;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = args.split;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(clusters * args.split);
  cfg.blockDim = dim3(threads<kCols>());
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  e = cudaLaunchKernelEx(&cfg, linear_few_kernel<kCols, kGated>, w, u, x, args);
  return e == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}

template <bool kGated>
int launch_cols(const spec_target &h, const LinearParams &P, cudaStream_t stream) {
  if (P.M <= 16) return launch<16, kGated>(h, P, stream);
  if (P.M <= 32) return launch<32, kGated>(h, P, stream);
  if (P.M <= 64) return launch<64, kGated>(h, P, stream);
  return launch<128, kGated>(h, P, stream);
}

}  // namespace

int launch_linear_few(const spec_target &h, const LinearParams &P, cudaStream_t stream) {
  return P.wu ? launch_cols<true>(h, P, stream) : launch_cols<false>(h, P, stream);
}

}  // namespace sv
