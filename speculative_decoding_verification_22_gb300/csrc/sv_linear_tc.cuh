// sv_linear_tc.cuh -- pieces that the tensor-core forms of the products share:
// bounded waits, accesses across a cluster, and tensor maps.
#pragma once

#include <cudaTypedefs.h>

#include "sv_linear.cuh"
#include "sv_tmem.cuh"

namespace sv {

constexpr int kLinBlk = 64;  // K elements of a block: 128 bytes, one swizzled row
constexpr uint64_t kLinCleanupNs = 2000000000ull;

// State of a CTA that its roles give up by.
struct LinAbort {
  int *status;
  uint64_t limit_ns;
  int *flag;  // shared
};
__device__ __noinline__ inline bool lin_give_up(const LinAbort &a, uint64_t &since) {
  const uint64_t now = globaltimer();
  if (since == 0) since = now;
  const volatile int *flag = a.flag;
  if (!__any_sync(0xffffffffu, now - since >= a.limit_ns || *flag)) return false;
  if ((threadIdx.x & 31) == 0) {
    *const_cast<volatile int *>(a.flag) = 1;
    set_status(a.status, SV_ERR_TIMEOUT);
  }
  __syncwarp();
  return true;
}
// As mbar_try_wait, seeing also what other CTAs of the cluster wrote.
__device__ __forceinline__ bool mbar_try_wait_cluster(uint32_t bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.b32 %0, 1, 0, p;\n\t}"
      : "=r"(done)
      : "r"(bar), "r"(parity)
      : "memory");
  return done != 0;
}
// Waits on a barrier with the whole warp; false: the limit ran out, or another
// role gave up.
template <bool kCluster = false>
__device__ __forceinline__ bool lin_wait(uint32_t bar, uint32_t parity, const LinAbort &a) {
  auto there = [&]() {
    return __all_sync(0xffffffffu, kCluster ? mbar_try_wait_cluster(bar, parity)
                                            : mbar_try_wait(bar, parity));
  };
  if (there()) return true;
  uint64_t since = 0;
  while (true) {
    for (int i = 0; i < 16; ++i)
      if (there()) return true;
    if (lin_give_up(a, since)) return false;
  }
}

__device__ __forceinline__ void lin_cluster_sync() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t lin_cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// The address of another CTA's shared memory in the cluster, and accesses there.
__device__ __forceinline__ uint32_t lin_remote(uint32_t smem_addr, uint32_t rank) {
  uint32_t at;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_addr), "r"(rank));
  return at;
}
// (the store counts its 16 bytes on a barrier of the same CTA, so that it needs no
// fence and no arrival of its own)
__device__ __forceinline__ void lin_store_remote(uint32_t at, const uint32_t *x, uint32_t bar) {
  asm volatile(
      "st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1, %2, %3, %4}, [%5];"
      ::"r"(at), "r"(x[0]), "r"(x[1]), "r"(x[2]), "r"(x[3]), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void lin_arrive_remote(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar)
               : "memory");
}

// Brings a box into L2.
__device__ __forceinline__ void lin_prefetch(const CUtensorMap *m, int32_t c0, int32_t c1) {
  asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global [%0, {%1, %2}];" ::"l"(
                   reinterpret_cast<uint64_t>(m)),
               "r"(c0), "r"(c1)
               : "memory");
}

// The end of a cluster of `ctas`, for all threads, after a __syncthreads: nobody goes
// while another may still write to it or complete a copy on its barriers.  Without a
// timeout everything on its way has been waited for; after one (in whichever CTA) what
// may still be on its way is given a millisecond, a thousand times what it takes.
__device__ __forceinline__ void lin_leave(int *abort, uint32_t ctas) {
  volatile int *gave_up = abort;
  if (threadIdx.x < ctas && *gave_up)
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(lin_remote(smem_u32(abort), threadIdx.x)),
                 "r"(1)
                 : "memory");
  lin_cluster_sync();
  if (*gave_up) {
    const uint64_t t0 = globaltimer();
    while (globaltimer() - t0 < 1000000) {
    }
    lin_cluster_sync();
  }
}

inline PFN_cuTensorMapEncodeTiled_v12000 lin_encode_fn() {
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
// 16-bit rows [rows, K]: boxes of `box` rows of 64 elements.  What lies past the
// rows or past K is read as zero.
inline bool lin_encode(CUtensorMap *map, const void *base, int64_t stride, int64_t K, int64_t rows,
                       int box) {
  if (rows <= 1) stride = (K + 7) / 8 * 8;  // (not looked at before)
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(K), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(stride) * 2};
  const cuuint32_t boxes[2] = {kLinBlk, static_cast<cuuint32_t>(box)};
  const cuuint32_t estr[2] = {1, 1};
  return lin_encode_fn()(map, CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, const_cast<void *>(base), dims,
                         strides, boxes, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                         CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// Rows that TMA can read: 16-byte aligned.
inline bool lin_rows_aligned(const void *p, int64_t stride, int64_t rows) {
  return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && (rows <= 1 || stride % 8 == 0);
}

// Launches of the forms; whether they take the call has been settled.
int launch_linear_few(const spec_target &h, const LinearParams &P, cudaStream_t stream);
int launch_linear_pair(const spec_target &h, const LinearParams &P, cudaStream_t stream);

}  // namespace sv
