// sv_attn.cu -- attention of new tokens over the pages: the form for every
// type, head size, page size and stride.
//
//   o = sum_j softmax_j(scale q . k_j) v_j over the keys that a token sees
//
// A warp takes one token and query head at a time (attend_row).  The path for
// what the tensor-core form does not take: fp32, head sizes above 128 or not a
// multiple of 8, page sizes that are not a power of two, odd alignments.  It is
// there for its results and far from any bound (64 single tokens over 512 to 2048,
// 8 cache heads of 256 in bf16: 5.4 ms, for bytes of 0.1): a lane walks its own
// key's elements one after another, the query heads of a cache head share nothing,
// and a sequence of one row is one warp's.
#include "sv_attn.cuh"

namespace sv {
namespace {

constexpr int kAnyWarps = 4;

template <class T>
__global__ void __launch_bounds__(32 * kAnyWarps)
    attention_any_kernel(const sv_attention_t a, int *status) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int b = blockIdx.y;
  pdl_wait();
  pdl_launch_dependents();
  bool bad;
  const SeqGeom s = seq_geom(a, b, &bad);
  if (bad && threadIdx.x == 0) set_status(status, SV_ERR_CACHE);
  const int64_t rows = static_cast<int64_t>(s.n) * a.Hq;
  for (int64_t r = static_cast<int64_t>(blockIdx.x) * kAnyWarps + warp; r < rows;
       r += static_cast<int64_t>(gridDim.x) * kAnyWarps) {
    const int i = static_cast<int>(r / a.Hq);
    attend_row<T>(a, s, b, i, static_cast<int>(r - static_cast<int64_t>(i) * a.Hq), lane,
                  status);
  }
}

}  // namespace

int launch_attention(const spec_target &h, const sv_attention_t &a, cudaStream_t stream) {
  const int tc = launch_attention_tc(h, a, stream);
  if (tc != kNotTaken) return tc;
  // enough blocks for every row of an even split of the tokens, at most a
  // few waves
  const int64_t want = (static_cast<int64_t>(a.T) * a.Hq + kAnyWarps - 1) / kAnyWarps;
  const int64_t cap = (16LL * h.num_sms + a.B - 1) / a.B;
  const dim3 grid(static_cast<unsigned>(want < cap ? want : cap), a.B), block(32 * kAnyWarps);
  cudaError_t e;
  switch (a.dtype) {
    case SV_BF16:
      e = launch_chained(attention_any_kernel<__nv_bfloat16>, grid, block, 0, stream, a, h.status);
      break;
    case SV_FP16:
      e = launch_chained(attention_any_kernel<__half>, grid, block, 0, stream, a, h.status);
      break;
    default:
      e = launch_chained(attention_any_kernel<float>, grid, block, 0, stream, a, h.status);
  }
  return e == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}

}  // namespace sv
