/*
 * spec_target.h -- C ABI of the operators that turn drafted tokens into the
 * final hidden states which spec_verify.h verifies: the serving side of one
 * layer of the target over a paged cache, on a GB300 (sm_103a).
 *
 *   residual RMS norm   -> 16/32-bit rows, or E4M3 with scales
 *   8-bit product       E4M3 x E4M3 with an fp32 scale per block of 128
 *   rotary + append     rotary positions; K and V written into cache pages
 *   attention           the new tokens of each sequence over its pages
 *
 * The target checks K+1 positions in one forward pass ("Speculative
 * Decoding: Two Models, One Voice", "The idea", step 2), which "works like a
 * tiny prefill" over the cache ("Speculative Decoding: Guess Several Tokens,
 * Check Them in One Pass", Step 1); a tree of drafts needs the tree's mask
 * (the same page, "Tree attention").  The pages give no code for these
 * steps; the formulas below are the common ones.
 *
 * Conventions: return values, error codes and ownership as in
 * spec_verify.h.  Every call takes the cudaStream_t it is enqueued on (NULL:
 * the legacy default stream), returns without synchronising, allocates
 * nothing and can be captured in a CUDA graph.  A handle belongs to the
 * device that was current when it was created and owns scratch that the
 * attention uses, so two calls on one handle that may overlap on the GPU (on
 * different streams) race; use one handle for each.  Outputs
 * are the same bit for bit when a call is repeated on the same inputs.
 * Strides are in elements; the innermost dimension is always dense.
 */
#ifndef SPEC_TARGET_H
#define SPEC_TARGET_H

#include "spec_verify.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element type FP16, beside SV_BF16, SV_FP32 and SV_FP8 of spec_verify.h. */
#define SV_FP16 3

/* Columns (and rows of a weight) that share one scale of the 8-bit product. */
#define SV_SCALE_BLOCK 128
#define SV_MAX_HEAD_DIM 256

typedef struct spec_target spec_target_t; /* opaque handle */

/* Creates a handle on the current CUDA device and allocates its scratch (a
 * fixed size, 44 MiB).  Errors: SV_ERR_ARG (null pointer), SV_ERR_ARCH,
 * SV_ERR_CUDA.  On error *out is set to NULL. */
int spec_target_create(spec_target_t **out);

/* Frees the handle (NULL is ignored); its calls must have finished. */
void spec_target_destroy(spec_target_t *h);

/* Synchronises `stream`, then returns and clears the handle's status word:
 * SV_OK, SV_ERR_CACHE (a slot, page, cache length or token range out of
 * bounds), SV_ERR_TOKEN (a tree's parent), SV_ERR_TIMEOUT (a bounded device-side wait ran out: the call's
 * outputs are not valid), or SV_ERR_CUDA if synchronisation failed. */
int spec_target_status(spec_target_t *h, void *stream);

/* Upper bound, in nanoseconds, of every device-side wait (default 1e9). */
int spec_target_set_wait_limit(spec_target_t *h, uint64_t limit_ns);

/* ---------------------------------------------------------------------------
 * Residual RMS norm.  For each row, with all arithmetic in fp32:
 *   h = x + residual            (h = x if residual is NULL)
 *   y = h / sqrt(mean(h^2) + eps) * weight
 * h is not rounded before the norm; residual_out receives it rounded once.
 *   x, residual   device, dtype, [rows, d] with row strides
 *   weight        device, dtype, [d]
 *   out           device, dtype, [rows, d]
 *   residual_out  device, dtype, [rows, d] or NULL; may be the residual or x
 *                 itself (in place), and out may be x
 *   dtype         SV_BF16, SV_FP16 or SV_FP32
 * Any d >= 1; rows of 16-byte alignment with d a multiple of 8 take 16-byte
 * loads.  rows == 0 is a no-op.  Errors: SV_ERR_ARG (null pointer, dtype,
 * eps negative or not finite, negative rows), SV_ERR_SHAPE (d < 1 or above
 * 2^20, a row stride below d), SV_ERR_ALIGN (a pointer not aligned to its
 * element), SV_ERR_CUDA. */
int spec_target_rms_norm(spec_target_t *h, const void *x, int64_t x_stride,
                         const void *residual, int64_t residual_stride, const void *weight,
                         float eps, int64_t rows, int64_t d, int32_t dtype, void *out,
                         int64_t out_stride, void *residual_out, int64_t residual_out_stride,
                         void *stream);

/* The same norm with y in 8 bits: per group of columns
 *   scale = max(max|y|, 1e-30) / 448,   out8 = E4M3(y * (1 / scale))
 * rounded to nearest even from the fp32 y.
 *   group   SV_SCALE_BLOCK: a scale for every 128 columns (the last group
 *           may be shorter), scale is fp32 [rows, ceil(d / 128)], what
 *           spec_target_matmul_fp8 reads; 0: one scale for the row, fp32
 *           [rows], what spec_verify_run_fp8 reads
 *   out8    device, E4M3 bytes [rows, d], dense
 * A group that holds a NaN or an infinity gets that as its scale, so its
 * product with anything is not finite.  Errors as above, SV_ERR_ARG for
 * another group. */
int spec_target_rms_norm_fp8(spec_target_t *h, const void *x, int64_t x_stride,
                             const void *residual, int64_t residual_stride, const void *weight,
                             float eps, int64_t rows, int64_t d, int32_t dtype, int32_t group,
                             void *out8, float *scale, void *residual_out,
                             int64_t residual_out_stride, void *stream);

/* ---------------------------------------------------------------------------
 * 8-bit product with block scales:
 *   out[m, n] = sum over blocks b of 128 columns of
 *       a_scale[m, b] * w_scale[n / 128, b] * sum_{k in b} a8[m, k] w8[n, k]
 *   a8       device, E4M3 bytes [M, K], dense
 *   a_scale  device, fp32 [M, ceil(K / 128)]
 *   w8       device, E4M3 bytes [N, K], dense (a linear layer's weight)
 *   w_scale  device, fp32 [ceil(N / 128), ceil(K / 128)]
 *   out      device, out_dtype (SV_BF16, SV_FP16, SV_FP32), [M, N] with row
 *            stride out_stride
 * The products of one block are summed by the tensor cores; the scaled
 * blocks are summed in fp32 with round to nearest.  M == 0 is a no-op.
 * Errors: SV_ERR_ARG, SV_ERR_SHAPE (K not a multiple of 16, or a size above
 * 2^24), SV_ERR_ALIGN (a8, w8 not 16-byte aligned, others not aligned to
 * their element), SV_ERR_CUDA; SV_ERR_TIMEOUT through the status word. */
int spec_target_matmul_fp8(spec_target_t *h, const void *a8, const float *a_scale,
                           const void *w8, const float *w_scale, int64_t M, int64_t N,
                           int64_t K, int32_t out_dtype, void *out, int64_t out_stride,
                           void *stream);

/* ---------------------------------------------------------------------------
 * Rotary positions.  The angle of position p and pair i is 2 pi p f[i], with
 * f in turns per position.  spec_target_rope_freqs fills f[0 .. rot_dim/2)
 * on the host (64 bits), and the magnitude m that cos and sin are multiplied
 * by (1 but for SV_ROPE_YARN).  With f0[i] = base^(-2i/rot_dim) / (2 pi):
 *   SV_ROPE_PLAIN   f = f0
 *   SV_ROPE_LINEAR  f = f0 / factor
 *   SV_ROPE_NTK     f0 of base * factor^(rot_dim / (rot_dim - 2))
 *   SV_ROPE_BANDED  t = clamp((L f0 - low) / (high - low), 0, 1),
 *                   f = (1 - t) f0 / factor + t f0: wavelengths above
 *                   L / low are stretched by factor, those below L / high kept
 *   SV_ROPE_YARN    a ramp t over the pair index, from 0 at the pair that
 *                   turns beta_fast times in L positions to 1 at the one that
 *                   turns beta_slow times (both rounded outwards):
 *                   f = t f0 / factor + (1 - t) f0, m = 0.1 ln(factor) + 1
 * Errors: SV_ERR_ARG (null pointer, unknown scaling, base <= 1, factor < 1,
 * or bad band limits), SV_ERR_SHAPE (rot_dim odd, < 2 or > 256). */
#define SV_ROPE_PLAIN 0
#define SV_ROPE_LINEAR 1
#define SV_ROPE_NTK 2
#define SV_ROPE_BANDED 3
#define SV_ROPE_YARN 4
typedef struct {
  int32_t rot_dim;
  int32_t scaling;
  double base;
  double factor;       /* LINEAR, NTK, BANDED, YARN                        */
  double original_len; /* L: BANDED, YARN                                  */
  double low, high;    /* BANDED                                           */
  double beta_fast, beta_slow; /* YARN                                     */
} sv_rope_t;
int spec_target_rope_freqs(const sv_rope_t *cfg, double *freqs, double *magnitude);

/* Rotates the queries and keys of T new tokens and writes K and V into their
 * cache slots, in one launch.  Of each head's D elements the first rot_dim
 * are rotated, as pairs (i, i + rot_dim/2) or, interleaved, (2i, 2i + 1):
 *   (a, b) -> m (a cos - b sin, a sin + b cos),
 * the others are copied.  The fraction of a turn p f is taken from the exact
 * product and rounded once, to fp32 (2^-25 of a turn at most), for positions and
 * turns up to 2^53.
 *   q, k, v     device, dtype (SV_BF16, SV_FP16, SV_FP32); token and head
 *               strides (they may be slices of one fused projection)
 *   positions   device, int64 [T] (a tree's nodes: the depth)
 *   slots       device, int64 [T]: page * page_size + offset; -1: K and V of
 *               this token are not written; another slot outside the cache
 *               is skipped and sets SV_ERR_CACHE
 *   freqs       device, fp64 [rot_dim / 2]
 *   q_out       device, dtype [T, Hq, D] with strides; may be q itself
 *   k_cache, v_cache  device, dtype [num_pages, page_size, Hkv, D] with page,
 *               token and head strides
 * T == 0 is a no-op.  Errors: SV_ERR_ARG, SV_ERR_SHAPE (D outside 1..256,
 * rot_dim odd or outside 0..D, more than 4096 heads, sizes), SV_ERR_ALIGN, SV_ERR_CUDA. */
typedef struct {
  const void *q, *k, *v;
  int64_t q_token, q_head, k_token, k_head, v_token, v_head;
  const int64_t *positions;
  const int64_t *slots;
  const double *freqs;
  void *q_out;
  int64_t qo_token, qo_head;
  void *k_cache, *v_cache;
  int64_t kc_page, kc_token, kc_head, vc_page, vc_token, vc_head;
  int64_t num_pages;
  int32_t page_size, T, Hq, Hkv, D, rot_dim, interleaved, dtype;
  float magnitude;
  int32_t pad;
} sv_rope_append_t;
int spec_target_rope_append(spec_target_t *h, const sv_rope_append_t *a, void *stream);

/* ---------------------------------------------------------------------------
 * Attention of new tokens over the pages.  Sequence b has the new tokens
 * q_start[b] .. q_start[b+1] - 1 (n of them), which are the last n of its
 * kv_len[b] cached tokens: their keys are in the cache already.  New token i
 * has index kv_len - n + i and sees the cached tokens j <= its index, with
 * window > 0 the last `window` of these, with a tree mask all j < kv_len - n
 * and those new tokens jj whose bit is set:
 *   o = sum_j softmax_j(scale q . k_j) v_j,  lse = log sum_j exp(scale q . k_j)
 * Query head h reads cache head h / (Hq / Hkv).  A token that sees nothing
 * gets o = 0 and lse = -inf; what is masked does not count even where the
 * cache holds NaN or infinities there.  Scores, their maximum, the sums and o
 * are fp32; on the tensor cores a weight is rounded to dtype before it
 * multiplies v_j, half a step of its value (2^-8 in bf16, 2^-11 in fp16, where
 * weights below 2^-21 of the row's largest are kept to 2^-32 of it).
 *   q          device, dtype [T, Hq, D], token and head strides
 *   k_cache, v_cache  as above
 *   page_table device, int32 [B, max_pages], row stride: page of the cached
 *              tokens page_size * i .. of sequence b
 *   q_start    device, int32 [B + 1], from 0 to T
 *   kv_len     device, int32 [B], at most max_pages * page_size
 *   tree_mask  device, int32 [T, tree_words] or NULL: bit jj % 32 of word
 *              jj / 32 of a new token's row says whether it sees new token
 *              jj of its sequence (further ones: no)
 *   out        device, dtype [T, Hq, D], token and head strides; apart from q
 *   lse        device, fp32 [T, Hq] or NULL
 * dtype: SV_BF16, SV_FP16 (tensor cores where D is a multiple of 8 up to
 * 128, page_size a power of two from 8, pointers and strides multiples of 16
 * bytes), SV_FP32.  Errors: SV_ERR_ARG (null pointers, dtype, Hq not a
 * multiple of Hkv, window < 0 or together with a tree, scale not finite),
 * SV_ERR_SHAPE, SV_ERR_ALIGN, SV_ERR_CUDA.  Through the status word:
 * SV_ERR_CACHE for a sequence whose kv_len or token range is out of bounds
 * (its outputs are o = 0, lse = -inf, as far as its tokens are known) or
 * with a page outside the cache of which a token sees a key (read as zeros).
 * Entries of pages that no token sees, as those below the window, may hold
 * anything. */
typedef struct {
  const void *q;
  const void *k_cache, *v_cache;
  const int32_t *page_table;
  const int32_t *q_start;
  const int32_t *kv_len;
  const int32_t *tree_mask;
  void *out;
  float *lse;
  int64_t q_token, q_head, o_token, o_head;
  int64_t kc_page, kc_token, kc_head, vc_page, vc_token, vc_head;
  int64_t table_stride;
  int64_t num_pages;
  int32_t T, B, Hq, Hkv, D, page_size, max_pages, tree_words, window, dtype;
  float scale;
  int32_t pad;
} sv_attention_t;
int spec_target_attention(spec_target_t *h, const sv_attention_t *a, void *stream);

/* The tree mask of spec_target_attention from the parents of
 * spec_verify_tree_greedy: for each of B sequences N + 1 rows, row 0 the
 * root, row 1 + j node j, each seeing itself and its ancestors.
 *   tree_parents  device, int32 [B, N], each in [-1, j)
 *   mask          device, int32 [B * (N + 1), ceil((N + 1) / 32)]
 * A parent outside [-1, j) ends the walk and sets SV_ERR_TOKEN.  Errors:
 * SV_ERR_ARG (null pointer, B < 1, N outside 1..SV_MAX_K), SV_ERR_CUDA. */
int spec_target_tree_mask(spec_target_t *h, const int32_t *tree_parents, int32_t B, int32_t N,
                          int32_t *mask, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* SPEC_TARGET_H */
