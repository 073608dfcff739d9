/*
 * spec_layer.h -- C ABI of the operators of the second half of a target layer,
 * and of what a service says of its answers, on a GB300 (sm_103a):
 *
 *   linear              product with bias, activation and residual
 *   gated linear        both projections of a gated feed-forward block, the
 *                       activation and the product
 *   block norm          norms after and before a block, gate, scale, residual
 *   log probabilities   of given tokens, entropy, top alternatives
 *
 * They stand beside the operators of spec_target.h, whose handle they take and
 * whose conventions hold here: return values, error codes and ownership; the
 * stream of a call; strides in elements with a dense innermost dimension; the
 * handle's status word.  They use no scratch, so calls on one handle may
 * overlap.  Nothing is synchronised or allocated, every call can be captured
 * in a CUDA graph, and outputs are the same bit for bit when a call is repeated.
 *
 * The pages have no code for these steps ("Speculative Decoding: Two Models,
 * One Voice", "The idea", step 2, has the target check K+1 positions in one
 * forward pass); the formulas below are the common ones.
 */
#ifndef SPEC_LAYER_H
#define SPEC_LAYER_H

#include "spec_target.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---------------------------------------------------------------------------
 * Products of a linear layer with what follows them, sums and epilogue in
 * fp32, each output rounded once:
 *   linear        out = act(x w^T + bias) + residual
 *   gated linear  out = act(x w_gate^T + bias_gate) * (x w_up^T + bias_up)
 * With SV_ACT_GELU act(v) = v Phi(v), SV_ACT_GELU_TANH its form with tanh,
 * SV_ACT_SILU v / (1 + exp(-v)).
 *   x         device, dtype, [M, K] with row stride
 *   w         device, dtype, [N, K] with row stride (a linear layer's weight);
 *             w_gate and w_up may be halves of one fused weight
 *   bias      device, dtype, [N] or NULL
 *   residual  device, out_dtype, [M, N] with row stride, or NULL; may be out
 *             itself (in place)
 *   out       device, out_dtype, [M, N] with row stride; apart from x and w
 * dtype and out_dtype: SV_BF16, SV_FP16 or SV_FP32.  16-bit x and w whose
 * rows are 16-byte aligned are multiplied on the tensor cores, whose
 * additions may cut instead of round (fp32 outputs of normal values are off by
 * about 1.1e-9 K of their norm where one CTA sums all of K: 4e-6 at K 4096,
 * 3e-5 at 28672); everything else by fp32 arithmetic.
 * M == 0 is a no-op.  Errors: SV_ERR_ARG (null pointer, types, activation),
 * SV_ERR_SHAPE (a negative M, N or K below 1, a size above 2^24, a stride
 * below its row or above 2^36), SV_ERR_ALIGN (a pointer not aligned to its
 * element), SV_ERR_CUDA; SV_ERR_TIMEOUT through the status word. */
#define SV_ACT_NONE 0
#define SV_ACT_RELU 1
#define SV_ACT_GELU 2
#define SV_ACT_GELU_TANH 3
#define SV_ACT_SILU 4
typedef struct {
  const void *x, *w, *bias, *residual;
  void *out;
  int64_t x_stride, w_stride, residual_stride, out_stride;
  int64_t M, N, K;
  int32_t dtype, out_dtype, activation, pad;
} sv_linear_t;
int spec_layer_linear(spec_target_t *h, const sv_linear_t *a, void *stream);

typedef struct {
  const void *x, *w_gate, *w_up, *bias_gate, *bias_up;
  void *out;
  int64_t x_stride, gate_stride, up_stride, out_stride;
  int64_t M, N, K;
  int32_t dtype, out_dtype, activation, pad;
} sv_gated_linear_t;
int spec_layer_gated_linear(spec_target_t *h, const sv_gated_linear_t *a, void *stream);

/* ---------------------------------------------------------------------------
 * The norms around a block, with its gate, its scale and the residual, in one
 * pass and in fp32:
 *   y   = x / sqrt(mean(x^2) + eps) * post_weight   (y = x without post_weight)
 *   h   = residual + branch_scale * gate * y
 *   out = h / sqrt(mean(h^2) + eps) * weight
 * Neither y nor h is rounded on the way; residual_out receives h rounded once.
 *   x, residual   device, dtype, [rows, d] with row strides
 *   post_weight   device, dtype, [d] or NULL
 *   gate          device, dtype, or NULL: element [r, c] lies at
 *                 r * gate_row + c * gate_col, gate_col 0 or 1 (gate_row 0: one
 *                 gate for all rows; gate_col 0: one for all columns)
 *   weight        device, dtype, [d]
 *   out           group -1: device, dtype, [rows, d] with row stride; group
 *                 SV_SCALE_BLOCK or 0: E4M3 bytes [rows, d], dense, with scales
 *                 as spec_target_rms_norm_fp8 (out_stride is not read)
 *   scale         device, fp32 [rows, ceil(d / 128)] or [rows] (group >= 0)
 *   residual_out  device, dtype, [rows, d] with row stride, or NULL; may be the
 *                 residual or x itself (in place), and out may be x or residual
 *                 where residual_out is not the same
 * rows == 0 is a no-op.  Errors as spec_target_rms_norm; SV_ERR_ARG for
 * another group, a gate_col that is not 0 or 1, a negative gate_row, or a
 * branch_scale that is not finite. */
typedef struct {
  const void *x, *residual, *post_weight, *gate, *weight;
  void *out;
  float *scale;
  void *residual_out;
  int64_t x_stride, residual_stride, out_stride, residual_out_stride, gate_row, gate_col;
  int64_t rows, d;
  int32_t dtype, group;
  float eps, branch_scale;
} sv_block_norm_t;
int spec_layer_block_norm(spec_target_t *h, const sv_block_norm_t *a, void *stream);

/* ---------------------------------------------------------------------------
 * What a service says of its answers: with z = logits / temperature and
 * lse = log sum_v exp(z_v), for each row
 *   log_probs[t] = z[tokens[t]] - lse       of the n given tokens
 *   entropy      = -sum_v exp(z_v - lse) (z_v - lse), in nats
 *   top          the `top` largest logits: ids, and their log probabilities in
 *                falling order; of equal logits the smaller id comes first
 *   logits   device, dtype (SV_BF16, SV_FP16, SV_FP32), [rows, V], row stride
 *   tokens   device, int32 [rows, n] or NULL (n = 0); -1 is no token and gets
 *            0; another one outside [0, V) gets NaN and sets SV_ERR_TOKEN
 *   log_probs      device, fp32 [rows, n]
 *   entropy        device, fp32 [rows] or NULL
 *   top_ids        device, int32 [rows, top]; top from 0 to SV_MAX_TOP and V
 *   top_log_probs  device, fp32 [rows, top]
 * Logits of -inf are tokens of probability 0.  A row with a NaN or +inf, or
 * with -inf alone, gets NaN throughout (but 0 for a token of -1) and ids of -1.
 * rows == 0 is a no-op.  Errors: SV_ERR_ARG (null pointer, dtype, n negative, a
 * temperature that is not above 0 or not finite, or for which 1.4427 / T is not
 * finite), SV_ERR_SHAPE (V outside 1..2^24, top outside 0..min(SV_MAX_TOP, V), n above
 * 2^16, rows negative or above 2^24, a stride below V), SV_ERR_ALIGN, SV_ERR_CUDA. */
#define SV_MAX_TOP 64
typedef struct {
  const void *logits;
  const int32_t *tokens;
  float *log_probs, *entropy;
  int32_t *top_ids;
  float *top_log_probs;
  int64_t stride, rows, V;
  int32_t dtype, n, top;
  float temperature;
} sv_log_probs_t;
int spec_layer_log_probs(spec_target_t *h, const sv_log_probs_t *a, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* SPEC_LAYER_H */
