/*
 * fp8moe.h -- C ABI of libfp8blk for any number of tokens and for mixtures of
 * experts: the blockwise-FP8 linear layer of fp8blk.h (its sources, readings
 * and conventions hold here too) from bf16 activations at any token count,
 * the router of a mixture of experts with its gradient, and a whole
 * mixture-of-experts layer for a few tokens.
 *
 * Conventions: those of fp8blk.h -- device pointers on the current device,
 * row-major tensors, bf16 as raw 16-bit patterns, work only enqueued on
 * `stream`, caller-owned buffers and workspaces (contents on entry
 * irrelevant; calls that run at the same time need separate ones), every
 * argument check on the host before any launch, FP8BLK_OK or a negative
 * FP8BLK_ERR_* code.  Outputs must not alias inputs or the workspace.
 */
#ifndef FP8MOE_H
#define FP8MOE_H

#include "fp8blk.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element type of router logits and of their gradient. */
enum fp8moe_dtype { FP8MOE_BF16 = 0, FP8MOE_FP32 = 1 };

/* fp8_linear sums products with fp32 faithfulness up to this many rows. */
#define FP8_LINEAR_FP32_ROWS 127

/* Limits of the mixture-of-experts entry points. */
#define FP8MOE_MAX_EXPERTS 1024 /* E */
#define FP8MOE_MAX_TOPK 16      /* k */
#define FP8MOE_MAX_TOKENS 512   /* T of fp8_moe_experts and fp8_moe_layer */

/*
 * Y = X W^T for any number of tokens, from bf16 activations: what
 * fp8_quantize_rowgroup of X followed by Fprop computes (the same codes and
 * scales, fp32 accumulation), without the multiple-of-128 limit on M.
 *   x   [M][K] bf16, row stride ld_x (>= K, multiple of 8, at most 2^26), M >= 1
 *   qw  [N][K] codes + sw [N/128][K/128] (from fp8_quantize_block of W)
 *   y   [M][N] dense, bf16 or fp32 (FP8BLK_OUT_FP32_ACCUM adds to it)
 *   scale_mode: the rule that made sw, and the rule x is quantized by.
 *   N, K positive multiples of 128; x, qw, y 16-byte aligned.  M < 2^27, N <
 *   2^27, K < 2^25; M N, M K, N K and M ld_x at most 2^40, M K / 128 < 2^31.
 *   workspace: at least fp8_linear_workspace_size(M, N, K, scale_mode) bytes,
 *     16-byte aligned; may be NULL when that size is 0 (a few rows, small
 *     products).
 * Up to FP8_LINEAR_FP32_ROWS rows the products are summed with fp32
 * faithfulness; above, with at least the accuracy of the GEMMs of fp8blk.h (on
 * the fp8 matrix instruction, 1.5e-5 to 4.5e-5 of the result's norm), which take
 * the multiples of 128 rows of large products.  Which kernel sums a row, and in
 * which order, is decided by M, N, K and scale_mode alone: equal calls give equal
 * bits, but a row may differ in its last bits between calls of different M.
 */
int fp8_linear(int64_t M, int64_t N, int64_t K, const uint16_t *x, int64_t ld_x,
               const uint8_t *qw, const float *sw, void *y, int out_dtype, int scale_mode,
               void *workspace, size_t ws_bytes, hipStream_t stream);

/* Workspace bytes of fp8_linear ((size_t)-1 for an invalid shape or mode). */
size_t fp8_linear_workspace_size(int64_t M, int64_t N, int64_t K, int scale_mode);

/*
 * The router's choice: for each token the k experts with the largest logits,
 * largest first, equal ones by lower index, and their softmax weights.
 *   logits [T][E] bf16 or fp32 (dtype: enum fp8moe_dtype), row stride ld >= E
 *   ids    [T][k] int32, dense;  weights [T][k] fp32, dense
 *   renormalize: 1, the softmax runs over the k chosen logits (the weights
 *     sum to 1); 0, over all E of them.
 * An expert whose logit is -infinity or NaN is masked out: it is never
 * chosen and takes no part in the softmax.  Where fewer than k are left, the
 * rest of the row is id -1 with weight 0.  A logit of +infinity outweighs
 * every finite one; several of them share evenly.
 *   1 <= T < 2^31, T ld at most 2^40, 1 <= E <= FP8MOE_MAX_EXPERTS, 1 <= k <=
 *   min(E, FP8MOE_MAX_TOPK).
 */
int fp8_moe_route(int64_t T, int64_t E, int k, const void *logits, int dtype, int64_t ld,
                  int renormalize, int32_t *ids, float *weights, hipStream_t stream);

/*
 * Gradient of the router's weights with respect to the logits, for the ids
 * that fp8_moe_route gave (the choice itself has none):
 *   renormalize 1: dlogit_j = w_j (g_j - sum_i g_i w_i) for chosen j, else 0;
 *   renormalize 0: dlogit_j = p_j ([j chosen] g_j - sum_i g_i w_i), p the
 *     softmax over all experts.
 *   logits as given to fp8_moe_route; ids [T][k]; dweights [T][k] fp32 (g);
 *   dlogits [T][E], the logits' type, row stride ld_d >= E; every element is
 *   written.  Ids outside [0, E) are none and their g is not read into any
 *   sum; masked-out experts get 0.  An id that stands twice in a row counts
 *   as one chosen expert whose g is the sum.
 */
int fp8_moe_route_backward(int64_t T, int64_t E, int k, const void *logits, int dtype, int64_t ld,
                           const int32_t *ids, const float *dweights, int renormalize,
                           void *dlogits, int64_t ld_d, hipStream_t stream);

/*
 * The experts of a mixture for a few tokens (gated linear units):
 *   y[t] = sum_i w[t][i] * Wd[e] h,  h = silu(G[e] x[t]) * (U[e] x[t]),
 *   e = ids[t][i]; terms whose id is outside [0, E) are left out, so a token
 *   with no expert (a padded one: ids -1) gets zeros.
 * Every product is the linear layer above: x[t] is quantized in groups of
 * 128 by scale_mode's rule; h is rounded to bf16 once and quantized by the
 * same rule; products, silu and the weighted sum are fp32.  Equal calls give
 * equal bits; in which order a token's terms are added may depend on the other
 * tokens of the call (on their number and on the experts that they reach).
 *   x   [T][H] bf16, row stride ld_x (>= H, multiple of 8, at most 2^26)
 *   ids [T][k] int32, weights [T][k] fp32, dense
 *   qw1 [E][2 I][H] codes, sw1 [E][2 I / 128][H / 128]: for each expert the
 *       I rows of G, then the I rows of U
 *   qw2 [E][H][I] codes, sw2 [E][H / 128][I / 128]: Wd
 *       (each as fp8_quantize_block quantizes the stacked matrix)
 *   y   [T][H] dense, bf16 or fp32 (no accumulation)
 *   1 <= T <= FP8MOE_MAX_TOKENS; H, I positive multiples of 128, at most 2^20,
 *   H I at most 2^29 and T k I < 2^31; E and k as for fp8_moe_route; codes, x
 *   and y 16-byte aligned, the rest 4-byte.
 *   workspace: at least fp8_moe_workspace_size(T, H, I, E, k) bytes, 16-byte
 *     aligned.
 */
int fp8_moe_experts(int64_t T, int64_t H, int64_t I, int64_t E, int k,
                    const uint16_t *x, int64_t ld_x, const int32_t *ids, const float *weights,
                    const uint8_t *qw1, const float *sw1, const uint8_t *qw2, const float *sw2,
                    void *y, int out_dtype, int scale_mode,
                    void *workspace, size_t ws_bytes, hipStream_t stream);

/*
 * A whole mixture-of-experts layer for a few tokens: the router's logits
 * x wr^T (bf16 operands, fp32 result), fp8_moe_route's choice of k experts
 * with their weights, and fp8_moe_experts of it.
 *   wr  [E][H] bf16 router weights, dense, 16-byte aligned
 *   ids, weights [T][k]: where the choice is written; both may be NULL.
 *   A token none of whose logits can be chosen (all NaN or -infinity: x[t] or
 *   wr is not finite, or their product overflows) has ids -1 and weights 0, and
 *   its row of y is NaN: unlike a caller's -1 it is no padding.
 *   everything else as for fp8_moe_route and fp8_moe_experts.
 */
int fp8_moe_layer(int64_t T, int64_t H, int64_t I, int64_t E, int k, int renormalize,
                  const uint16_t *x, int64_t ld_x, const uint16_t *wr,
                  const uint8_t *qw1, const float *sw1, const uint8_t *qw2, const float *sw2,
                  void *y, int out_dtype, int scale_mode, int32_t *ids, float *weights,
                  void *workspace, size_t ws_bytes, hipStream_t stream);

/* Workspace bytes of fp8_moe_experts and fp8_moe_layer ((size_t)-1 for an
 * invalid shape). */
size_t fp8_moe_workspace_size(int64_t T, int64_t H, int64_t I, int64_t E, int k);

#ifdef __cplusplus
}
#endif

#endif /* FP8MOE_H */
