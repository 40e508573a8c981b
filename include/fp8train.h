/*
 * fp8train.h -- C ABI of libfp8blk for training a mixture of experts on the
 * blockwise-FP8 linear layer (fp8blk.h and fp8moe.h; their readings and
 * conventions hold here too): tokens sorted by expert, their rows quantized as
 * they are gathered, every expert's products over its own rows, the rows back
 * to their tokens with weights, the gradients of all of these; and what the
 * backward pass needs kept in 8 bits -- the gated unit's inputs and the operand
 * of the weights' gradient.
 *
 * One layer's training step (ids, weights: fp8_moe_route's):
 *   rows, source, offsets = fp8_moe_sort(ids)
 *   (qx, sx) = fp8_moe_gather(x)              kept: the linear's operand is the checkpoint
 *   gu = fp8_moe_gemm_fprop(qx, W1)
 *   (qh, sh), (qc, sc) = fp8_gated_forward(gu)      kept: (qc, sc), instead of gu and h
 *   z = fp8_moe_gemm_fprop(qh, W2)                  kept for the weights' gradient
 *   y = fp8_moe_combine(z, weights)
 * and back:
 *   dz in both orientations, dweights = fp8_moe_combine_backward(dy, z)
 *   dh = fp8_moe_gemm_dgrad(dz, W2)
 *   dgu in both orientations, h for Wgrad = fp8_gated_backward(dh, qc, sc)
 *   dW2 = fp8_moe_gemm_wgrad(dz, h)
 *   dx = fp8_moe_combine(fp8_moe_gemm_dgrad(dgu, W1), no weights)
 *   dW1 = fp8_moe_gemm_wgrad(dgu, fp8_requantize_colgroup(qx, sx))
 *   dlogits = fp8_moe_route_backward(dweights)
 *
 * Sorted rows.  The T k choices (choice c = t k + i is the i-th expert of token
 * t) become rows of a buffer of R rows: expert e's segment is rows
 * [offsets[e], offsets[e + 1]), a multiple of 128 of them, its choices first, in
 * the order of c, then padding.  R = fp8_moe_sorted_rows(T, E, k) holds any
 * choice, so nothing has to be known on the host.  The rows from offsets[E] on
 * are behind the last segment: no call of this header reads them and none
 * writes them.  `used` arguments are a DEVICE pointer to one int32, the number
 * of rows in use (offsets + E of the sort), or NULL for all of them; a value
 * outside [0, rows] counts as the nearer end.  Where groups of 128 rows are
 * quantized, or rows are multiplied, it is rounded up to a multiple of 128, and
 * the rows up to there have to hold values (fp8_gated_forward, whose groups lie
 * along the rows, stops at the row itself).
 *
 * Values that are not finite: a group of 128 with a NaN or an infinity has the
 * codes and the scale that the quantizers of fp8blk.h give it, and leaves the
 * other groups as they are.
 */
#ifndef FP8TRAIN_H
#define FP8TRAIN_H

#include "fp8moe.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Rows that any choice of k of E experts by T tokens fits in: T k, and 127 of
 * padding for each expert that can be reached, rounded up to 512.  (size_t)-1
 * for an invalid shape: T >= 1, T < 2^24, E and k as for fp8_moe_route. */
size_t fp8_moe_sorted_rows(int64_t T, int64_t E, int k);

/* Workspace bytes of fp8_moe_sort ((size_t)-1 for an invalid shape). */
size_t fp8_moe_sort_workspace_size(int64_t T, int64_t E, int k);

/*
 * The sorted order of a choice.
 *   ids     [T][k] int32 (fp8_moe_route's); ids outside [0, E) are no expert
 *           (padding), an id that stands twice in a row has two rows
 *   rows    [T][k] int32: the row of each choice, -1 for none
 *   source  [R] int32, R = fp8_moe_sorted_rows(T, E, k): the choice of each row,
 *           -1 for padding and for the rows behind the last segment
 *   offsets [E + 1] int32: the segments' first rows, and where the last one ends
 *   workspace: at least fp8_moe_sort_workspace_size(T, E, k) bytes, 16-byte
 *     aligned; may be NULL when that size is 0.
 * Stable (an expert's choices keep their order) and the same on every call.
 */
int fp8_moe_sort(int64_t T, int64_t E, int k, const int32_t *ids, int32_t *rows, int32_t *source,
                 int32_t *offsets, void *workspace, size_t ws_bytes, hipStream_t stream);

/*
 * The tokens' rows in sorted order, quantized: row r is x[source[r] / k], or
 * bf16(weights[source[r]] * x[source[r] / k]) where weights are given; rows
 * whose source is outside [0, T k) are zeros (codes 0, scale 1).
 *   x       [T][H] bf16, row stride ld_x (>= H, multiple of 8)
 *   source  [R] int32;  weights [T k] fp32 or NULL;  used as above
 *   q [R][H] codes (row stride ld_q >= H, multiple of 16), s [R][H/128]: as
 *     fp8_quantize_rowgroup of those rows
 *   qT [H][R] codes (row stride ld_qT >= R, multiple of 16), sT [H][R/128]: as
 *     fp8_quantize_colgroup of them; both NULL to skip
 *   workspace: at least fp8_moe_gather_workspace_size(T, H, R, k, qT != NULL)
 *     bytes, 16-byte aligned; may be NULL when that size is 0.
 *   H and R positive multiples of 128; 1 <= k <= FP8MOE_MAX_TOPK; T < 2^24,
 *   R < 2^31, R H < 2^37, T ceil(H / 512) < 2^25; T ld_x, R ld_q and H ld_qT at
 *   most 2^40.
 */
int fp8_moe_gather(int64_t T, int64_t H, int64_t R, int k, const uint16_t *x, int64_t ld_x,
                   const int32_t *source, const float *weights, const int32_t *used,
                   uint8_t *q, int64_t ld_q, float *s, uint8_t *qT, int64_t ld_qT, float *sT,
                   int scale_mode, void *workspace, size_t ws_bytes, hipStream_t stream);

/* Workspace bytes of fp8_moe_gather, with (transpose != 0) or without qT and sT
 * ((size_t)-1 for an invalid shape). */
size_t fp8_moe_gather_workspace_size(int64_t T, int64_t H, int64_t R, int k, int transpose);

/*
 * Sorted rows back to their tokens: y[t] = sum_i weights[t][i] z[rows[t][i]], in
 * the order of i, in fp32; entries of rows outside [0, R) are left out, and a
 * token with none of them gets zeros.
 *   z [R][H] bf16, row stride ld_z (>= H, multiple of 8)
 *   rows [T][k] int32;  weights [T][k] fp32, or NULL for 1 (the gradient of
 *   fp8_moe_gather without weights: dx from the gradients of its rows)
 *   y [T][H] dense, bf16 or fp32 (FP8BLK_OUT_FP32_ACCUM adds to it)
 *   limits as for fp8_moe_gather; R a positive multiple of 128.
 */
int fp8_moe_combine(int64_t T, int64_t H, int64_t R, int k, const uint16_t *z, int64_t ld_z,
                    const int32_t *rows, const float *weights, void *y, int out_dtype, hipStream_t stream);

/*
 * Gradient of fp8_moe_combine with weights:
 *   dz[r] = weights[source[r]] dy[source[r] / k], rounded to bf16 once and
 *     quantized in both orientations (fp8_moe_gather of dy with weights);
 *   dweights[t][i] = sum_h dy[t][h] z[rows[t][i]][h] in fp32, 0 where rows[t][i]
 *     is outside [0, R).
 *   dy [T][H] bf16, row stride ld_dy;  z as fp8_moe_combine took it;  rows,
 *   source: fp8_moe_sort's;  weights, dweights [T][k] fp32.
 */
int fp8_moe_combine_backward(int64_t T, int64_t H, int64_t R, int k, const uint16_t *dy, int64_t ld_dy,
                             const uint16_t *z, int64_t ld_z, const int32_t *rows, const int32_t *source,
                             const float *weights, const int32_t *used,
                             uint8_t *q, int64_t ld_q, float *s, uint8_t *qT, int64_t ld_qT, float *sT,
                             float *dweights, int scale_mode, hipStream_t stream);

/*
 * Every expert's product with its own segment: the contractions of fp8blk.h
 * with the weights of the row's expert.
 *   Fprop  y[r]  = x[r] W_e^T:  qx [R][K] + sx [R][K/128], qw [E][N][K] + sw
 *          [E][N/128][K/128], y [R][N]
 *   Dgrad  dx[r] = dy[r] W_e:   qdy [R][N] + sdy [R][N/128], qw and sw as
 *          quantized, dx [R][K]
 *   Wgrad  dW_e  = sum over e's rows r of dy[r]^T x[r]: qdyT [N][R] + sdyT
 *          [N][R/128], qxT [K][R] + sxT [K][R/128], dw [E][N][K]; an expert
 *          without rows has zeros (with FP8BLK_OUT_FP32_ACCUM, what was there)
 *   offsets [E + 1] int32 (fp8_moe_sort's): multiples of 128, ascending, at most R.
 *     Others count as the multiple of 128 below, inside [0, R]; descending ones
 *     give no defined result, but nothing outside the operands is touched.
 *   out_dtype: FP8BLK_OUT_BF16, FP8BLK_OUT_FP32 or FP8BLK_OUT_FP32_ACCUM.
 *   scale_mode: the rule that made all the scales.
 * Rows of y and dx outside the segments are not written.  All operands dense,
 * 16-byte aligned (offsets 4-byte); R, N, K positive multiples of 128, R < 2^29,
 * N, K < 2^25, E <= FP8MOE_MAX_EXPERTS, R N and R K at most 2^40, E N K 2^38.
 * For given sizes an expert's results do not depend on how the other rows are
 * spread over the other experts; sums are fp32 with the accuracy of the GEMMs of
 * fp8blk.h.
 */
int fp8_moe_gemm_fprop(int64_t R, int64_t N, int64_t K, int64_t E, const uint8_t *qx, const float *sx,
                       const uint8_t *qw, const float *sw, const int32_t *offsets, void *y, int out_dtype,
                       int scale_mode, hipStream_t stream);
int fp8_moe_gemm_dgrad(int64_t R, int64_t N, int64_t K, int64_t E, const uint8_t *qdy, const float *sdy,
                       const uint8_t *qw, const float *sw, const int32_t *offsets, void *dx, int out_dtype,
                       int scale_mode, hipStream_t stream);
int fp8_moe_gemm_wgrad(int64_t R, int64_t N, int64_t K, int64_t E, const uint8_t *qdyT, const float *sdyT,
                       const uint8_t *qxT, const float *sxT, const int32_t *offsets, void *dw, int out_dtype,
                       int scale_mode, hipStream_t stream);

/*
 * The gated unit between two linears, h = silu(g) u, rounded to bf16 once and
 * quantized for the second one, and its inputs kept in 8 bits.
 *   gu [M][2 I] bf16, row stride ld_gu (>= 2 I, multiple of 8): g's I columns,
 *      then u's (the output of a gate/up linear)
 *   q  [M][I] codes (row stride ld_q), s [M][I/128]: as fp8_quantize_rowgroup of h
 *   qc [M][2 I] codes (row stride ld_qc), sc [M][2 I/128]: the checkpoint, as
 *      fp8_quantize_rowgroup of gu; both NULL to skip
 *   M >= 1 (any value), I a positive multiple of 128; M < 2^31, M I < 2^35;
 *   M ld_gu, M ld_q and M ld_qc at most 2^40.
 */
int fp8_gated_forward(int64_t M, int64_t I, const uint16_t *gu, int64_t ld_gu, const int32_t *used,
                      uint8_t *q, int64_t ld_q, float *s, uint8_t *qc, int64_t ld_qc, float *sc,
                      int scale_mode, hipStream_t stream);

/*
 * The gated unit's gradient from the checkpoint: with g and u what its codes
 * stand for (rounded to bf16 where the scales are amax / 448) and sig = 1 / (1 + e^-g),
 *   du = dh g sig,  dg = dh u sig (1 + g (1 - sig)),
 * each rounded to bf16 once and quantized in both orientations, and h =
 * bf16(g sig u) once more, in the orientation that the second linear's Wgrad
 * takes.  As h in the forward pass, they are right for all finite values: where sig, dh u
 * or a code's value leaves fp32's range, and the result does not, in 64 bits.
 *   dh [M][I] bf16, row stride ld_dh;  qc, sc: fp8_gated_forward's checkpoint
 *   q [M][2 I] + s [M][2 I/128], qT [2 I][M] + sT [2 I][M/128]: (dg, du)
 *   qhT [I][M] + shT [I][M/128]: h
 *   scale_mode: the checkpoint's rule, and the results'.
 *   M and I positive multiples of 128; limits as for fp8_gated_forward.
 */
int fp8_gated_backward(int64_t M, int64_t I, const uint16_t *dh, int64_t ld_dh,
                       const uint8_t *qc, int64_t ld_qc, const float *sc, const int32_t *used,
                       uint8_t *q, int64_t ld_q, float *s, uint8_t *qT, int64_t ld_qT, float *sT,
                       uint8_t *qhT, int64_t ld_qhT, float *shT, int scale_mode, hipStream_t stream);

/*
 * Row groups to column groups: the values that (q, s) stand for, rounded to bf16
 * (exact for power-of-two scales from 2^-124 on; 2^128, which a code of the largest
 * one may stand for, is infinity), quantized as fp8_quantize_colgroup does.  The operand that Fprop read and that was kept
 * becomes the one that Wgrad reads, so no second copy lives through the step.
 *   q [rows][cols] codes (row stride ld_q), s [rows][cols/128]
 *   qT [cols][rows] codes (row stride ld_qT), sT [cols][rows/128]
 *   scale_mode: the result's rule; s may hold any scales.
 *   rows and cols positive multiples of 128; rows < 2^31, rows cols < 2^37; rows
 *   ld_q and cols ld_qT at most 2^40.
 */
int fp8_requantize_colgroup(const uint8_t *q, int64_t rows, int64_t cols, int64_t ld_q, const float *s,
                            const int32_t *used, uint8_t *qT, int64_t ld_qT, float *sT, int scale_mode,
                            hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* FP8TRAIN_H */
