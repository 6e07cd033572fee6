/*
 * fp8q_moe.h -- MoE routing part of the C ABI of libfp8q: the row layout that
 * the grouped products and the scattering quantizers take, and the balance
 * loss that keeps the experts evenly loaded, with its gradient. Conventions,
 * status codes and enums are those of fp8q.h, which includes this header.
 *
 * Both take the experts that the router chose: ids, device int32
 * [tokens][topk] (topk 1..8). An id outside the range of experts is no route.
 */
#ifndef FP8Q_MOE_H
#define FP8Q_MOE_H

#include <stdint.h>

#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

#define FP8Q_MOE_MAX_EXPERTS 1024
#define FP8Q_MOE_MAX_TOPK    8
#define FP8Q_MOE_MAX_SEQS    32768

#define FP8Q_SCORE_SOFTMAX 0 /* s = softmax(logits)                                */
#define FP8Q_SCORE_SIGMOID 1 /* s = sigmoid(logits) / sum over experts             */

#define FP8Q_LOGITS_BF16 0
#define FP8Q_LOGITS_F32  1

/*
 * moe_dispatch -- expert-sorted row layout of a batch's routes.
 *
 * The experts of this layout are [first, first + experts). With
 * rows[e] = number of routes to expert first + e:
 *   group_rows[e]    = rows[e]
 *   group_offsets[e] = sum over e' < e of rows[e'] rounded up to `align`
 *   dst_rows[t][k]   = group_offsets[e] + number of routes to e before (t, k)
 *                      in row-major order, or -1 for an id outside the range.
 * (What fp8_quantize_act_scatter, fp4_quantize_mx_scatter and the grouped
 * GEMMs take; align = 128 for the FP8 ones, 16 or more for FP4.)
 *
 * ids           device int32 [tokens][topk], contiguous.
 * group_offsets device int32 [experts + 1]; group_rows device int32 [experts];
 *               dst_rows device int32 [tokens][topk], may not overlap ids.
 * workspace     device scratch, 4-byte aligned, of at least
 *               FP8Q_MOE_DISPATCH_WORKSPACE_BYTES; contents need no
 *               initialisation.
 * Shapes: experts 1..FP8Q_MOE_MAX_EXPERTS, topk 1..8, align >= 1, first >= 0,
 *         tokens * topk + experts * (align - 1) < 2^31. tokens == 0: the
 *         offsets and rows are written as zeros (ids and dst_rows may be NULL).
 * Errors: FP8Q_ERR_NULL, FP8Q_ERR_SHAPE, FP8Q_ERR_ALIGN, FP8Q_ERR_HIP.
 */
#define FP8Q_MOE_DISPATCH_WORKSPACE_BYTES 262144LL /* 64 counts of every expert */

int moe_dispatch(const int32_t *ids, int64_t tokens, int32_t topk, int32_t first, int32_t experts, int32_t align,
                 int32_t *group_offsets, int32_t *group_rows, int32_t *dst_rows, void *workspace,
                 int64_t workspace_bytes, hipStream_t stream);

/*
 * moe_balance_loss -- balance loss and per-expert counts.
 *
 * The tokens are cut into sequences s; token t is counted if one of its ids
 * is a valid expert. With T_s the counted tokens of s, counts[s][e] the routes
 * to e, R_s their sum, E = experts, s_te the scores of a row (see
 * FP8Q_SCORE_*) and S' the number of sequences with a counted token:
 *   f[s][e] = E counts[s][e] / R_s          P[s][e] = 1 / T_s sum_t s_te
 *   loss    = alpha / S' sum_s sum_e f[s][e] P[s][e]   (0 if S' = 0)
 *   coef[s][e] = alpha f[s][e] / (T_s S')   = d loss / d s_te of its tokens
 * The counts carry no gradient. A row without a finite score (all logits
 * -inf) has scores of zero; -inf logits have scores of zero; a NaN in a
 * counted row makes the loss NaN (what uncounted rows hold does not matter).
 *
 * logits      [tokens][ld], bf16 or fp32 by logits_dtype, ld >= experts.
 * seq_offsets device int32 [seqs + 1]: non-decreasing, from 0 to tokens; NULL
 *             with seqs == 1: one sequence.
 * loss        device fp32 [1]; counts device int32 [seqs][experts]; coef
 *             device fp32 [seqs][experts].
 * workspace   device scratch, 4-byte aligned, of at least
 *             moe_balance_workspace_bytes(tokens, experts, seqs) bytes.
 * The sums are taken in a fixed order: results repeat bit for bit.
 * Shapes: experts 1..FP8Q_MOE_MAX_EXPERTS, topk 1..8, seqs 1..FP8Q_MOE_MAX_SEQS,
 *         tokens * topk < 2^31 (the counts are int32).
 *         tokens == 0: loss, counts and coef are written as zeros.
 * seq_offsets is trusted to keep its contract; values that break it give
 * unspecified numbers (no access outside the arrays).
 * Errors: FP8Q_ERR_NULL, FP8Q_ERR_SHAPE, FP8Q_ERR_ALIGN, FP8Q_ERR_ENUM,
 *         FP8Q_ERR_HIP.
 */
int64_t moe_balance_workspace_bytes(int64_t tokens, int32_t experts, int64_t seqs);

int moe_balance_loss(const void *logits, int logits_dtype, int64_t tokens, int32_t experts, int64_t ld,
                     const int32_t *ids, int32_t topk, const int32_t *seq_offsets, int64_t seqs, int score,
                     float alpha, float *loss, int32_t *counts, float *coef, void *workspace,
                     int64_t workspace_bytes, hipStream_t stream);

/*
 * moe_balance_loss_backward -- d loss / d logits.
 *
 * With u = logits (softmax) or log sigmoid(logits), s = softmax(u):
 *   du_te = grad s_te (coef[s][e] - sum_j s_tj coef[s][j])
 *   dlogits_te = du_te (softmax), du_te (1 - sigmoid(logits_te)) (sigmoid)
 * and 0 in rows that are not counted.
 *
 * coef        as moe_balance_loss wrote it, with the same ids, seq_offsets,
 *             seqs and score.
 * grad        device fp32 [1], the loss's own gradient; NULL: 1.
 * dlogits     [tokens][ld_d] of logits_dtype, ld_d >= experts; may be logits
 *             itself (with ld_d == ld).
 * tokens == 0: returns FP8Q_OK without launching.
 * Errors: as moe_balance_loss.
 */
int moe_balance_loss_backward(const void *logits, int logits_dtype, int64_t tokens, int32_t experts, int64_t ld,
                              const int32_t *ids, int32_t topk, const int32_t *seq_offsets, int64_t seqs, int score,
                              const float *coef, const float *grad, void *dlogits, int64_t ld_d,
                              hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* FP8Q_MOE_H */
