/*
 * fp8q_gemv.h -- products of few bf16 rows with FP4 weights: the weight-only
 * part of the C ABI of libfp8q, for serving. Conventions, status codes and
 * enums are those of fp8q.h, which includes this header; FP4 matrices are laid
 * out as fp8q_mx4.h says and made by fp4_quantize_mx.
 */
#ifndef FP8Q_GEMV_H
#define FP8Q_GEMV_H

#include <stdint.h>

#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

#define FP4Q_GEMV_MAX_EXPERTS 1024
#define FP4Q_GEMV_MAX_ROUTES  4096 /* tokens * topk of a call with ids */
#define FP4Q_GEMV_MAX_TOPK    32

/*
 * fp4_gemv_mx -- Y = X dequant(W)^T with FP32 sums, X in bf16.
 *
 * Without ids: X has `tokens` rows (topk == 1, experts == 1), W is one matrix.
 * With ids, DEVICE int32 [tokens][topk]: route (t, j) multiplies its row of X
 * with the matrix of expert ids[t][j] - first, and an id outside [first, first
 * + experts) gives a row of zeros (a dropped route, another rank's expert).
 *
 * n, k      W has n rows with K = k: codes w (ld_w row tiles between K tiles,
 *           experts stride_w bytes apart, % 16 == 0), scales w_scale (ld_ws,
 *           stride_ws words).
 * x         bf16: row of route (t, j) at x + t * ld_x + j * ld_xj (ld_xj == 0:
 *           the routes of a token share its row). Only its first k elements are
 *           read. Rows that start on 16-byte boundaries are read faster.
 * y         row t * topk + j at y + (t * topk + j) * ld_y, ld_y >= n; out_dtype
 *           FP8Q_OUT_BF16 (rounded once, to nearest even) or FP8Q_OUT_F32.
 * The weights are exact in bf16 except where codes times 2^e pass its largest
 * value (infinite there). Every weight row is read once for up to 16 rows of X
 * (64 with more than 32 rows, 32 with more than 16); products of many rows
 * belong to fp4_gemm_mx and fp4_grouped_gemm_mx. The sums are taken in an order
 * that the sizes alone (tokens, topk, experts, n, k) choose: results repeat bit
 * for bit, and a row's do not depend on its place or on what the other rows
 * hold. How many they are may change the last places of its FP32 sums.
 * k == 0, and with ids experts == 0 (a rank without any), write zeros (x and
 * weights may be NULL). tokens, topk or n == 0: returns FP8Q_OK without
 * launching.
 * Limits: n <= FP4Q_MAX_GEMM_ROWS, k <= FP4Q_MAX_GEMM_K, 64 * 65535 rows;
 *         with ids FP4Q_GEMV_MAX_EXPERTS experts, _MAX_ROUTES routes, _MAX_TOPK.
 * Errors: FP8Q_ERR_NULL, FP8Q_ERR_SHAPE, FP8Q_ERR_ALIGN (w not 16-byte, w_scale
 *         and ids not 4-byte, x and y not element aligned), FP8Q_ERR_ENUM,
 *         FP8Q_ERR_HIP.
 */
int fp4_gemv_mx(int64_t tokens, int32_t topk, const int32_t *ids, int32_t first, int32_t experts, int64_t n, int64_t k,
                const uint16_t *x, int64_t ld_x, int64_t ld_xj, const uint8_t *w, int64_t ld_w, int64_t stride_w,
                const uint32_t *w_scale, int64_t ld_ws, int64_t stride_ws, void *y, int64_t ld_y, int out_dtype,
                hipStream_t stream);

/*
 * fp4_gated_gemv_mx -- H = act(X Wg^T) * (X Wu^T): the first half of a gated
 * feed-forward block for few rows, both products in FP32 and H rounded once.
 * w, w_scale are the gate's matrix, the up one stands stride_up bytes (% 16 ==
 * 0) and stride_ups words behind it; act is FP8Q_ACT_SILU or FP8Q_ACT_GELU
 * (fp8q_gated.h). Everything else as fp4_gemv_mx.
 */
int fp4_gated_gemv_mx(int64_t tokens, int32_t topk, const int32_t *ids, int32_t first, int32_t experts, int64_t n,
                      int64_t k, const uint16_t *x, int64_t ld_x, int64_t ld_xj, const uint8_t *w, int64_t ld_w,
                      int64_t stride_up, int64_t stride_w, const uint32_t *w_scale, int64_t ld_ws, int64_t stride_ups,
                      int64_t stride_ws, int act, void *y, int64_t ld_y, int out_dtype, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* FP8Q_GEMV_H */
