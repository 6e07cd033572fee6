/*
 * fp8q_gated.h -- the gated feed-forward block of the C ABI of libfp8q: both
 * projections, the activation and the product in one kernel, dense or for the
 * experts of an expert-sorted layout, and the gradient. Conventions, status
 * codes and enums are those of fp8q.h, which includes this header.
 */
#ifndef FP8Q_GATED_H
#define FP8Q_GATED_H

#include <stdint.h>

#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

#define FP8Q_ACT_SILU 0 /* act(g) = g sigmoid(g)                                       */
#define FP8Q_ACT_GELU 1 /* act(g) = g/2 (1 + tanh(sqrt(2/pi) (g + 0.044715 g^3)))      */

#define FP8Q_OUT_E4M3 2 /* codes and scales of 1x128 tiles (beside FP8Q_OUT_BF16, _F32) */

/*
 * fp8_gated_gemm -- H = act(A Wg^T) * (A Wu^T).
 *
 * G and U, the two products, are those of fp8_gemm with FP8Q_BSCALE_BLOCK128:
 * FP32, promoted once per 128-element slab. The activation and the product are
 * computed in FP32 from them; H is rounded once, to its output type.
 *
 * a, a_scale  codes [m][lda] and scales [k/128][ld_as] (1x128 tiles).
 * b           gate codes [n][ldb], and the up codes stride_b bytes behind them
 *             (a [2][n][k] tensor: stride_b = n ldb; weights quantized as one
 *             [2n][k] matrix are that where n % 128 == 0).
 * b_scale     gate scales [ceil(n/128)][ld_bs], the up scales stride_bs floats
 *             behind them.
 * out         out_dtype FP8Q_OUT_BF16, FP8Q_OUT_F32: [m][ldo], ldo >= n.
 *             FP8Q_OUT_E4M3 (n % 128 == 0): codes [m][ldo] and, in out_scale,
 *             scales [n/128][ld_os], ld_os >= m, of H's FP32 values in 1x128
 *             tiles, as fp8_quantize_act makes them of bf16 ones: the operand of
 *             the down product.
 * gate_up     NULL, or bf16 [m][ldg], ldg >= 2n: G in columns [0, n) and U in
 *             [n, 2n), which fp8_gated_backward reads.
 * workspace   DEVICE scratch of workspace_bytes bytes, 16-byte aligned, or
 *             NULL. Only FP8Q_OUT_E4M3 of few rows uses it, and runs faster with
 *             the fp8_gated_workspace_bytes(m, n, k) bytes it needs (0: none).
 *             Its contents need no initialisation; calls whose work overlaps in
 *             time must not share it.
 * Shapes:  m, n >= 0, k % 128 == 0, the limits of fp8_gemm; k == 0 gives zeros.
 *          stride_b, stride_bs >= 0 (they are only read), stride_bs below
 *          FP8Q_MAX_SCALE_SPAN.
 * Alignment: a, b 16-byte aligned; lda, ldb, stride_b % 16 == 0; scales 4-byte
 *          aligned; E4M3 output 16-byte aligned, ldo % 16 == 0. Other outputs
 *          and gate_up: elements only (rows whose columns 4 i start on 8 bytes,
 *          in FP32 16, are written faster).
 * m == 0 or n == 0: returns FP8Q_OK without launching.
 * Errors: FP8Q_ERR_NULL, FP8Q_ERR_SHAPE, FP8Q_ERR_ALIGN, FP8Q_ERR_ENUM,
 *         FP8Q_ERR_HIP.
 */
int64_t fp8_gated_workspace_bytes(int64_t m, int64_t n, int64_t k);

int fp8_gated_gemm(int64_t m, int64_t n, int64_t k, const uint8_t *a, int64_t lda, const float *a_scale,
                   int64_t ld_as, const uint8_t *b, int64_t ldb, int64_t stride_b, const float *b_scale,
                   int64_t ld_bs, int64_t stride_bs, int act, void *out, int64_t ldo, int out_dtype,
                   float *out_scale, int64_t ld_os, uint16_t *gate_up, int64_t ldg, void *workspace,
                   int64_t workspace_bytes, hipStream_t stream);

/*
 * fp8_grouped_gated_gemm -- the same for the experts of an expert-sorted
 * layout: rows [group_offsets[e], group_offsets[e+1]) of A with the weights at
 * b + e * stride_e (bytes) and b_scale + e * stride_es (floats).
 *
 * groups, group_offsets, group_rows, m_total: as fp8_grouped_gemm takes them
 * (offsets in whole 128 rows, group_offsets[groups] == m_total). Rows of a
 * segment past its group_rows[e] are padding: their rows of out (codes and
 * scales too) and of gate_up are written as zeros, whatever A holds there.
 * Without group_rows all rows are real, and the sums may be taken in another
 * order than with counts that say the same.
 * workspace: for E4M3 output, fp8_grouped_gated_workspace_bytes(m_total, n).
 * Everything else as fp8_gated_gemm with m = m_total. FP8Q_DEBUG applies as in
 * fp8_grouped_gemm.
 */
int64_t fp8_grouped_gated_workspace_bytes(int64_t m_total, int64_t n);

int fp8_grouped_gated_gemm(int32_t groups, const int32_t *group_offsets, const int32_t *group_rows, int64_t m_total,
                           int64_t n, int64_t k, const uint8_t *a, int64_t lda, const float *a_scale, int64_t ld_as,
                           const uint8_t *b, int64_t ldb, int64_t stride_b, int64_t stride_e, const float *b_scale,
                           int64_t ld_bs, int64_t stride_bs, int64_t stride_es, int act, void *out, int64_t ldo,
                           int out_dtype, float *out_scale, int64_t ld_os, uint16_t *gate_up, int64_t ldg,
                           void *workspace, int64_t workspace_bytes, hipStream_t stream);

/*
 * fp8_gated_backward -- the gradients of gate and up.
 *
 * With H = act(G) * U and dH the gradient of H:
 *   dG = dH * U * act'(G)        dU = dH * act(G)
 * in FP32 from the bf16 inputs, written side by side as D [m][2n] (dG in
 * columns [0, n)):
 *   out_dtype FP8Q_OUT_BF16: bf16 D [m][ldo], ldo >= 2n; any n. out_scale,
 *             out_t and out_t_scale are NULL.
 *   out_dtype FP8Q_OUT_E4M3 (n % 128 == 0): codes [m][ldo] with scales
 *             out_scale [2n/128][ld_os], ld_os >= m, in 1x128 tiles (A of the
 *             product with the weights, dX), and, where out_t is not NULL (m %
 *             128 == 0), codes TRANSPOSED, out_t [2n][ld_t], ld_t >= m, with
 *             scales out_t_scale [m/128][ld_ts], ld_ts >= 2n, in 128x1 token
 *             tiles (A of the product with X, dW). Both from one pass, each
 *             of the FP32 values: scale fl32(amax / 448), codes E4M3(fl32(x /
 *             scale)), as everywhere (fp8q.h). A tile that holds a NaN or an
 *             infinity reads back with nothing finite in it.
 * dh          bf16 [m][ld_dh], ld_dh >= n; gate_up bf16 [m][ldg], ldg >= 2n.
 * Alignment: bf16 output: elements only (16-byte aligned rows are faster).
 *          E4M3 output: dh, gate_up, out, out_t 16-byte aligned; ld_dh, ldg %
 *          8 == 0; ldo, ld_t % 16 == 0; scales 4-byte aligned.
 * m == 0 or n == 0: returns FP8Q_OK without launching.
 * Errors: as fp8_gated_gemm.
 */
int fp8_gated_backward(int64_t m, int64_t n, const uint16_t *dh, int64_t ld_dh, const uint16_t *gate_up, int64_t ldg,
                       int act, int out_dtype, void *out, int64_t ldo, float *out_scale, int64_t ld_os,
                       uint8_t *out_t, int64_t ld_t, float *out_t_scale, int64_t ld_ts, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* FP8Q_GATED_H */
