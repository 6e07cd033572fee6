/*
 * fp8q_mx4.h -- FP4 microscaling (OCP MX, E2M1 elements) part of the C ABI of
 * libfp8q. Conventions, status codes and enums are those of fp8q.h, which
 * includes this header.
 *
 * Numeric contract. 32 consecutive elements along K share a power-of-two
 * scale 2^e, e = floor(log2(amax)) - 2 clamped to [-127, 127] (-127 for an
 * all-zero block), held as the E8M0 byte e + 127; a code is E2M1(x / 2^e)
 * (magnitudes 0, 0.5, 1, 1.5, 2, 3, 4, 6), rounded to nearest, ties to the
 * even code, saturating to +-6, with the sign of x. The value of a code is
 * dec(code) * 2^e. A block that holds an infinity or a NaN gets the byte 255
 * (NaN) and zero codes: it reads back as NaN, and every output that its row
 * takes part in is NaN.
 *
 * Layout of an FP4 matrix with `rows` rows and K = `k`: tiles of 16 rows x
 * 128 k, kt = ceil(k / 128) K tiles and rt = ceil(rows / 16) row tiles.
 *   codes   tile (t, u) is the 1024 bytes at (t * ld + u) * 1024. In a tile,
 *           row r occupies bytes [64 r, 64 r + 64); its block b (32 elements,
 *           16 bytes, the even element in the low nibble) stands at
 *           64 r + 16 (b ^ ((r >> 2) & 3)).
 *   scales  64 uint32 words at (t / 4 * ld_s + u) * 64 for four K tiles: word
 *           4 r + b holds block b of row r, its byte t % 4 that of K tile t.
 * ld and ld_s count row tiles (ld, ld_s >= rt), so a range of row tiles of a
 * larger matrix is a matrix with the same ld. Rows and elements past the
 * matrix, up to whole tiles, are written as zero codes; scale bytes of whole
 * blocks past it, up to 16 rows and 512 k, as 0.
 * Alignment: codes 16 bytes, scales 4 bytes. Products of many rows are faster
 * with scales (and experts' scales) that start on 16-byte boundaries.
 */
#ifndef FP8Q_MX4_H
#define FP8Q_MX4_H

#include <stdint.h>

#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

#define FP4Q_TILE_1x32 0 /* blocks along the rows of x                              */
#define FP4Q_TILE_32x1 1 /* blocks along the columns of x: the transposed operand   */

/*
 * Limits of every call: its launch holds fewer than 2^32 work-items, that is
 * fewer than 2^26 units of 16 rows x 512 k (1x32, scatter, read-back) or 2^23
 * units of 256 rows x 128 columns of x (32x1), parts of units counted whole.
 * Limits of the products: rows of A, B and C are numbered with 32 bits (a
 * tile of 256 rows may start at the last one). Codes and scales are addressed
 * with 64 bits. Larger values return FP8Q_ERR_SHAPE before any launch.
 */
#define FP4Q_MAX_GEMM_ROWS 2147483136LL   /* 2^31 - 512: m, n, m_total */
#define FP4Q_MAX_GEMM_K    137438953472LL /* 2^37                     */

/*
 * fp4_quantize_mx -- bf16 to FP4 codes and scales.
 *
 * x       groups matrices [rows][ld_x], ld_x >= cols, stride_x elements apart
 *         (stride_x >= 0: they are only read and may overlap).
 * tiling  FP4Q_TILE_1x32: K runs along the columns of x; writes FP4 matrices
 *           of `rows` rows with K = cols.
 *         FP4Q_TILE_32x1: K runs along the rows of x; writes FP4 matrices of
 *           `cols` rows with K = rows (x transposed: the operands that
 *           contract over tokens, or a weight for the input gradient).
 * q       codes; ld_q row tiles between K tiles, stride_q bytes between
 *         matrices (groups > 1: stride_q >= kt * ld_q * 1024, % 16 == 0).
 * scale   words; ld_s row tiles between K groups, stride_s words between
 *         matrices (groups > 1: stride_s >= ceil(kt / 4) * ld_s * 64).
 * Any rows, cols >= 0 within the limits and any ld_x; rows of x that start on 16-byte
 * boundaries (x, ld_x and stride_x so aligned) are read faster.
 * groups, rows or cols == 0: returns FP8Q_OK without launching.
 * Errors: FP8Q_ERR_NULL, FP8Q_ERR_SHAPE, FP8Q_ERR_ALIGN (x not 2-byte
 *         aligned, q not 16, scale not 4), FP8Q_ERR_ENUM, FP8Q_ERR_HIP.
 */
int fp4_quantize_mx(int32_t groups, const uint16_t *x, int64_t rows, int64_t cols, int64_t ld_x, int64_t stride_x,
                    int tiling, uint8_t *q, int64_t ld_q, int64_t stride_q, uint32_t *scale, int64_t ld_s,
                    int64_t stride_s, hipStream_t stream);

/*
 * fp4_quantize_mx_scatter -- quantize each token once and store it to the
 * rows of the expert-sorted layout that its routes name (the A operand of
 * fp4_grouped_gemm_mx): fp8_quantize_act_scatter's contract with FP4 output.
 *
 * x        bf16 tokens [tokens][ld_x], ld_x >= cols.
 * topk     destinations per token, 1..8.
 * dst_rows device int32 [tokens][topk], -1 for no route; values >= m_total
 *          are ignored. Each row should be named once.
 * q, scale FP4 matrix of m_total rows with K = cols. Rows that no route names
 *          are not written.
 * tokens, cols or m_total == 0: returns FP8Q_OK without launching.
 * Errors: as fp4_quantize_mx; FP8Q_ERR_SHAPE also for topk outside 1..8,
 *         FP8Q_ERR_ALIGN also for dst_rows not 4-byte aligned.
 */
int fp4_quantize_mx_scatter(const uint16_t *x, int64_t tokens, int64_t cols, int64_t ld_x, int32_t topk,
                            const int32_t *dst_rows, int64_t m_total, uint8_t *q, int64_t ld_q, uint32_t *scale,
                            int64_t ld_s, hipStream_t stream);

/*
 * fp4_dequantize_mx -- an FP4 matrix back to row-major values.
 *
 * q, scale FP4 matrix of `rows` rows with K = cols.
 * y        [rows][ld_y], ld_y >= cols; out_dtype FP8Q_OUT_BF16 or
 *          FP8Q_OUT_F32 (every value that fp4_quantize_mx can store is exact
 *          in both). Only the rows x cols window is written.
 * rows or cols == 0: returns FP8Q_OK without launching.
 * Errors: FP8Q_ERR_NULL, FP8Q_ERR_SHAPE, FP8Q_ERR_ALIGN (q not 16-byte, scale
 *         not 4-byte, y not element aligned), FP8Q_ERR_ENUM, FP8Q_ERR_HIP.
 */
int fp4_dequantize_mx(const uint8_t *q, int64_t ld_q, const uint32_t *scale, int64_t ld_s, int64_t rows,
                      int64_t cols, void *y, int64_t ld_y, int out_dtype, hipStream_t stream);

/*
 * fp4_gemm_mx -- C = dequant(A) * dequant(B)^T with FP32 accumulation.
 *
 * a, a_scale  FP4 matrix of m rows with K = k.
 * b, b_scale  FP4 matrix of n rows with K = k (padding past k must be zero
 *             codes in both, as the quantizers write it).
 * c           [m][ldc], ldc >= n; out_dtype FP8Q_OUT_BF16 (rounded once, to
 *             nearest even) or FP8Q_OUT_F32. Every element of the m x n window
 *             is written; k == 0 writes zeros (a, b and scales may be NULL).
 * Any m, n, k >= 0 within the limits, and any ldc. m == 0 or n == 0: returns FP8Q_OK.
 * Errors: FP8Q_ERR_NULL, FP8Q_ERR_SHAPE, FP8Q_ERR_ALIGN (a, b not 16-byte,
 *         scales not 4-byte, c not element aligned), FP8Q_ERR_ENUM,
 *         FP8Q_ERR_HIP.
 */
int fp4_gemm_mx(int64_t m, int64_t n, int64_t k, const uint8_t *a, int64_t ld_a, const uint32_t *a_scale,
                int64_t ld_as, const uint8_t *b, int64_t ld_b, const uint32_t *b_scale, int64_t ld_bs, void *c,
                int64_t ldc, int out_dtype, hipStream_t stream);

/*
 * fp4_grouped_gemm_mx -- the experts' products over an expert-sorted layout.
 *
 * Expert e owns rows [group_offsets[e], group_offsets[e+1]) of A and C; its
 * first group_rows[e] rows are real and get dequant(A_e) * dequant(W_e)^T,
 * the rest of the segment, and the rows from group_offsets[groups] to
 * m_total, are written as zeros whatever A holds there.
 *
 * groups        number of experts, >= 0.
 * group_offsets DEVICE int32[groups + 1]: non-decreasing multiples of 16,
 *               group_offsets[0] == 0, group_offsets[groups] <= m_total (a
 *               program that has not copied the offsets to the host passes
 *               the rows that it set aside).
 * group_rows    DEVICE int32[groups], 0 <= group_rows[e] <= segment e; NULL:
 *               every row of every segment is real.
 * m_total       rows of A and C, % 16 == 0.
 * b, b_scale    expert e's FP4 matrix of n rows at b + e * stride_b (bytes,
 *               % 16 == 0) and b_scale + e * stride_bs (words); strides >= 0.
 * c             [m_total][ldc]; out_dtype as in fp4_gemm_mx.
 * The device arrays are trusted: offsets that break the contract give
 * unspecified output, within the m_total rows.
 * groups, m_total or n == 0: returns FP8Q_OK without launching.
 * Errors: as fp4_gemm_mx; FP8Q_ERR_ALIGN also for group_offsets or group_rows
 *         not 4-byte aligned.
 */
int fp4_grouped_gemm_mx(int32_t groups, const int32_t *group_offsets, const int32_t *group_rows, int64_t m_total,
                        int64_t n, int64_t k, const uint8_t *a, int64_t ld_a, const uint32_t *a_scale,
                        int64_t ld_as, const uint8_t *b, int64_t ld_b, int64_t stride_b, const uint32_t *b_scale,
                        int64_t ld_bs, int64_t stride_bs, void *c, int64_t ldc, int out_dtype, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* FP8Q_MX4_H */
