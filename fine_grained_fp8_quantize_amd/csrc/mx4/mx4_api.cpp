// mx4_api.cpp -- the FP4 microscaling entry points of the C ABI (declared in
// include/fp8q_mx4.h): argument checks on the host, then one launch on the
// caller's stream. Nothing here allocates, frees or synchronizes.
#include "fp8q.h"

#include "host_checks.hpp"
#include "mx4/mx4.h"

namespace {

using namespace fp8q;
using namespace fp8q::mx4;

// Sizes past these cannot be a tensor; below them no product of two sizes
// that the checks or the kernels form overflows 64 bits.
constexpr int64_t kMaxSize = 1LL << 40;
constexpr int64_t kMaxBytes = 1LL << 60;

bool size_ok(int64_t v) { return v >= 0 && v <= kMaxSize; }

int64_t tiles_of(int64_t v, int64_t per) { return ceil_div(v, per); }

// Units of 16 rows x 512 k of `groups` matrices stay below what the launch
// sizes can be computed from.
bool units_ok(int64_t groups, int64_t rows, int64_t k) {
    const int64_t units = mul_limit(tiles_of(rows, kTileRows), tiles_of(k, kGroupK), kMaxSize);
    return units >= 0 && mul_limit(units, groups, kMaxSize) >= 0;
}

// ld row tiles between `outer` slabs of `unit` elements hold the matrix and
// stay addressable.
bool tiles_ok(int64_t outer, int64_t ld, int64_t rt, int64_t unit) {
    return ld >= rt && ld <= kMaxSize && mul_limit(outer, ld, kMaxBytes / unit) >= 0;
}

// An FP4 matrix of `rows` rows with K = k.
int check_matrix(const uint8_t* q, int64_t ld_q, const uint32_t* scale, int64_t ld_s, int64_t rows, int64_t k) {
    if (!q || !scale) return FP8Q_ERR_NULL;
    const int64_t kt = tiles_of(k, kTileK), rt = tiles_of(rows, kTileRows);
    if (!tiles_ok(kt, ld_q, rt, kTileBytes) || !tiles_ok(tiles_of(kt, kGroupTiles), ld_s, rt, 4 * kScaleWords))
        return FP8Q_ERR_SHAPE;
    if (!is_aligned(q, 16) || !is_aligned(scale, 4)) return FP8Q_ERR_ALIGN;
    return FP8Q_OK;
}

int check_gemm(int64_t m, int64_t n, int64_t k, const uint8_t* a, int64_t ld_a, const uint32_t* a_scale,
               int64_t ld_as, const uint8_t* b, int64_t ld_b, const uint32_t* b_scale, int64_t ld_bs, const void* c,
               int64_t ldc, int out_dtype) {
    if (!c) return FP8Q_ERR_NULL;
    if (m > FP4Q_MAX_GEMM_ROWS || n > FP4Q_MAX_GEMM_ROWS || k > FP4Q_MAX_GEMM_K) return FP8Q_ERR_SHAPE;
    if (k > 0) {
        int st = check_matrix(a, ld_a, a_scale, ld_as, m, k);
        if (st == FP8Q_OK) st = check_matrix(b, ld_b, b_scale, ld_bs, n, k);
        if (st != FP8Q_OK) return st;
    }
    if (ldc < n || mul_limit(m, ldc, kMaxBytes / 4) < 0) return FP8Q_ERR_SHAPE;
    if (!is_aligned(c, out_dtype == FP8Q_OUT_F32 ? 4 : 2)) return FP8Q_ERR_ALIGN;
    return FP8Q_OK;
}

GemmArgs gemm_args(int64_t m, int64_t n, int64_t k, const uint8_t* a, int64_t ld_a, const uint32_t* a_scale,
                   int64_t ld_as, const uint8_t* b, int64_t ld_b, const uint32_t* b_scale, int64_t ld_bs, void* c,
                   int64_t ldc, int out_dtype) {
    GemmArgs p = {};
    p.m = (int32_t)m; p.n = (int32_t)n; p.kt = (int32_t)tiles_of(k, kTileK);
    p.a = a; p.ld_a = ld_a; p.a_scale = a_scale; p.ld_as = ld_as;
    p.b = b; p.ld_b = ld_b; p.b_scale = b_scale; p.ld_bs = ld_bs;
    p.c = c; p.ldc = ldc; p.out_f32 = out_dtype == FP8Q_OUT_F32;
    p.c_vec = ldc % 4 == 0 && is_aligned(c, p.out_f32 ? 16 : 8);
    p.scales16 = is_aligned(a_scale, 16) && is_aligned(b_scale, 16);
    p.c_vec16 = ldc % (p.out_f32 ? 4 : 8) == 0 && is_aligned(c, 16);
    return p;
}

}  // namespace

extern "C" {

int fp4_quantize_mx(int32_t groups, const uint16_t* x, int64_t rows, int64_t cols, int64_t ld_x, int64_t stride_x,
                    int tiling, uint8_t* q, int64_t ld_q, int64_t stride_q, uint32_t* scale, int64_t ld_s,
                    int64_t stride_s, hipStream_t stream) {
    if (tiling != FP4Q_TILE_1x32 && tiling != FP4Q_TILE_32x1) return FP8Q_ERR_ENUM;
    if (groups < 0 || !size_ok(rows) || !size_ok(cols)) return FP8Q_ERR_SHAPE;
    if (groups == 0 || rows == 0 || cols == 0) return FP8Q_OK;
    if (!x) return FP8Q_ERR_NULL;
    const bool along_rows = tiling == FP4Q_TILE_1x32;
    const int64_t out_rows = along_rows ? rows : cols, k = along_rows ? cols : rows;
    const int st = check_matrix(q, ld_q, scale, ld_s, out_rows, k);
    if (st != FP8Q_OK) return st;
    if (ld_x < cols || mul_limit(rows, ld_x, kMaxBytes / 2) < 0 || stride_x < 0 || stride_q < 0 || stride_s < 0)
        return FP8Q_ERR_SHAPE;
    const int64_t kt = tiles_of(k, kTileK), kg = tiles_of(kt, kGroupTiles);
    if (groups > 1) {
        // outputs of different matrices must not overlap
        if (stride_q < kt * ld_q * kTileBytes || stride_s < kg * ld_s * kScaleWords) return FP8Q_ERR_SHAPE;
        if (mul_limit(groups, stride_q, kMaxBytes) < 0 || mul_limit(groups, stride_s, kMaxBytes / 4) < 0 ||
            mul_limit(groups, stride_x, kMaxBytes / 2) < 0)
            return FP8Q_ERR_SHAPE;
    }
    if (!is_aligned(x, 2) || (groups > 1 && stride_q % 16 != 0)) return FP8Q_ERR_ALIGN;
    if (!units_ok(groups, out_rows, k)) return FP8Q_ERR_SHAPE;
    if (!launchable(along_rows ? quant_rows_shape(groups, rows, cols) : quant_cols_shape(groups, rows, cols)))
        return FP8Q_ERR_SHAPE;
    QuantArgs p = {};
    p.x = x; p.rows = rows; p.cols = cols; p.ld_x = ld_x; p.stride_x = groups > 1 ? stride_x : 0;
    p.q = q; p.ld_q = ld_q; p.stride_q = groups > 1 ? stride_q : 0;
    p.scale = scale; p.ld_s = ld_s; p.stride_s = groups > 1 ? stride_s : 0;
    p.groups = groups;
    p.vec = is_aligned(x, 16) && ld_x % 8 == 0 && p.stride_x % 8 == 0;
    return hip_status(along_rows ? launch_quant_rows(p, stream) : launch_quant_cols(p, stream));
}

int fp4_quantize_mx_scatter(const uint16_t* x, int64_t tokens, int64_t cols, int64_t ld_x, int32_t topk,
                            const int32_t* dst_rows, int64_t m_total, uint8_t* q, int64_t ld_q, uint32_t* scale,
                            int64_t ld_s, hipStream_t stream) {
    if (!size_ok(tokens) || !size_ok(cols) || !size_ok(m_total) || topk < 1 || topk > 8) return FP8Q_ERR_SHAPE;
    if (tokens == 0 || cols == 0 || m_total == 0) return FP8Q_OK;
    if (!x || !dst_rows) return FP8Q_ERR_NULL;
    const int st = check_matrix(q, ld_q, scale, ld_s, m_total, cols);
    if (st != FP8Q_OK) return st;
    if (ld_x < cols || mul_limit(tokens, ld_x, kMaxBytes / 2) < 0) return FP8Q_ERR_SHAPE;
    if (!is_aligned(x, 2) || !is_aligned(dst_rows, 4)) return FP8Q_ERR_ALIGN;
    if (!units_ok(1, tokens, cols) || !launchable(quant_rows_shape(1, tokens, cols))) return FP8Q_ERR_SHAPE;
    ScatterArgs p = {};
    p.x = x; p.tokens = tokens; p.cols = cols; p.ld_x = ld_x;
    p.topk = topk; p.dst = dst_rows; p.m_total = m_total;
    p.q = q; p.ld_q = ld_q; p.scale = scale; p.ld_s = ld_s;
    p.vec = is_aligned(x, 16) && ld_x % 8 == 0;
    return hip_status(launch_quant_scatter(p, stream));
}

int fp4_dequantize_mx(const uint8_t* q, int64_t ld_q, const uint32_t* scale, int64_t ld_s, int64_t rows,
                      int64_t cols, void* y, int64_t ld_y, int out_dtype, hipStream_t stream) {
    if (out_dtype != FP8Q_OUT_BF16 && out_dtype != FP8Q_OUT_F32) return FP8Q_ERR_ENUM;
    if (!size_ok(rows) || !size_ok(cols)) return FP8Q_ERR_SHAPE;
    if (rows == 0 || cols == 0) return FP8Q_OK;
    if (!y) return FP8Q_ERR_NULL;
    const int st = check_matrix(q, ld_q, scale, ld_s, rows, cols);
    if (st != FP8Q_OK) return st;
    const bool f32 = out_dtype == FP8Q_OUT_F32;
    if (ld_y < cols || mul_limit(rows, ld_y, kMaxBytes / 4) < 0) return FP8Q_ERR_SHAPE;
    if (!is_aligned(y, f32 ? 4 : 2)) return FP8Q_ERR_ALIGN;
    if (!units_ok(1, rows, cols) || !launchable(quant_rows_shape(1, rows, cols))) return FP8Q_ERR_SHAPE;
    DequantArgs p = {};
    p.q = q; p.ld_q = ld_q; p.scale = scale; p.ld_s = ld_s;
    p.rows = rows; p.cols = cols; p.y = y; p.ld_y = ld_y; p.f32 = f32;
    p.vec = is_aligned(y, 16) && ld_y % (f32 ? 4 : 8) == 0;
    return hip_status(launch_dequant(p, stream));
}

int fp4_gemm_mx(int64_t m, int64_t n, int64_t k, const uint8_t* a, int64_t ld_a, const uint32_t* a_scale,
                int64_t ld_as, const uint8_t* b, int64_t ld_b, const uint32_t* b_scale, int64_t ld_bs, void* c,
                int64_t ldc, int out_dtype, hipStream_t stream) {
    if (out_dtype != FP8Q_OUT_BF16 && out_dtype != FP8Q_OUT_F32) return FP8Q_ERR_ENUM;
    if (!size_ok(m) || !size_ok(n) || !size_ok(k)) return FP8Q_ERR_SHAPE;
    if (m == 0 || n == 0) return FP8Q_OK;
    const int st = check_gemm(m, n, k, a, ld_a, a_scale, ld_as, b, ld_b, b_scale, ld_bs, c, ldc, out_dtype);
    if (st != FP8Q_OK) return st;
    // the kernels number output tiles, of 16 x 16 at the least, with 32 bits
    if (!blocks_ok(mul_limit(tiles_of(m, 16), tiles_of(n, 16), kMaxSize))) return FP8Q_ERR_SHAPE;
    const GemmArgs p = gemm_args(m, n, k, a, ld_a, a_scale, ld_as, b, ld_b, b_scale, ld_bs, c, ldc, out_dtype);
    if (!launchable(gemm_shape(gemm_form(m, n, p.scales16), m, n, p.kt))) return FP8Q_ERR_SHAPE;
    return hip_status(launch_gemm(p, stream));
}

int fp4_grouped_gemm_mx(int32_t groups, const int32_t* group_offsets, const int32_t* group_rows, int64_t m_total,
                        int64_t n, int64_t k, const uint8_t* a, int64_t ld_a, const uint32_t* a_scale,
                        int64_t ld_as, const uint8_t* b, int64_t ld_b, int64_t stride_b, const uint32_t* b_scale,
                        int64_t ld_bs, int64_t stride_bs, void* c, int64_t ldc, int out_dtype, hipStream_t stream) {
    if (out_dtype != FP8Q_OUT_BF16 && out_dtype != FP8Q_OUT_F32) return FP8Q_ERR_ENUM;
    if (groups < 0 || !size_ok(m_total) || !size_ok(n) || !size_ok(k)) return FP8Q_ERR_SHAPE;
    if (groups == 0 || m_total == 0 || n == 0) return FP8Q_OK;
    if (!group_offsets) return FP8Q_ERR_NULL;
    const int st = check_gemm(m_total, n, k, a, ld_a, a_scale, ld_as, b, ld_b, b_scale, ld_bs, c, ldc, out_dtype);
    if (st != FP8Q_OK) return st;
    if (m_total % kTileRows != 0 || stride_b < 0 || stride_bs < 0) return FP8Q_ERR_SHAPE;
    if (mul_limit(groups, stride_b, kMaxBytes) < 0 || mul_limit(groups, stride_bs, kMaxBytes / 4) < 0)
        return FP8Q_ERR_SHAPE;
    if (!is_aligned(group_offsets, 4) || !is_aligned(group_rows, 4) || stride_b % 16 != 0) return FP8Q_ERR_ALIGN;
    if (!blocks_ok(mul_limit(m_total / 16 + groups + 1, tiles_of(n, 16), kMaxSize))) return FP8Q_ERR_SHAPE;
    GemmArgs p = gemm_args(m_total, n, k, a, ld_a, a_scale, ld_as, b, ld_b, b_scale, ld_bs, c, ldc, out_dtype);
    p.groups = groups; p.group_offsets = group_offsets; p.group_rows = group_rows;
    p.stride_b = stride_b; p.stride_bs = stride_bs;
    p.scales16 = p.scales16 && (groups == 1 || stride_bs % 4 == 0);
    if (!launchable(grouped_shape(grouped_form(m_total, n, groups, p.scales16), m_total, n, p.kt, groups)))
        return FP8Q_ERR_SHAPE;
    return hip_status(launch_grouped_gemm(p, stream));
}

}  // extern "C"
