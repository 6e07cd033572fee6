// gated_api.cpp -- the gated feed-forward entry points of the C ABI (declared
// in include/fp8q_gated.h): argument checks on the host, then the launches on
// the caller's stream. Nothing here allocates, frees or synchronizes.
#include "fp8q.h"

#include "gated/gated.h"
#include "host_checks.hpp"

namespace {

using namespace fp8q;
using namespace fp8q::gated;

constexpr int64_t kMaxSize = 1LL << 40;
constexpr int64_t kMaxBytes = 1LL << 60;

bool size_ok(int64_t v) { return v >= 0 && v <= kMaxSize; }

// rows x ld elements of `bytes` each hold `cols` columns and stay addressable
bool matrix_ok(int64_t rows, int64_t cols, int64_t ld, int64_t bytes) {
    return ld >= cols && ld <= kMaxSize && mul_limit(rows, ld, kMaxBytes / bytes) >= 0;
}

bool span_ok(int64_t rows, int64_t ld) {
    return ld >= 0 && ld < FP8Q_MAX_SCALE_SPAN && mul_limit(rows, ld, FP8Q_MAX_SCALE_SPAN - 1) >= 0;
}

int check_gated(int64_t m, int64_t n, int64_t k, const uint8_t* a, int64_t lda, const float* a_scale, int64_t ld_as,
                const uint8_t* b, int64_t ldb, int64_t stride_b, const float* b_scale, int64_t ld_bs,
                int64_t stride_bs, const void* out, int64_t ldo, int out_dtype, const float* out_scale,
                int64_t ld_os, const uint16_t* gate_up, int64_t ldg) {
    const bool e4m3 = out_dtype == FP8Q_OUT_E4M3;
    if (!out || (e4m3 && !out_scale)) return FP8Q_ERR_NULL;
    if (k > 0 && (!a || !a_scale || !b || !b_scale)) return FP8Q_ERR_NULL;
    if (k % 128 != 0 || (e4m3 && n % 128 != 0)) return FP8Q_ERR_SHAPE;
    if (k > 0) {
        if (lda < k || ldb < k || lda > FP8Q_MAX_GEMM_LD || ldb > FP8Q_MAX_GEMM_LD) return FP8Q_ERR_SHAPE;
        if (ld_as < m || ld_bs < k / 128 || !span_ok(k / 128, ld_as) || !span_ok((n + 127) / 128, ld_bs))
            return FP8Q_ERR_SHAPE;
        if (stride_b < 0 || stride_b > kMaxBytes || stride_bs < 0 || stride_bs >= FP8Q_MAX_SCALE_SPAN)
            return FP8Q_ERR_SHAPE;
        if (!is_aligned(a, 16) || !is_aligned(b, 16) || lda % 16 != 0 || ldb % 16 != 0 || stride_b % 16 != 0 ||
            !is_aligned(a_scale, 4) || !is_aligned(b_scale, 4))
            return FP8Q_ERR_ALIGN;
    }
    if (!matrix_ok(m, n, ldo, out_dtype == FP8Q_OUT_F32 ? 4 : 2)) return FP8Q_ERR_SHAPE;
    if (e4m3 && !matrix_ok(n / 128, m, ld_os, 4)) return FP8Q_ERR_SHAPE;
    if (gate_up && !matrix_ok(m, 2 * n, ldg, 2)) return FP8Q_ERR_SHAPE;
    if (e4m3 ? !is_aligned(out, 16) || ldo % 16 != 0 || !is_aligned(out_scale, 4)
             : !is_aligned(out, out_dtype == FP8Q_OUT_F32 ? 4 : 2))
        return FP8Q_ERR_ALIGN;
    if (!is_aligned(gate_up, 2)) return FP8Q_ERR_ALIGN;
    return FP8Q_OK;
}

bool out_ok(int out_dtype) {
    return out_dtype == FP8Q_OUT_BF16 || out_dtype == FP8Q_OUT_F32 || out_dtype == FP8Q_OUT_E4M3;
}
bool act_ok(int act) { return act == FP8Q_ACT_SILU || act == FP8Q_ACT_GELU; }

GatedArgs gated_args(int64_t m, int64_t n, int64_t k, const uint8_t* a, int64_t lda, const float* a_scale,
                     int64_t ld_as, const uint8_t* b, int64_t ldb, int64_t stride_b, const float* b_scale,
                     int64_t ld_bs, int64_t stride_bs, int act, void* out, int64_t ldo, int out_dtype,
                     float* out_scale, int64_t ld_os, uint16_t* gate_up, int64_t ldg) {
    GatedArgs p = {};
    p.g.m = m; p.g.n = n; p.g.k = k;
    p.g.a = a; p.g.lda = lda; p.g.a_scale = a_scale; p.g.ld_as = ld_as;
    p.g.b = b; p.g.ldb = ldb; p.g.b_scale = b_scale; p.g.ld_bs = ld_bs;
    p.g.c = out; p.g.ldc = ldo; p.g.out_f32 = out_dtype == FP8Q_OUT_F32;
    p.stride_up = stride_b; p.stride_ups = stride_bs; p.act = act;
    p.e4m3 = out_dtype == FP8Q_OUT_E4M3; p.out_scale = out_scale; p.ld_os = ld_os;
    p.gate_up = gate_up; p.ldg = ldg;
    return p;
}

}  // namespace

extern "C" {

int64_t fp8_gated_workspace_bytes(int64_t m, int64_t n, int64_t k) {
    if (!size_ok(m) || !size_ok(n) || !size_ok(k) || mul_limit(m, n, kMaxSize) < 0) return 0;
    return workspace_bytes(m, n, k);
}

int64_t fp8_grouped_gated_workspace_bytes(int64_t m_total, int64_t n) {
    if (!size_ok(m_total) || !size_ok(n) || mul_limit(m_total, n, kMaxSize) < 0) return 0;
    return grouped_workspace_bytes(m_total, n);
}

int fp8_gated_gemm(int64_t m, int64_t n, int64_t k, const uint8_t* a, int64_t lda, const float* a_scale,
                   int64_t ld_as, const uint8_t* b, int64_t ldb, int64_t stride_b, const float* b_scale,
                   int64_t ld_bs, int64_t stride_bs, int act, void* out, int64_t ldo, int out_dtype,
                   float* out_scale, int64_t ld_os, uint16_t* gate_up, int64_t ldg, void* workspace,
                   int64_t workspace_bytes, hipStream_t stream) {
    if (!act_ok(act) || !out_ok(out_dtype)) return FP8Q_ERR_ENUM;
    if (!size_ok(m) || !size_ok(n) || !size_ok(k) || workspace_bytes < 0) return FP8Q_ERR_SHAPE;
    if (m == 0 || n == 0) return FP8Q_OK;
    const int st = check_gated(m, n, k, a, lda, a_scale, ld_as, b, ldb, stride_b, b_scale, ld_bs, stride_bs, out, ldo,
                               out_dtype, out_scale, ld_os, gate_up, ldg);
    if (st != FP8Q_OK) return st;
    if (!is_aligned(workspace, 16)) return FP8Q_ERR_ALIGN;
    // (the rows kernel's launches are within kRowsMostPieces by its rule)
    if (mul_limit(m, n, kMaxBytes) < 0 || !launchable(tiles_shape(m, n))) return FP8Q_ERR_SHAPE;
    const GatedArgs p = gated_args(m, n, k, a, lda, a_scale, ld_as, b, ldb, stride_b, b_scale, ld_bs, stride_bs, act,
                                   out, ldo, out_dtype, out_scale, ld_os, gate_up, ldg);
    const bool enough = workspace && workspace_bytes >= fp8q::gated::workspace_bytes(m, n, k);
    return hip_status(launch_gated(p, enough ? static_cast<float*>(workspace) : nullptr, stream));
}

int fp8_grouped_gated_gemm(int32_t groups, const int32_t* group_offsets, const int32_t* group_rows, int64_t m_total,
                           int64_t n, int64_t k, const uint8_t* a, int64_t lda, const float* a_scale, int64_t ld_as,
                           const uint8_t* b, int64_t ldb, int64_t stride_b, int64_t stride_e, const float* b_scale,
                           int64_t ld_bs, int64_t stride_bs, int64_t stride_es, int act, void* out, int64_t ldo,
                           int out_dtype, float* out_scale, int64_t ld_os, uint16_t* gate_up, int64_t ldg,
                           void* workspace, int64_t workspace_bytes, hipStream_t stream) {
    if (!act_ok(act) || !out_ok(out_dtype)) return FP8Q_ERR_ENUM;
    if (groups < 0 || workspace_bytes < 0 || !size_ok(m_total) || !size_ok(n) || !size_ok(k)) return FP8Q_ERR_SHAPE;
    if (groups == 0 || m_total == 0 || n == 0) return FP8Q_OK;
    if (!group_offsets) return FP8Q_ERR_NULL;
    const int st = check_gated(m_total, n, k, a, lda, a_scale, ld_as, b, ldb, stride_b, b_scale, ld_bs, stride_bs, out,
                               ldo, out_dtype, out_scale, ld_os, gate_up, ldg);
    if (st != FP8Q_OK) return st;
    if (m_total % 128 != 0 || m_total > 0x7FFFFFFFLL) return FP8Q_ERR_SHAPE;
    if (k > 0 && (stride_e < 0 || stride_es < 0 || mul_limit(groups, stride_e, kMaxBytes) < 0 ||
                  mul_limit(groups, stride_es, kMaxBytes / 4) < 0))
        return FP8Q_ERR_SHAPE;
    if ((k > 0 && stride_e % 16 != 0) || !is_aligned(group_offsets, 4) || !is_aligned(group_rows, 4) ||
        !is_aligned(workspace, 16))
        return FP8Q_ERR_ALIGN;
    if (!launchable(grouped_shape(m_total, n))) return FP8Q_ERR_SHAPE;
    const int seg = debug_segments(groups, group_offsets, group_rows, m_total, stream);
    if (seg != FP8Q_OK) return seg;
    GatedArgs p = gated_args(m_total, n, k, a, lda, a_scale, ld_as, b, ldb, stride_b, b_scale, ld_bs, stride_bs, act,
                             out, ldo, out_dtype, out_scale, ld_os, gate_up, ldg);
    p.g.groups = groups; p.g.group_offsets = group_offsets; p.g.group_rows = group_rows;
    p.g.stride_b = stride_e; p.g.stride_bs = stride_es;
    const bool enough = workspace && workspace_bytes >= grouped_workspace_bytes(m_total, n);
    return hip_status(launch_grouped_gated(p, enough ? static_cast<float*>(workspace) : nullptr, stream));
}

int fp8_gated_backward(int64_t m, int64_t n, const uint16_t* dh, int64_t ld_dh, const uint16_t* gate_up, int64_t ldg,
                       int act, int out_dtype, void* out, int64_t ldo, float* out_scale, int64_t ld_os,
                       uint8_t* out_t, int64_t ld_t, float* out_t_scale, int64_t ld_ts, hipStream_t stream) {
    if (!act_ok(act) || (out_dtype != FP8Q_OUT_BF16 && out_dtype != FP8Q_OUT_E4M3)) return FP8Q_ERR_ENUM;
    if (!size_ok(m) || !size_ok(n)) return FP8Q_ERR_SHAPE;
    if (m == 0 || n == 0) return FP8Q_OK;
    const bool e4m3 = out_dtype == FP8Q_OUT_E4M3;
    if (!e4m3 && (out_scale || out_t || out_t_scale)) return FP8Q_ERR_ENUM;
    if (!dh || !gate_up || !out || (e4m3 && !out_scale) || (out_t && !out_t_scale)) return FP8Q_ERR_NULL;
    if (!matrix_ok(m, n, ld_dh, 2) || !matrix_ok(m, 2 * n, ldg, 2) || !matrix_ok(m, 2 * n, ldo, 2))
        return FP8Q_ERR_SHAPE;
    if (e4m3) {
        if (n % 128 != 0 || !matrix_ok(2 * n / 128, m, ld_os, 4)) return FP8Q_ERR_SHAPE;
        if (out_t && (m % 128 != 0 || !matrix_ok(2 * n, m, ld_t, 1) || !matrix_ok(m / 128, 2 * n, ld_ts, 4)))
            return FP8Q_ERR_SHAPE;
        if (!is_aligned(dh, 16) || !is_aligned(gate_up, 16) || !is_aligned(out, 16) || !is_aligned(out_t, 16) ||
            ld_dh % 8 != 0 || ldg % 8 != 0 || ldo % 16 != 0 || (out_t && ld_t % 16 != 0) ||
            !is_aligned(out_scale, 4) || !is_aligned(out_t_scale, 4))
            return FP8Q_ERR_ALIGN;
    } else {
        if (!is_aligned(dh, 2) || !is_aligned(gate_up, 2) || !is_aligned(out, 2)) return FP8Q_ERR_ALIGN;
    }
    if (mul_limit(m, parts_of(n, 8), kMaxSize) < 0) return FP8Q_ERR_SHAPE;
    if (!launchable(out_t ? panel_shape(m, n) : backward_shape(m, n))) return FP8Q_ERR_SHAPE;
    BackwardArgs p = {};
    p.m = m; p.n = n;
    p.dh = dh; p.ld_dh = ld_dh; p.gate_up = gate_up; p.ldg = ldg; p.act = act;
    p.e4m3 = e4m3; p.out = out; p.ldo = ldo; p.out_scale = out_scale; p.ld_os = ld_os;
    p.out_t = out_t; p.ld_t = ld_t; p.out_t_scale = out_t_scale; p.ld_ts = ld_ts;
    p.vec = n % 8 == 0 && ld_dh % 8 == 0 && ldg % 8 == 0 && ldo % 8 == 0 && is_aligned(dh, 16) &&
            is_aligned(gate_up, 16) && is_aligned(out, 16);
    return hip_status(launch_backward(p, stream));
}

}  // extern "C"
