// gemv_api.cpp -- the weight-only FP4 entry points of the C ABI (declared in
// include/fp8q_gemv.h): argument checks on the host, then one launch on the
// caller's stream. Nothing here allocates, frees or synchronizes.
#include "fp8q.h"

#include "gemv/gemv.h"
#include "host_checks.hpp"

namespace {

using namespace fp8q;
using gemv::Args;
using mx4::ceil_div;

constexpr int64_t kMaxSize = 1LL << 40;
constexpr int64_t kMaxBytes = 1LL << 60;
constexpr int64_t kMaxRows = 64LL * 65535;

bool tiles_ok(int64_t outer, int64_t ld, int64_t rt, int64_t unit) {
    return ld >= rt && ld <= kMaxSize && mul_limit(outer, ld, kMaxBytes / unit) >= 0;
}

bool stride_ok(int64_t count, int64_t stride, int64_t unit) {
    return stride >= 0 && mul_limit(count, stride, kMaxBytes / unit) >= 0;
}

int run(const Args& p, int out_dtype, hipStream_t stream) {
    if (out_dtype != FP8Q_OUT_BF16 && out_dtype != FP8Q_OUT_F32) return FP8Q_ERR_ENUM;
    if (p.tokens < 0 || p.topk < 0 || p.n < 0 || p.k < 0 || p.n > FP4Q_MAX_GEMM_ROWS || p.k > FP4Q_MAX_GEMM_K)
        return FP8Q_ERR_SHAPE;
    if (p.tokens == 0 || p.topk == 0 || p.n == 0) return FP8Q_OK;
    if (p.tokens > kMaxRows) return FP8Q_ERR_SHAPE;
    if (p.ids) {
        if (p.topk > gemv::kMaxTopk || p.tokens * p.topk > gemv::kMaxRoutes || p.experts < 0 ||
            p.experts > gemv::kMaxExperts || p.first < 0 || (int64_t)p.first + p.experts > 0x7FFFFFFFLL)
            return FP8Q_ERR_SHAPE;
        if (!is_aligned(p.ids, 4)) return FP8Q_ERR_ALIGN;
    } else if (p.topk != 1 || p.experts != 1) {
        return FP8Q_ERR_SHAPE;
    }
    if (!p.y) return FP8Q_ERR_NULL;
    const int64_t routes = p.tokens * p.topk;
    if (p.ld_y < p.n || mul_limit(routes, p.ld_y, kMaxBytes / 4) < 0) return FP8Q_ERR_SHAPE;
    if (!is_aligned(p.y, p.f32 ? 4 : 2)) return FP8Q_ERR_ALIGN;
    if (p.k > 0 && p.experts > 0) {
        if (!p.x || !p.w || !p.s) return FP8Q_ERR_NULL;
        const int64_t kt = ceil_div(p.k, mx4::kTileK), rt = ceil_div(p.n, mx4::kTileRows);
        if (!tiles_ok(kt, p.ld_w, rt, mx4::kTileBytes) ||
            !tiles_ok(ceil_div(kt, mx4::kGroupTiles), p.ld_s, rt, 4 * mx4::kScaleWords))
            return FP8Q_ERR_SHAPE;
        // (rows may overlap: they are only read)
        if (!stride_ok(p.tokens, p.ld_x, 2) || !stride_ok(p.topk, p.ld_xj, 2) ||
            !stride_ok(p.experts, p.stride_w, 1) || !stride_ok(p.experts, p.stride_s, 4) ||
            !stride_ok(1, p.stride_up, 1) || !stride_ok(1, p.stride_ups, 4))
            return FP8Q_ERR_SHAPE;
        if (!is_aligned(p.x, 2) || !is_aligned(p.w, 16) || !is_aligned(p.s, 4) || p.stride_w % 16 != 0 ||
            p.stride_up % 16 != 0)
            return FP8Q_ERR_ALIGN;
    }
    if (!launchable({gemv::column_groups(p.n, p.gated), 64 * gemv::max_waves(1)})) return FP8Q_ERR_SHAPE;
    Args a = p;
    a.kt = (int32_t)ceil_div(p.k, mx4::kTileK);
    if (a.experts == 0) a.k = a.kt = 0;  // zeros: nothing is read but the ids
    a.x_vec = is_aligned(p.x, 16) && p.ld_x % 8 == 0 && p.ld_xj % 8 == 0 && p.k % 8 == 0;
    a.y_vec = is_aligned(p.y, p.f32 ? 16 : 8) && p.ld_y % 4 == 0;
    return hip_status(gemv::launch(a, stream));
}

Args common(int64_t tokens, int32_t topk, const int32_t* ids, int32_t first, int32_t experts, int64_t n, int64_t k,
            const uint16_t* x, int64_t ld_x, int64_t ld_xj, const uint8_t* w, int64_t ld_w, int64_t stride_w,
            const uint32_t* s, int64_t ld_s, int64_t stride_s, void* y, int64_t ld_y, int out_dtype) {
    Args p = {};
    p.tokens = tokens; p.topk = topk; p.ids = ids; p.first = first; p.experts = experts;
    p.n = n; p.k = k;
    p.x = x; p.ld_x = ld_x; p.ld_xj = ld_xj;
    p.w = w; p.ld_w = ld_w; p.stride_w = stride_w;
    p.s = s; p.ld_s = ld_s; p.stride_s = stride_s;
    p.y = y; p.ld_y = ld_y; p.f32 = out_dtype == FP8Q_OUT_F32;
    return p;
}

}  // namespace

static_assert(FP4Q_GEMV_MAX_EXPERTS == gemv::kMaxExperts && FP4Q_GEMV_MAX_ROUTES == gemv::kMaxRoutes &&
                  FP4Q_GEMV_MAX_TOPK == gemv::kMaxTopk,
              "the limits in fp8q_gemv.h");

extern "C" {

int fp4_gemv_mx(int64_t tokens, int32_t topk, const int32_t* ids, int32_t first, int32_t experts, int64_t n, int64_t k,
                const uint16_t* x, int64_t ld_x, int64_t ld_xj, const uint8_t* w, int64_t ld_w, int64_t stride_w,
                const uint32_t* w_scale, int64_t ld_ws, int64_t stride_ws, void* y, int64_t ld_y, int out_dtype,
                hipStream_t stream) {
    return run(common(tokens, topk, ids, first, experts, n, k, x, ld_x, ld_xj, w, ld_w, stride_w, w_scale, ld_ws,
                      stride_ws, y, ld_y, out_dtype),
               out_dtype, stream);
}

int fp4_gated_gemv_mx(int64_t tokens, int32_t topk, const int32_t* ids, int32_t first, int32_t experts, int64_t n,
                      int64_t k, const uint16_t* x, int64_t ld_x, int64_t ld_xj, const uint8_t* w, int64_t ld_w,
                      int64_t stride_up, int64_t stride_w, const uint32_t* w_scale, int64_t ld_ws, int64_t stride_ups,
                      int64_t stride_ws, int act, void* y, int64_t ld_y, int out_dtype, hipStream_t stream) {
    if (act != FP8Q_ACT_SILU && act != FP8Q_ACT_GELU) return FP8Q_ERR_ENUM;
    Args p = common(tokens, topk, ids, first, experts, n, k, x, ld_x, ld_xj, w, ld_w, stride_w, w_scale, ld_ws,
                    stride_ws, y, ld_y, out_dtype);
    p.gated = true; p.act = act; p.stride_up = stride_up; p.stride_ups = stride_ups;
    return run(p, out_dtype, stream);
}

}  // extern "C"
