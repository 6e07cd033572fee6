// moe_api.cpp -- the MoE routing entry points of the C ABI (declared in
// include/fp8q_moe.h): argument checks on the host, then the launches on the
// caller's stream. Nothing here allocates, frees or synchronizes.
#include "fp8q.h"

#include "host_checks.hpp"
#include "moe/moe.h"

namespace {

using namespace fp8q;
using namespace fp8q::moe;

constexpr int64_t kMaxInt = 0x7FFFFFFFLL;
constexpr int64_t kMaxBytes = 1LL << 60;

int check_balance(const void* logits, int logits_dtype, int64_t tokens, int32_t experts, int64_t ld,
                  const int32_t* ids, int32_t topk, const int32_t* seq_offsets, int64_t seqs, int score) {
    if (logits_dtype != FP8Q_LOGITS_BF16 && logits_dtype != FP8Q_LOGITS_F32) return FP8Q_ERR_ENUM;
    if (score != FP8Q_SCORE_SOFTMAX && score != FP8Q_SCORE_SIGMOID) return FP8Q_ERR_ENUM;
    if (tokens < 0 || tokens > kMaxInt || experts < 1 || experts > kMaxExperts || topk < 1 ||
        topk > FP8Q_MOE_MAX_TOPK || seqs < 1 || seqs > kMaxSeqs)
        return FP8Q_ERR_SHAPE;
    // a sequence may hold every route: its totals and counts are int32
    if (tokens * topk > kMaxInt) return FP8Q_ERR_SHAPE;
    if (!seq_offsets && seqs != 1) return FP8Q_ERR_NULL;
    if (!is_aligned(seq_offsets, 4)) return FP8Q_ERR_ALIGN;
    if (tokens == 0) return FP8Q_OK;
    if (!logits || !ids) return FP8Q_ERR_NULL;
    if (ld < experts || mul_limit(tokens, ld, kMaxBytes / 4) < 0) return FP8Q_ERR_SHAPE;
    if (!is_aligned(logits, logits_dtype == FP8Q_LOGITS_F32 ? 4 : 2) || !is_aligned(ids, 4)) return FP8Q_ERR_ALIGN;
    return FP8Q_OK;
}

BalanceArgs balance_args(const void* logits, int logits_dtype, int64_t tokens, int32_t experts, int64_t ld,
                         const int32_t* ids, int32_t topk, const int32_t* seq_offsets, int64_t seqs, int score) {
    BalanceArgs p = {};
    p.logits = logits; p.f32 = logits_dtype == FP8Q_LOGITS_F32;
    p.tokens = tokens; p.experts = experts; p.ld = ld;
    p.ids = ids; p.topk = topk;
    p.seq_offsets = seq_offsets; p.seqs = (int32_t)seqs;
    p.sigmoid = score == FP8Q_SCORE_SIGMOID;
    return p;
}

}  // namespace

static_assert(FP8Q_MOE_MAX_EXPERTS == kMaxExperts, "the limit in fp8q_moe.h");
static_assert(FP8Q_MOE_MAX_SEQS == kMaxSeqs, "the limit in fp8q_moe.h");
static_assert(FP8Q_MOE_DISPATCH_WORKSPACE_BYTES == (int64_t)kDispatchParts * kMaxExperts * sizeof(int32_t),
              "the workspace size in fp8q_moe.h holds every part's counts");

extern "C" {

int moe_dispatch(const int32_t* ids, int64_t tokens, int32_t topk, int32_t first, int32_t experts, int32_t align,
                 int32_t* group_offsets, int32_t* group_rows, int32_t* dst_rows, void* workspace,
                 int64_t workspace_bytes, hipStream_t stream) {
    if (tokens < 0 || tokens > kMaxInt || topk < 1 || topk > FP8Q_MOE_MAX_TOPK || experts < 1 ||
        experts > kMaxExperts || align < 1 || first < 0 || (int64_t)first + experts > kMaxInt)
        return FP8Q_ERR_SHAPE;
    if (tokens * topk + (int64_t)experts * (align - 1) > kMaxInt) return FP8Q_ERR_SHAPE;
    if (!group_offsets || !group_rows || !workspace || (tokens > 0 && (!ids || !dst_rows))) return FP8Q_ERR_NULL;
    if (workspace_bytes < FP8Q_MOE_DISPATCH_WORKSPACE_BYTES) return FP8Q_ERR_SHAPE;
    if (!is_aligned(ids, 4) || !is_aligned(group_offsets, 4) || !is_aligned(group_rows, 4) ||
        !is_aligned(dst_rows, 4) || !is_aligned(workspace, 4))
        return FP8Q_ERR_ALIGN;
    DispatchArgs p = {};
    p.ids = ids; p.routes = tokens * topk;
    p.first = first; p.experts = experts; p.align = align;
    p.offsets = group_offsets; p.rows = group_rows; p.dst = dst_rows;
    p.counts = static_cast<int32_t*>(workspace);
    return hip_status(launch_dispatch(p, stream));
}

int64_t moe_balance_workspace_bytes(int64_t tokens, int32_t experts, int64_t seqs) {
    if (tokens < 0 || tokens > kMaxInt || experts < 1 || experts > kMaxExperts || seqs < 1 ||
        seqs > kMaxSeqs)
        return 0;
    return balance_workspace_bytes(tokens, experts, seqs);
}

int moe_balance_loss(const void* logits, int logits_dtype, int64_t tokens, int32_t experts, int64_t ld,
                     const int32_t* ids, int32_t topk, const int32_t* seq_offsets, int64_t seqs, int score,
                     float alpha, float* loss, int32_t* counts, float* coef, void* workspace,
                     int64_t workspace_bytes, hipStream_t stream) {
    const int st = check_balance(logits, logits_dtype, tokens, experts, ld, ids, topk, seq_offsets, seqs, score);
    if (st != FP8Q_OK) return st;
    if (!loss || !counts || !coef || !workspace) return FP8Q_ERR_NULL;
    if (workspace_bytes < balance_workspace_bytes(tokens, experts, seqs)) return FP8Q_ERR_SHAPE;
    if (!is_aligned(loss, 4) || !is_aligned(counts, 4) || !is_aligned(coef, 4) || !is_aligned(workspace, 4))
        return FP8Q_ERR_ALIGN;
    BalanceArgs p = balance_args(logits, logits_dtype, tokens, experts, ld, ids, topk, seq_offsets, seqs, score);
    p.alpha = alpha;
    p.loss = loss; p.counts = counts; p.coef = coef;
    p.workspace = workspace;
    return hip_status(launch_balance(p, stream));
}

int moe_balance_loss_backward(const void* logits, int logits_dtype, int64_t tokens, int32_t experts, int64_t ld,
                              const int32_t* ids, int32_t topk, const int32_t* seq_offsets, int64_t seqs, int score,
                              const float* coef, const float* grad, void* dlogits, int64_t ld_d,
                              hipStream_t stream) {
    const int st = check_balance(logits, logits_dtype, tokens, experts, ld, ids, topk, seq_offsets, seqs, score);
    if (st != FP8Q_OK) return st;
    if (tokens == 0) return FP8Q_OK;
    if (!coef || !dlogits) return FP8Q_ERR_NULL;
    if (ld_d < experts || mul_limit(tokens, ld_d, kMaxBytes / 4) < 0) return FP8Q_ERR_SHAPE;
    if (dlogits == logits && ld_d != ld) return FP8Q_ERR_SHAPE;
    if (!is_aligned(coef, 4) || !is_aligned(grad, 4) || !is_aligned(dlogits, logits_dtype == FP8Q_LOGITS_F32 ? 4 : 2))
        return FP8Q_ERR_ALIGN;
    BalanceArgs p = balance_args(logits, logits_dtype, tokens, experts, ld, ids, topk, seq_offsets, seqs, score);
    p.coef = const_cast<float*>(coef); p.grad = grad; p.dlogits = dlogits; p.ld_d = ld_d;
    return hip_status(launch_balance_backward(p, stream));
}

}  // extern "C"
