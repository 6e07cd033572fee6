// adamw_api.cpp -- the optimizer entry point of the C ABI (declared in
// include/fp8q_adamw.h): argument checks on the host, then the launches on the
// caller's stream. Nothing here allocates, frees or synchronizes.
#include "fp8q.h"

#include <cmath>

#include "adamw/adamw.h"
#include "host_checks.hpp"

namespace {

using namespace fp8q;
using namespace fp8q::adamw;

constexpr int64_t kMaxNumel = 1LL << 40;

int check_tensor(const fp8q_adamw_tensor& t, const void* grad, bool param_f32, bool grad_f32, bool bits8) {
    if (t.numel < 0 || t.numel > kMaxNumel) return FP8Q_ERR_SHAPE;
    if (t.numel == 0 || !grad) return FP8Q_OK;
    if (t.numel > FP8Q_ADAMW_MAX_NUMEL) return FP8Q_ERR_SHAPE;  // (before any other tensor's launch)
    if (!t.param || !t.exp_avg || !t.exp_avg_sq) return FP8Q_ERR_NULL;
    if (bits8 != (t.exp_avg_scale != nullptr) || bits8 != (t.exp_avg_sq_scale != nullptr)) return FP8Q_ERR_NULL;
    if (t.copy && !param_f32) return FP8Q_ERR_ENUM;
    if (!is_aligned(t.param, param_f32 ? 4 : 2) || !is_aligned(grad, grad_f32 ? 4 : 2) || !is_aligned(t.copy, 2) ||
        (!bits8 && (!is_aligned(t.exp_avg, 4) || !is_aligned(t.exp_avg_sq, 4))) ||
        !is_aligned(t.exp_avg_scale, 4) || !is_aligned(t.exp_avg_sq_scale, 4))
        return FP8Q_ERR_ALIGN;
    return FP8Q_OK;
}

}  // namespace

extern "C" {

int adamw_step(int32_t count, const fp8q_adamw_tensor* tensors, const void* const* grads, int param_dtype,
               int grad_dtype, int state_bits, double lr, double beta1, double beta2, double eps, double weight_decay,
               int64_t step, const float* lr_dev, const int64_t* step_dev, const float* grad_scale, uint64_t seed,
               hipStream_t stream) {
    if ((param_dtype != FP8Q_ADAMW_BF16 && param_dtype != FP8Q_ADAMW_F32) ||
        (grad_dtype != FP8Q_ADAMW_BF16 && grad_dtype != FP8Q_ADAMW_F32) || (state_bits != 32 && state_bits != 8))
        return FP8Q_ERR_ENUM;
    if (count < 0 || (!step_dev && step < 1)) return FP8Q_ERR_SHAPE;
    // (comparisons that a NaN fails; eps is an FP32 number in the kernels, and 0 only where the caller's is)
    const float eps32 = (float)eps;
    if (!(beta1 >= 0.0 && beta1 < 1.0) || !(beta2 >= 0.0 && beta2 < 1.0) || !(eps >= 0.0) ||
        !std::isfinite(eps32) || (eps32 == 0.0f && eps > 0.0) || !std::isfinite(lr) || !std::isfinite(weight_decay))
        return FP8Q_ERR_SHAPE;
    if (count == 0) return FP8Q_OK;
    if (!tensors || !grads) return FP8Q_ERR_NULL;
    if (!is_aligned(lr_dev, 4) || !is_aligned(step_dev, 8) || !is_aligned(grad_scale, 4)) return FP8Q_ERR_ALIGN;
    const bool param_f32 = param_dtype == FP8Q_ADAMW_F32, grad_f32 = grad_dtype == FP8Q_ADAMW_F32;
    bool work = false;
    for (int32_t i = 0; i < count; ++i) {
        const int st = check_tensor(tensors[i], grads[i], param_f32, grad_f32, state_bits == 8);
        if (st != FP8Q_OK) return st;
        work |= grads[i] && tensors[i].numel > 0;
    }
    if (!work) return FP8Q_OK;
    Options o = {};
    o.lr = lr; o.beta1 = beta1; o.beta2 = beta2; o.weight_decay = weight_decay;
    o.eps = eps32; o.step = step;
    o.lr_dev = lr_dev; o.step_dev = step_dev; o.grad_scale = grad_scale; o.seed = seed;
    o.param_f32 = param_f32; o.grad_f32 = grad_f32; o.bits8 = state_bits == 8;
    return hip_status(launch_step(count, tensors, grads, o, stream));
}

}  // extern "C"
