// adamw.h -- the optimizer kernels of libfp8q: argument table and launcher
// (internal; arguments are already validated by adamw_api.cpp).
#pragma once

#include <hip/hip_runtime_api.h>
#include <stdint.h>

#include "fp8q_adamw.h"

namespace fp8q {
namespace adamw {

constexpr int kThreads = 256;

struct Options {
    double lr, beta1, beta2, weight_decay;
    float eps;
    int64_t step;
    const float* lr_dev;
    const int64_t* step_dev;
    const float* grad_scale;
    uint64_t seed;
    bool param_f32, grad_f32, bits8;
};

hipError_t launch_step(int32_t count, const fp8q_adamw_tensor* tensors, const void* const* grads, const Options& o,
                       hipStream_t stream);

}  // namespace adamw
}  // namespace fp8q
