// gemv.h -- the kernels of few bf16 rows times FP4 weights: host-side launcher
// (internal; arguments are already validated by gemv_api.cpp).
#pragma once

#include <hip/hip_runtime_api.h>
#include <stdint.h>

#include "gemv/gemv_launch.hpp"

namespace fp8q {
namespace gemv {

struct Args {
    int64_t tokens;
    int32_t topk;
    const int32_t* ids;  // NULL: one matrix
    int32_t first, experts;
    int64_t n, k;
    int32_t kt;          // K tiles
    const uint16_t* x;
    int64_t ld_x, ld_xj;
    bool x_vec;          // rows of x are whole pieces of 16 bytes on 16-byte boundaries
    const uint8_t* w;
    int64_t ld_w, stride_up, stride_w;
    const uint32_t* s;
    int64_t ld_s, stride_ups, stride_s;
    void* y;
    int64_t ld_y;
    bool f32, y_vec;     // four adjacent outputs of a row may be stored together
    bool gated;
    int act;
};

hipError_t launch(const Args& p, hipStream_t stream);

}  // namespace gemv
}  // namespace fp8q
