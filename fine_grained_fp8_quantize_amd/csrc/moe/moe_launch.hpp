// moe_launch.hpp -- launch sizes of the MoE routing kernels (internal, host
// code only).
#pragma once

#include "launch_shape.hpp"

namespace fp8q {
namespace moe {

// The gradient's kernel: four waves of four rows each. One launch takes up to
// kBackwardTokens of a batch (2^31 work-items), longer batches take several.
constexpr int kBackwardThreads = 256;
constexpr int64_t kBackwardRows = 16;  // per workgroup
constexpr int64_t kBackwardTokens = 1LL << 27;

inline LaunchShape backward_shape(int64_t tokens) {
    return {(tokens + kBackwardRows - 1) / kBackwardRows, kBackwardThreads};
}

}  // namespace moe
}  // namespace fp8q
