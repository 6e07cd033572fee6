// gated.h -- the gated feed-forward kernels of libfp8q: host-side launchers
// (internal; arguments are already validated by gated_api.cpp).
#pragma once

#include <hip/hip_runtime_api.h>
#include <stdint.h>

#include "gated/gated_launch.hpp"
#include "launch.h"

namespace fp8q {
namespace gated {

struct GatedArgs {
    GemmProblem g;       // b, b_scale: the gate's; n: columns of one matrix; c: H
    int64_t stride_up;   // bytes from the gate's weights to the up ones
    int64_t stride_ups;  // floats from the gate's scales to the up ones
    int act;
    bool e4m3;           // c holds codes, out_scale their scales
    float* out_scale;
    int64_t ld_os;
    uint16_t* gate_up;
    int64_t ldg;
};

struct BackwardArgs {
    int64_t m, n;
    const uint16_t* dh;
    int64_t ld_dh;
    const uint16_t* gate_up;
    int64_t ldg;
    int act;
    bool e4m3;
    void* out;
    int64_t ldo;
    float* out_scale;
    int64_t ld_os;
    uint8_t* out_t;
    int64_t ld_t;
    float* out_t_scale;
    int64_t ld_ts;
    bool vec;  // bf16 output: rows of all arrays start on 16-byte boundaries
};

// workspace: FP32 [m][n] where E4M3 output of few rows needs it (see
// gated_launch.hpp), else unused.
hipError_t launch_gated(const GatedArgs& p, float* workspace, hipStream_t stream);
hipError_t launch_grouped_gated(const GatedArgs& p, float* workspace, hipStream_t stream);
hipError_t launch_backward(const BackwardArgs& p, hipStream_t stream);

}  // namespace gated
}  // namespace fp8q
