// moe.h -- host-side launchers of the MoE routing kernels (internal;
// arguments are already validated by moe_api.cpp).
#pragma once

#include <hip/hip_runtime_api.h>
#include <stdint.h>

namespace fp8q {
namespace moe {

constexpr int kMaxExperts = 1024;
constexpr int kMaxSeqs = 32768;

struct DispatchArgs {
    const int32_t* ids;
    int64_t routes;  // tokens * topk
    int32_t first, experts, align;
    int32_t* offsets;
    int32_t* rows;
    int32_t* dst;
    int32_t* counts;  // workspace: [parts][experts]
};

// The routes are counted in at most this many parts.
constexpr int kDispatchParts = 64;

hipError_t launch_dispatch(const DispatchArgs& p, hipStream_t stream);

struct BalanceArgs {
    const void* logits;
    bool f32;
    int64_t tokens;
    int32_t experts;
    int64_t ld;
    const int32_t* ids;
    int32_t topk;
    const int32_t* seq_offsets;
    int32_t seqs;
    bool sigmoid;
    float alpha;
    float* loss;
    int32_t* counts;
    float* coef;
    void* workspace;
    // backward only
    const float* grad;
    void* dlogits;
    int64_t ld_d;
    int64_t token0;  // the launch's first token
};

int64_t balance_workspace_bytes(int64_t tokens, int64_t experts, int64_t seqs);
hipError_t launch_balance(const BalanceArgs& p, hipStream_t stream);
hipError_t launch_balance_backward(const BalanceArgs& p, hipStream_t stream);

}  // namespace moe
}  // namespace fp8q
