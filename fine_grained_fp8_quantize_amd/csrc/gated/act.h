// act.h -- the activations of gated feed-forward blocks, and how their results
// are stored (internal, device code).
#pragma once

#include "fp8q.h"
#include "fp8q_device.h"

namespace fp8q {
namespace {

// 1 / (1 + e^-w). e^-w = 2^t (1 + d ln 2) with t the rounded and d the rest of
// -w log2(e): without d the result would lose |w| places in the last bit. Past
// +-256 the result is 0 or 1 in any case, and d would be the difference of two
// infinities. (An infinite power gives exactly 0, whatever w's factor is.)
__device__ __forceinline__ float logistic(float w) {
    constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;
    constexpr float kLog2eRest = 1.92596299112661746887e-8f;  // log2(e) - kLog2e
    w = __builtin_amdgcn_fmed3f(w, -256.0f, 256.0f);
    const float t = -w * kLog2e;
    const float d = __builtin_fmaf(-w, kLog2eRest, __builtin_fmaf(-w, kLog2e, -t));
    const float e = __builtin_amdgcn_exp2f(t);
    return __builtin_amdgcn_rcpf(1.0f + e * __builtin_fmaf(d, kLn2, 1.0f));
}

// Both activations are g times a logistic function: sigmoid(g), or, as (1 +
// tanh z) / 2 = sigmoid(2z), of 2 sqrt(2/pi) (g + 0.044715 g^3).
constexpr float kGeluScale = 1.59576912160573071176f;  // 2 sqrt(2/pi)
constexpr float kGeluCube = 0.044715f;

__device__ __forceinline__ float gate_share(int act, float g) {
    const float w = act == FP8Q_ACT_SILU ? g : kGeluScale * __builtin_fmaf(kGeluCube * g * g, g, g);
    return logistic(w);
}
__device__ __forceinline__ float gate_act(int act, float g) { return g * gate_share(act, g); }

// Four floats to columns n..n+3 of a row of `cols`, together where they all
// exist and the address allows it (vec): as they are, or as bf16.
template <class V4>
__device__ __forceinline__ void store4_f32(float* dst, const V4& v, int64_t n, int64_t cols, bool vec) {
    if (vec && n + 3 < cols) {
        *reinterpret_cast<V4*>(dst) = v;
    } else {
#pragma unroll
        for (int r = 0; r < 4; ++r)
            if (n + r < cols) dst[r] = v[r];
    }
}
template <class V4>
__device__ __forceinline__ void store4_bf16(uint16_t* dst, const V4& v, int64_t n, int64_t cols, bool vec) {
    const uint32_t lo = pack_bf16x2(v[0], v[1]), hi = pack_bf16x2(v[2], v[3]);
    if (vec && n + 3 < cols) {
        *reinterpret_cast<uint2*>(dst) = make_uint2(lo, hi);
    } else {
        const uint16_t h[4] = {(uint16_t)lo, (uint16_t)(lo >> 16), (uint16_t)hi, (uint16_t)(hi >> 16)};
#pragma unroll
        for (int r = 0; r < 4; ++r)
            if (n + r < cols) dst[r] = h[r];
    }
}

// E4M3 codes of four floats of a group.
template <class V4>
__device__ __forceinline__ uint32_t e4m3x4(const V4& v, const GroupScale& gs) {
    float q[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) q[i] = quot_fast(__builtin_fabsf(v[i]), gs);
    if (gs.slow) {
#pragma unroll
        for (int i = 0; i < 4; ++i) q[i] = quot_slow(__builtin_fabsf(v[i]), gs);
    }
    const uint32_t signs = gather_byte4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                                        __float_as_uint(v[3]), 3);
    return pack_e4m3x4(q[0], q[1], q[2], q[3], signs);
}

}  // namespace
}  // namespace fp8q
