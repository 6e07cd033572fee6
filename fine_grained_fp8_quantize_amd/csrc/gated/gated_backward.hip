// gated_backward.hip -- the gradients of gate and up for gfx950.
//
// dG = dH U act'(G), dU = dH act(G): 6 bytes read per element of H, 4 written
// in bf16, 2 in E4M3 along the rows and 2 more along the columns. HBM bounds
// it. Both E4M3 tilings are made in one pass over the inputs: apart they would
// be a pass that writes bf16 and two that read it, 22 bytes instead of 10.
// 8192 x 2048: 38.2 us with both tilings, 4.4 TB/s (16384 x 2048: 66, 5.1), 27.8
// along the rows alone, 4.8 TB/s; 203 x 512: 3.5 us, the launch. A CU holds two
// panels, so that 8192 x 2048 is two rounds whose loads, arithmetic and stores
// overlap little.
#include "gated/gated.h"

#include <hip/hip_runtime.h>

#include "gated/act.h"

namespace fp8q {
namespace gated {
namespace {

typedef float v4f __attribute__((ext_vector_type(4)));

// Eight bf16 as four words, and their floats.
struct Eight {
    uint32_t w[4];
    __device__ __forceinline__ float at(int i) const { return i & 1 ? bf16_hi(w[i >> 1]) : bf16_lo(w[i >> 1]); }
};
template <bool VEC>
__device__ __forceinline__ Eight load8(const uint16_t* p, int64_t left) {
    if constexpr (VEC) {
        const uint4 v = load_nt16(p);
        return {{v.x, v.y, v.z, v.w}};
    } else {
        Eight e = {};
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < left) e.w[i >> 1] |= (uint32_t)p[i] << (16 * (i & 1));
        return e;
    }
}

// The logistic is that of act.h, correction included: with it as many codes as
// in the same formulas in elementary FP32 operations lie on the other side of a
// border from the exact gradient's (8192 x 2048: 58 and 58 of 33.5 million);
// without it, and with 1 / s uncorrected, 123. From +-16 on gelu's share is 0 or
// 1 exactly: the powers of g that would overflow are taken of that (but a NaN
// stays).
__device__ __forceinline__ void gradients(int act, float dh, float g, float u, float& dg, float& du) {
    float w = g, by = 1.0f, c = g;
    if (act != FP8Q_ACT_SILU) {
        c = __builtin_fabsf(g) > 16.0f ? __builtin_copysignf(16.0f, g) : g;
        w = kGeluScale * __builtin_fmaf(kGeluCube * c * c, c, g);
        by = kGeluScale * __builtin_fmaf(3.0f * kGeluCube * c, c, 1.0f);
    }
    const float s = logistic(w);
    const float r = c * (1.0f - s);
    const float ds = dh * s;
    du = ds * g;
    dg = (ds * u) * (act != FP8Q_ACT_SILU ? __builtin_fmaf(r, by, 1.0f) : 1.0f + r);
}

// The scale of a tile and what its quotients take, by the library's contract:
// s = fl(amax / 448), codes of fl(x / s). Both quotients are made of a product
// with a reciprocal and one correction of its residual (Markstein's, as in
// fp8q_device.h): fl(1 / 448) is a constant, and v_rcp_f32 corrected in the
// same way is fl(1 / s) (for every significand of s, compared on the GPU, where
// 1 / s is normal, s < 2^126; a scale is below 2^120). The sign is that of x,
// zeros' included: the residual is negated twice, so that +-0 stays as it is.
// Scales whose residuals may be subnormal, zero, NaN and infinity take divisions.
// The product with fl(1 / s) alone would be 1.8 us less of 38 (8192 x 2048, both
// tilings) and give other codes next to a border.
struct TileScale {
    float s, y;
    bool slow;
};
__device__ __forceinline__ TileScale tile_scale(float amax) {
    constexpr float kBy = 1.0f / kE4M3Max;
    TileScale t;
    const float q = amax * kBy;
    t.s = __builtin_fmaf(__builtin_fmaf(-q, kE4M3Max, amax), kBy, q);
    t.slow = !(t.s >= kSmallScale);
    if (t.slow) t.s = amax / kE4M3Max;
    const float y = __builtin_amdgcn_rcpf(t.s);
    t.y = __builtin_fmaf(__builtin_fmaf(-t.s, y, 1.0f), y, y);
    return t;
}
__device__ __forceinline__ float quotient(float x, const TileScale& t) {
    const float q = x * t.y;
    return __builtin_fmaf(-__builtin_fmaf(q, t.s, -x), t.y, q);
}
__device__ __forceinline__ float slow_quotient(float x, float s) {
    return s == 0.0f ? __builtin_copysignf(0.0f, x) : __builtin_fminf(__builtin_fmaxf(x / s, -kE4M3Max), kE4M3Max);
}
// (the largest quotient may lie a last place above 448, whose code it gets)
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d, const TileScale& t) {
    float q[4] = {quotient(a, t), quotient(b, t), quotient(c, t), quotient(d, t)};
    if (t.slow) {
        q[0] = slow_quotient(a, t.s);
        q[1] = slow_quotient(b, t.s);
        q[2] = slow_quotient(c, t.s);
        q[3] = slow_quotient(d, t.s);
    }
    uint32_t w = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(q[0], q[1], 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(q[2], q[3], (int)w, true);
}
// A NaN is the largest (v_maximum3_f32): its tile gets a scale of NaN, which
// its other elements, zeros among them, could not hide.
__device__ __forceinline__ float max_nan(float a, float b) { return __builtin_elementwise_maximum(a, b); }
__device__ __forceinline__ float max_abs(float m, float a, float b) {
    return max_nan(max_nan(m, __builtin_fabsf(a)), __builtin_fabsf(b));
}
// The largest of 16 lanes' values >= 0, whose bits are ordered as they are (a
// NaN's, of either sign, behind them).
__device__ __forceinline__ float row_max(float m) { return __uint_as_float(row16_max(__float_as_uint(m))); }

// Eight columns of a row per thread; 16 lanes hold a 1x128 tile.
template <bool E4M3, bool VEC>
__global__ __launch_bounds__(kBackwardThreads) void backward_rows_kernel(BackwardArgs p) {
    const uint32_t t = blockIdx.x * kBackwardThreads + threadIdx.x;  // (a launch has fewer than 2^32 threads)
    const uint32_t per = (uint32_t)((p.n + 7) / 8), row = t / per;
    if (row >= p.m) return;  // E4M3: whole tiles
    const int64_t c = (int64_t)(t - row * per) * 8, left = p.n - c;
    const uint16_t* const gate = p.gate_up + row * p.ldg + c;
    const Eight dh = load8<VEC>(p.dh + row * p.ld_dh + c, left);
    const Eight g = load8<VEC>(gate, left), u = load8<VEC>(gate + p.n, left);
    float d[2][8];
#pragma unroll
    for (int i = 0; i < 8; ++i) gradients(p.act, dh.at(i), g.at(i), u.at(i), d[0][i], d[1][i]);
#pragma unroll
    for (int o = 0; o < 2; ++o) {
        const float(&v)[8] = d[o];
        if constexpr (E4M3) {
            float top = 0.0f;
#pragma unroll
            for (int i = 0; i < 8; i += 2) top = max_abs(top, v[i], v[i + 1]);
            const TileScale ts = tile_scale(row_max(top));
            *reinterpret_cast<uint2*>(static_cast<uint8_t*>(p.out) + row * p.ldo + o * p.n + c) =
                make_uint2(codes4(v[0], v[1], v[2], v[3], ts), codes4(v[4], v[5], v[6], v[7], ts));
            if (c % 128 == 0) p.out_scale[(o * p.n + c) / 128 * p.ld_os + row] = ts.s;
        } else {
            uint16_t* const dst = static_cast<uint16_t*>(p.out) + row * p.ldo + o * p.n + c;
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
            if constexpr (VEC) {
                *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (i < left) dst[i] = (uint16_t)(w[i >> 1] >> (16 * (i & 1)));
            }
        }
    }
}

// max(a, b) of two values per lane, one of them kept by each half (HALF: 32
// lanes) or each odd and even row of 16 lanes: the lower lanes get a's maximum
// with their partner's a, the upper ones b's with theirs.
template <int HALF>
__device__ __forceinline__ float fold(float a, float b) {
    const uint32_t x = __float_as_uint(a), y = __float_as_uint(b);
    if constexpr (HALF == 32) {
        const auto r = __builtin_amdgcn_permlane32_swap(x, y, false, false);
        return max_nan(__uint_as_float(r[0]), __uint_as_float(r[1]));
    } else {
        const auto r = __builtin_amdgcn_permlane16_swap(x, y, false, false);
        return max_nan(__uint_as_float(r[0]), __uint_as_float(r[1]));
    }
}

// Both tilings: a workgroup takes the panel of 128 tokens by 128 columns of
// dG and of dU. Thread (r = t / 16, g = t % 16) has tokens 4 r..4 r + 3 and
// columns 8 g..8 g + 7: a token's 1x128 tile is one row of 16 lanes, a column's
// 128x1 tile the threads of one g, joined over a wave's four rows of lanes by
// folding (16 columns' maxima, 8 of each output, end as four in each lane) and
// over the waves through LDS. Codes along the columns pass through LDS, so that
// both sides write whole 128-byte lines. The 16-byte chunks of a transposed row
// are placed by an XOR with the column's group, so that the 16 groups' writes
// of one row index spread over the banks.
constexpr int kWaves = kPanelThreads / 64;
__device__ __forceinline__ int panel_chunk(int chunk, int col) { return chunk ^ ((col >> 3) & 7); }

__global__ __launch_bounds__(kPanelThreads, 4) void backward_panel_kernel(BackwardArgs p) {
    __shared__ __attribute__((aligned(16))) uint8_t codes[2][128 * 128];
    __shared__ float red[kWaves][2][128];
    __shared__ float row_s[2][128];
    __shared__ float2 col_scale[2][128];  // a tile's s and y
    const int t = threadIdx.x, lane = t & 63, wave = t >> 6, g = t & 15, r = t >> 4;
    const int64_t panels = p.n / 128, tb = blockIdx.x / panels, cb = blockIdx.x - tb * panels;
    const int64_t t0 = tb * 128, c0 = cb * 128;

    Eight dh[4], gt[4], up[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t row = t0 + 4 * r + i;
        const uint16_t* const gate = p.gate_up + row * p.ldg + c0 + 8 * g;
        dh[i] = load8<true>(p.dh + row * p.ld_dh + c0 + 8 * g, 8);
        gt[i] = load8<true>(gate, 8);
        up[i] = load8<true>(gate + p.n, 8);
    }
    float d[2][4][8];
    float col[2][8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            gradients(p.act, dh[i].at(k), gt[i].at(k), up[i].at(k), d[0][i][k], d[1][i][k]);
        // along the rows
#pragma unroll
        for (int o = 0; o < 2; ++o) {
            const float(&v)[8] = d[o][i];
            float top = 0.0f;
#pragma unroll
            for (int k = 0; k < 8; k += 2) top = max_abs(top, v[k], v[k + 1]);
            const TileScale ts = tile_scale(row_max(top));
            *reinterpret_cast<uint2*>(static_cast<uint8_t*>(p.out) + (t0 + 4 * r + i) * p.ldo + o * p.n + c0 + 8 * g) =
                make_uint2(codes4(v[0], v[1], v[2], v[3], ts), codes4(v[4], v[5], v[6], v[7], ts));
            if (g == 0) row_s[o][4 * r + i] = ts.s;
        }
    }
    // the largest of the wave's 16 tokens in each column: lanes 0..31 keep dG's, 32..63 dU's, of those even rows of
    // lanes the columns 8 g..8 g + 3, odd ones the next four
#pragma unroll
    for (int o = 0; o < 2; ++o)
#pragma unroll
        for (int k = 0; k < 8; ++k)
            col[o][k] = max_abs(max_abs(0.0f, d[o][0][k], d[o][1][k]), d[o][2][k], d[o][3][k]);
    float half[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) half[k] = fold<32>(col[0][k], col[1][k]);
    v4f mine;
#pragma unroll
    for (int k = 0; k < 4; ++k) mine[k] = fold<16>(half[k], half[k + 4]);
    *reinterpret_cast<v4f*>(&red[wave][lane >> 5][8 * g + 4 * ((lane >> 4) & 1)]) = mine;
    __syncthreads();
    if (t < 256) {
        const int o = t >> 7, c = t & 127;
        float top = 0.0f;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) top = max_nan(top, red[w][o][c]);
        const TileScale ts = tile_scale(top);
        col_scale[o][c] = make_float2(ts.s, ts.y);
        p.out_t_scale[tb * p.ld_ts + o * p.n + c0 + c] = ts.s;
        p.out_scale[(o * p.n + c0) / 128 * p.ld_os + t0 + c] = row_s[o][c];
    }
    __syncthreads();
#pragma unroll
    for (int o = 0; o < 2; ++o)
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int c = 8 * g + k;
            const float2 sy = col_scale[o][c];
            const TileScale ts = {sy.x, sy.y, !(sy.x >= kSmallScale) || sy.x == __builtin_inff()};
            *reinterpret_cast<uint32_t*>(&codes[o][c * 128 + panel_chunk(r >> 2, c) * 16 + (r & 3) * 4]) =
                codes4(d[o][0][k], d[o][1][k], d[o][2][k], d[o][3][k], ts);
        }
    __syncthreads();
#pragma unroll
    for (int o = 0; o < 2; ++o) {
        const int c = t >> 2, part = t & 3;
        uint8_t* const dst = p.out_t + (o * p.n + c0 + c) * p.ld_t + t0 + 32 * part;
#pragma unroll
        for (int h = 0; h < 2; ++h)
            *reinterpret_cast<uint4*>(dst + 16 * h) =
                *reinterpret_cast<const uint4*>(&codes[o][c * 128 + panel_chunk(2 * part + h, c) * 16]);
    }
}

}  // namespace

hipError_t launch_backward(const BackwardArgs& p, hipStream_t stream) {
    const LaunchShape s = p.out_t ? panel_shape(p.m, p.n) : backward_shape(p.m, p.n);
    const dim3 grid((unsigned)s.blocks), block(s.threads);
    if (p.out_t)
        hipLaunchKernelGGL(backward_panel_kernel, grid, block, 0, stream, p);
    else if (p.e4m3)
        hipLaunchKernelGGL((backward_rows_kernel<true, true>), grid, block, 0, stream, p);
    else if (p.vec)
        hipLaunchKernelGGL((backward_rows_kernel<false, true>), grid, block, 0, stream, p);
    else
        hipLaunchKernelGGL((backward_rows_kernel<false, false>), grid, block, 0, stream, p);
    return hipGetLastError();
}

}  // namespace gated
}  // namespace fp8q
