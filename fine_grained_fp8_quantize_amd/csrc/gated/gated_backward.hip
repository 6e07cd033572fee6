// gated_backward.hip -- the gradients of gate and up for gfx950.
//
// dG = dH U act'(G), dU = dH act(G): 6 bytes read per element of H, 4 written
// in bf16, 2 in E4M3 along the rows and 2 more along the columns. HBM bounds
// it. Both E4M3 tilings are made in one pass over the inputs: apart they would
// be a pass that writes bf16 and two that read it, 22 bytes instead of 10.
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

__device__ __forceinline__ void gradients(int act, float dh, float g, float u, float& dg, float& du) {
    float slope;
    du = dh * gate_act_slope(act, g, slope);
    dg = dh * u * slope;
}

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
        if constexpr (E4M3) {
            uint32_t top = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) top = umax32(top, __float_as_uint(d[o][i]) & 0x7FFFFFFFu);
            const GroupScale gs = group_scale_f32(__uint_as_float(row16_max(top)));
            const v4f lo = {d[o][0], d[o][1], d[o][2], d[o][3]}, hi = {d[o][4], d[o][5], d[o][6], d[o][7]};
            *reinterpret_cast<uint2*>(static_cast<uint8_t*>(p.out) + row * p.ldo + o * p.n + c) =
                make_uint2(e4m3x4(lo, gs), e4m3x4(hi, gs));
            if (c % 128 == 0) p.out_scale[(o * p.n + c) / 128 * p.ld_os + row] = gs.s;
        } else {
            uint16_t* const dst = static_cast<uint16_t*>(p.out) + row * p.ldo + o * p.n + c;
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = pack_bf16x2(d[o][2 * i], d[o][2 * i + 1]);
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

// Both tilings: a workgroup takes the panel of 128 tokens by 128 columns of
// dG and of dU. Thread (r = t / 16, g = t % 16) has tokens 4 r..4 r + 3 and
// columns 8 g..8 g + 7: a token's 1x128 tile is one row of 16 lanes, a column's
// 128x1 tile the threads of one g, joined over the wave by shuffles and over
// the waves through LDS. Codes along the columns pass through LDS, so that both
// sides write whole 128-byte lines. The 16-byte chunks of a transposed row are
// placed by an XOR with the column's group, so that the 16 groups' writes of
// one row index spread over the banks.
constexpr int kWaves = kPanelThreads / 64;
__device__ __forceinline__ int panel_chunk(int chunk, int col) { return chunk ^ ((col >> 3) & 7); }

__global__ __launch_bounds__(kPanelThreads) void backward_panel_kernel(BackwardArgs p) {
    __shared__ __attribute__((aligned(16))) uint8_t codes[2][128 * 128];
    __shared__ uint32_t red[kWaves][2][128];
    __shared__ float row_s[2][128], col_s[2][128], col_y[2][128];
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
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int k = 0; k < 8; ++k)
            gradients(p.act, dh[i].at(k), gt[i].at(k), up[i].at(k), d[0][i][k], d[1][i][k]);
#pragma unroll
    for (int o = 0; o < 2; ++o) {
        // along the rows
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t top = 0;
#pragma unroll
            for (int k = 0; k < 8; ++k) top = umax32(top, __float_as_uint(d[o][i][k]) & 0x7FFFFFFFu);
            const GroupScale gs = group_scale_f32(__uint_as_float(row16_max(top)));
            const v4f lo = {d[o][i][0], d[o][i][1], d[o][i][2], d[o][i][3]};
            const v4f hi = {d[o][i][4], d[o][i][5], d[o][i][6], d[o][i][7]};
            *reinterpret_cast<uint2*>(static_cast<uint8_t*>(p.out) + (t0 + 4 * r + i) * p.ldo + o * p.n + c0 + 8 * g) =
                make_uint2(e4m3x4(lo, gs), e4m3x4(hi, gs));
            if (g == 0) row_s[o][4 * r + i] = gs.s;
        }
        // the largest of the wave's 16 tokens in each column
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            uint32_t top = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) top = umax32(top, __float_as_uint(d[o][i][k]) & 0x7FFFFFFFu);
            top = umax32(top, (uint32_t)__shfl_xor((int)top, 16));
            top = umax32(top, (uint32_t)__shfl_xor((int)top, 32));
            if (lane < 16) red[wave][o][8 * g + k] = top;
        }
    }
    __syncthreads();
    if (t < 256) {
        const int o = t >> 7, c = t & 127;
        uint32_t top = 0;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) top = umax32(top, red[w][o][c]);
        const GroupScale gs = group_scale_f32(__uint_as_float(top));
        col_s[o][c] = gs.s;
        col_y[o][c] = gs.y;
        p.out_t_scale[tb * p.ld_ts + o * p.n + c0 + c] = gs.s;
        p.out_scale[(o * p.n + c0) / 128 * p.ld_os + t0 + c] = row_s[o][c];
    }
    __syncthreads();
#pragma unroll
    for (int o = 0; o < 2; ++o)
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int c = 8 * g + k;
            GroupScale gs;
            gs.s = col_s[o][c];
            gs.y = col_y[o][c];
            gs.slow = !(gs.s >= kSmallScale);
            const v4f v = {d[o][0][k], d[o][1][k], d[o][2][k], d[o][3][k]};
            *reinterpret_cast<uint32_t*>(&codes[o][c * 128 + panel_chunk(r >> 2, c) * 16 + (r & 3) * 4]) = e4m3x4(v, gs);
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
