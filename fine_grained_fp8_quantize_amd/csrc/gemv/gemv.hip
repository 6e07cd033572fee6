// gemv.hip -- few bf16 rows times FP4 weights for gfx950.
//
// y[n] = sum_k x[k] w[n][k] 2^(e(n, k / 32)). The weights are streamed from HBM
// straight to registers, a tile of 16 rows x 128 k (1 KB) per load of a wave,
// turned into bf16 with their scales (v_cvt_scalef32_pk_bf16_fp4: exact, a code
// has two significant bits) and multiplied by v_mfma_f32_16x16x32_bf16, whose
// other operand holds up to 16 rows of x: the products are exact, the sums
// FP32. HBM bounds it, so that 16 rows cost what one does until the reads of x
// through the L2 (2 bytes an element beside 17/32 of the weights) come near.
//
// In a tile's register a lane has one block of 32 k of one row: it goes through
// the MFMA in four steps of 8 k per lane group. The order of k inside an MFMA
// is free as long as both operands share it, so that step q of lane group b
// stands for k = 32 b + 8 q.., and x is read in 16-byte pieces as it lies.
#include "gemv/gemv.h"

#include <hip/hip_runtime.h>

#include "fp8q_device.h"
#include "gated/act.h"

namespace fp8q {
namespace gemv {
namespace {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int kTilesInFlight = 4;

// 2^(byte - 127) as a float (2^-127 is subnormal; 255 is the infinity that
// makes the block's values NaN).
__device__ __forceinline__ float block_scale(uint32_t byte) {
    return __uint_as_float(byte == 0u ? 0x00400000u : byte << 23);
}

__device__ __forceinline__ bf16x8 dequant8(uint32_t codes, float scale) {
    uint4 w;
    w.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 0));
    w.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 1));
    w.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 2));
    w.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 3));
    return __builtin_bit_cast(bf16x8, w);
}

// Elements k..k + 7 of a row of x, zeros from `end` on.
template <bool VEC>
__device__ __forceinline__ bf16x8 load_x(const uint16_t* row, int64_t k, int64_t end) {
    if (VEC && k + 8 <= end) return *reinterpret_cast<const bf16x8*>(row + k);
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (k + i < end) w[i >> 1] |= (uint32_t)row[k + i] << (16 * (i & 1));
    return __builtin_bit_cast(bf16x8, make_uint4(w[0], w[1], w[2], w[3]));
}

template <bool F32>
__device__ __forceinline__ void store4(const Args& p, int64_t route, int64_t n, v4f v) {
    if constexpr (F32)
        store4_f32(static_cast<float*>(p.y) + route * p.ld_y + n, v, n, p.n, p.y_vec);
    else
        store4_bf16(static_cast<uint16_t*>(p.y) + route * p.ld_y + n, v, n, p.n, p.y_vec);
}

// The routes of a workgroup's expert. Which experts have any is a bit mask in
// LDS; workgroup row `slot` takes the slot-th of them, so that a launch needs no
// more rows than there are routes, and every one reads the (few) ids itself.
// The last row of the grid takes the routes that have no expert here.
struct Routes {
    uint32_t mask[kMaxExperts / 32];
    int count;
    uint16_t list[kMaxRoutes];  // in no particular order: a row's result does not depend on the others
};

__device__ __forceinline__ void append(Routes& r, bool mine, int route) {
    const unsigned long long hit = __ballot(mine);
    if (hit == 0) return;  // wave-uniform
    const int lane = threadIdx.x & 63, leader = __ffsll(hit) - 1;
    int at = 0;
    if (lane == leader) at = atomicAdd(&r.count, __popcll(hit));
    at = __shfl(at, leader) + __popcll(hit & ((1ULL << lane) - 1));
    if (mine) r.list[at] = (uint16_t)route;
}

// The expert of row `slot` (experts: none of them), its routes in r.list. -1: no
// such expert. Every thread takes part.
__device__ __forceinline__ int find_routes(const Args& p, Routes& r, int slot, bool none) {
    const int routes = (int)p.tokens * p.topk, tid = threadIdx.x, threads = blockDim.x, lane = tid & 63;
    if (tid < kMaxExperts / 32) r.mask[tid] = 0;
    if (tid == 0) r.count = 0;
    __syncthreads();
    // (every lane of a wave takes part in a step, also where its route is past the last)
    const int steps = (routes + threads - 1) / threads;
    int want = -1;
    if (!none) {
        for (int s = 0; s < steps; ++s) {
            const int i = s * threads + tid;
            const uint32_t e = i < routes ? (uint32_t)p.ids[i] - (uint32_t)p.first : ~0u;
            if (e < (uint32_t)p.experts) atomicOr(&r.mask[e >> 5], 1u << (e & 31));
        }
        __syncthreads();
        // lane l < 32: experts 32 l..32 l + 31
        const uint32_t word = lane < kMaxExperts / 32 ? r.mask[lane] : 0;
        int before = __popc(word);
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int u = __shfl_up(before, d);
            if (lane >= d) before += u;
        }
        const int up_to = before;
        before -= __popc(word);
        const unsigned long long hit = __ballot(lane < 32 && before <= slot && slot < up_to);
        if (hit == 0) return -1;
        const int l = __ffsll(hit) - 1;
        uint32_t bits = (uint32_t)__builtin_amdgcn_readlane((int)word, l);
        int skip = slot - __builtin_amdgcn_readlane(before, l);
        while (skip-- > 0) bits &= bits - 1;
        want = __builtin_amdgcn_readfirstlane(32 * l + __ffs(bits) - 1);
    }
    for (int s = 0; s < steps; ++s) {
        const int i = s * threads + tid;
        const uint32_t e = i < routes ? (uint32_t)p.ids[i] - (uint32_t)p.first : 0u;
        append(r, i < routes && (none ? e >= (uint32_t)p.experts : e == (uint32_t)want), i);
    }
    __syncthreads();
    return none ? p.experts : want;
}

// A workgroup owns 16 MS rows by 16 columns (GATED: 8 gate and 8 up columns):
// wave w takes `tiles` K tiles from w * tiles on, four of them in flight; the
// waves' partials are added in wave order through LDS, so the result does not
// depend on timing.
template <int MS, bool GATED, bool F32, bool VEC>
__global__ __launch_bounds__(64 * kMaxWaves) void gemv_kernel(Args p, int tiles) {
    extern __shared__ v4f partial[];  // [waves][MS][64]
    __shared__ Routes found;
    constexpr int COLS = GATED ? 8 : 16;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
    const int i = lane & 15, b = lane >> 4;
    const int64_t n0 = (int64_t)blockIdx.x * COLS;
    const bool routed = p.ids != nullptr;
    int expert = 0, rows = 0, row0 = 0;
    if (routed) {
        const bool none = blockIdx.y == gridDim.y - 1;
        expert = find_routes(p, found, (int)blockIdx.y, none);
        if (expert < 0) return;
        rows = found.count;
        if (none) {
            for (int x = threadIdx.x; x < rows * (COLS / 4); x += blockDim.x)
                store4<F32>(p, found.list[x / (COLS / 4)], n0 + x % (COLS / 4) * 4, v4f{0.f, 0.f, 0.f, 0.f});
            return;
        }
    } else {
        row0 = (int)blockIdx.y * 16 * MS;
        rows = (int)min(p.tokens - row0, (int64_t)16 * MS);
    }
    // GATED: rows 0..7 of the MFMA's operand are gate columns n0.., 8..15 up ones
    const int r = GATED ? (int)(n0 & 15) + (i & 7) : i;
    const bool up = GATED && i >= 8;
    const uint8_t* const w = p.w + expert * p.stride_w + (up ? p.stride_up : 0) + n0 / 16 * mx4::kTileBytes + r * 64 +
                             ((b ^ (r >> 2)) & 3) * 16;
    const uint32_t* const sw = p.s + expert * p.stride_s + (up ? p.stride_ups : 0) + n0 / 16 * mx4::kScaleWords + 4 * r + b;
    const int first = wave * tiles, last = min(first + tiles, p.kt);
    for (int done = 0; done < rows; done += 16 * MS) {
        const int left = rows - done;  // rows of this pass, and behind it
        const uint16_t* xr[MS];
        v4f acc[MS];
#pragma unroll
        for (int s = 0; s < MS; ++s) {
            const int at = done + min(16 * s + i, left - 1);  // rows past the last repeat it: not stored
            const int route = routed ? found.list[at] : row0 + at;
            const int t = route / p.topk;
            xr[s] = p.x + t * p.ld_x + (route - t * p.topk) * p.ld_xj;
            acc[s] = v4f{0.f, 0.f, 0.f, 0.f};
        }
        for (int kt = first; kt < last; kt += kTilesInFlight) {
            v4i codes[kTilesInFlight];
            uint32_t words[kTilesInFlight];
#pragma unroll
            for (int u = 0; u < kTilesInFlight; ++u) {
                const int64_t t = min(kt + u, last - 1);  // past the wave's last tile: skipped below
                codes[u] = __builtin_nontemporal_load(reinterpret_cast<const v4i*>(w + t * p.ld_w * mx4::kTileBytes));
                words[u] = sw[t / mx4::kGroupTiles * p.ld_s * mx4::kScaleWords];
            }
#pragma unroll
            for (int u = 0; u < kTilesInFlight; ++u) {
                if (kt + u >= last) break;
                const float scale = block_scale((words[u] >> (8 * ((kt + u) % mx4::kGroupTiles))) & 255u);
                const int64_t k0 = (int64_t)(kt + u) * mx4::kTileK + 32 * b;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const bf16x8 wv = dequant8((uint32_t)codes[u][q], scale);
#pragma unroll
                    for (int s = 0; s < MS; ++s) {
                        const bf16x8 xv = load_x<VEC>(xr[s], k0 + 8 * q, p.k);
                        acc[s] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wv, xv, acc[s], 0, 0, 0);
                    }
                }
            }
        }
        if (done > 0) __syncthreads();  // the partials of the rows before have been read
#pragma unroll
        for (int s = 0; s < MS; ++s) partial[(wave * MS + s) * 64 + lane] = acc[s];
        __syncthreads();
        // a lane's result: row l % 16 of x, columns 4 (l / 16)..; GATED: gate for l < 32, up for the same columns
        // 32 lanes on
        constexpr int LANES = GATED ? 32 : 64;
        for (int x = threadIdx.x; x < MS * LANES; x += blockDim.x) {
            const int l = x % LANES, s = x / LANES, row = 16 * s + (l & 15);
            if (row >= left) continue;
            v4f v = partial[s * 64 + l];
            for (int k = 1; k < waves; ++k) v += partial[(k * MS + s) * 64 + l];
            if constexpr (GATED) {
                v4f u = partial[s * 64 + 32 + l];
                for (int k = 1; k < waves; ++k) u += partial[(k * MS + s) * 64 + 32 + l];
#pragma unroll
                for (int j = 0; j < 4; ++j) v[j] = gate_act(p.act, v[j]) * u[j];
            }
            const int64_t route = routed ? found.list[done + row] : row0 + done + row;
            store4<F32>(p, route, n0 + 4 * (l >> 4), v);
        }
    }
}

template <int MS, bool GATED, bool F32>
void launch_ms(const Args& p, const Form& f, dim3 grid, hipStream_t stream) {
    const dim3 block(64 * f.waves);
    const size_t lds = (size_t)f.waves * MS * 64 * sizeof(v4f);
    if (p.x_vec)
        hipLaunchKernelGGL((gemv_kernel<MS, GATED, F32, true>), grid, block, lds, stream, p, f.tiles);
    else
        hipLaunchKernelGGL((gemv_kernel<MS, GATED, F32, false>), grid, block, lds, stream, p, f.tiles);
}

template <bool GATED, bool F32>
void launch_form(const Args& p, hipStream_t stream) {
    // with ids, no expert gets more than the tokens' routes, and mostly one of each token at the most
    const Form f = form(p.tokens, p.k);
    const unsigned columns = (unsigned)column_groups(p.n, GATED);
    const int64_t routes = p.tokens * p.topk;
    const unsigned rows = p.ids ? (unsigned)(routes < p.experts ? routes : p.experts) + 1
                                : (unsigned)ceil_div(p.tokens, 16 * f.ms);
    const dim3 grid(columns, rows);
    if (f.ms == 1) launch_ms<1, GATED, F32>(p, f, grid, stream);
    else if (f.ms == 2) launch_ms<2, GATED, F32>(p, f, grid, stream);
    else launch_ms<4, GATED, F32>(p, f, grid, stream);
}

}  // namespace

hipError_t launch(const Args& p, hipStream_t stream) {
    if (p.gated) {
        if (p.f32) launch_form<true, true>(p, stream);
        else launch_form<true, false>(p, stream);
    } else {
        if (p.f32) launch_form<false, true>(p, stream);
        else launch_form<false, false>(p, stream);
    }
    return hipGetLastError();
}

}  // namespace gemv
}  // namespace fp8q
