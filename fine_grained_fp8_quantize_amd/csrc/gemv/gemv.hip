// gemv.hip -- few bf16 rows times FP4 weights for gfx950.
//
// y[n] = sum_k x[k] w[n][k] 2^(e(n, k / 32)). The weights are streamed from HBM
// straight to registers, a tile of 16 rows x 128 k (1 KB) per load of a wave,
// turned into bf16 with their scales (v_cvt_scalef32_pk_bf16_fp4: exact, a code
// has two significant bits) and multiplied by v_mfma_f32_16x16x32_bf16, whose
// other operand holds up to 16 rows of x: the products are exact, the sums
// FP32. HBM bounds large weights (1 x 16384 x 7168, 62 MB: 14.4 us, 4.3 TB/s; 16
// tokens through 28 of 32 experts' 2 x 2048 x 7168, 437 MB: 79 us, 5.5 TB/s),
// launch, one wait for the loads and the join small ones (1 x 7168 x 2048, 7.8
// MB: 5.2 us; 5 x 2 x 2050 x 7136: 10.7), and the reads of x through the L2 many
// rows (2 bytes an element beside 17/32 of the weights: 2 x 2048 x 7168 with 1
// row 8.1 us, 16: 13.2, 32: 23, 64: 39). All of a wave's x in registers before
// the first product was no faster (5.2 and 10.7 us), and spilled with one group.
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

constexpr int kInFlight = 4;  // tiles of weights that a wave loads at once

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

// Elements k..k + 7 of a row of x, zeros from `end` on. VEC: rows start on
// 16-byte boundaries and `end` is a multiple of 8.
template <bool VEC>
__device__ __forceinline__ bf16x8 load_x(const uint16_t* row, int64_t k, int64_t end) {
    uint4 w = {};
    if constexpr (VEC) {
        if (k < end) w = *reinterpret_cast<const uint4*>(row + k);
    } else {
        uint32_t h[4] = {0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (k + i < end) h[i >> 1] |= (uint32_t)row[k + i] << (16 * (i & 1));
        w = make_uint4(h[0], h[1], h[2], h[3]);
    }
    return __builtin_bit_cast(bf16x8, w);
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
    uint16_t list[kMaxRoutes];  // in no particular order: a row's result does not depend on its place
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

// A workgroup owns 16 MS rows by NT groups of 16 columns (GATED: of 8 gate and 8
// up columns): wave w takes `tiles` K tiles from w * tiles on, with its loads of
// x serving all NT groups; the waves' partials are added in wave order through
// LDS, so the result does not depend on timing.
template <int MS, int NT, bool GATED, bool F32, bool VEC>
__global__ __launch_bounds__(64 * max_waves(MS)) void gemv_kernel(Args p, int tiles) {
    extern __shared__ v4f partial[];  // [waves][NT][MS][64]
    __shared__ Routes found;
    constexpr int COLS = GATED ? 8 : 16;
    constexpr int TI = kInFlight / NT;
    // x of a step: one row tile and up to two K tiles at once, so that all loads of the step are in flight together;
    // one K tile at a time with four of them, one piece of 8 k at a time with more row tiles: more registers would be
    // spilled (1 x 1024 x 512, four K tiles at once: 4.3 instead of 3.1 us).
    constexpr int Q = MS == 1 ? 4 : 1;
    constexpr bool AHEAD = MS == 1 && TI < 4;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
    const int i = lane & 15, b = lane >> 4;
    const int64_t g0 = (int64_t)blockIdx.x * NT, groups = (p.n + COLS - 1) / COLS;
    const bool routed = p.ids != nullptr;
    int expert = 0, rows = 0, row0 = 0;
    if (routed) {
        const bool none = blockIdx.y == gridDim.y - 1;
        expert = find_routes(p, found, (int)blockIdx.y, none);
        if (expert < 0) return;
        rows = found.count;
        if (none) {
            constexpr int QUADS = NT * COLS / 4;
            for (int x = threadIdx.x; x < rows * QUADS; x += blockDim.x)
                store4<F32>(p, found.list[x / QUADS], g0 * COLS + x % QUADS * 4, v4f{0.f, 0.f, 0.f, 0.f});
            return;
        }
    } else {
        row0 = (int)blockIdx.y * 16 * MS;
        rows = (int)min(p.tokens - row0, (int64_t)16 * MS);
    }
    // GATED: rows 0..7 of the MFMA's operand are gate columns, 8..15 up ones
    const bool up = GATED && i >= 8;
    const uint8_t* w[NT];
    const uint32_t* sw[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
        const int64_t n0 = min(g0 + j, groups - 1) * COLS;  // groups past the last repeat it: not stored
        const int r = GATED ? (int)(n0 & 15) + (i & 7) : i;
        w[j] = p.w + expert * p.stride_w + (up ? p.stride_up : 0) + n0 / 16 * mx4::kTileBytes + r * 64 +
               ((b ^ (r >> 2)) & 3) * 16;
        sw[j] = p.s + expert * p.stride_s + (up ? p.stride_ups : 0) + n0 / 16 * mx4::kScaleWords + 4 * r + b;
    }
    const int first = wave * tiles, last = min(first + tiles, p.kt);
    for (int done = 0; done < rows; done += 16 * MS) {
        const int left = rows - done;  // rows of this pass, and behind it
        const uint16_t* xr[MS];
        v4f acc[NT][MS];
#pragma unroll
        for (int s = 0; s < MS; ++s) {
            const int at = done + min(16 * s + i, left - 1);
            const int route = routed ? found.list[at] : row0 + at;
            const int t = route / p.topk;
            xr[s] = p.x + t * p.ld_x + (route - t * p.topk) * p.ld_xj;
#pragma unroll
            for (int j = 0; j < NT; ++j) acc[j][s] = v4f{0.f, 0.f, 0.f, 0.f};
        }
        // (lanes of rows past the last load nothing: zeros)
        int64_t end[MS];
#pragma unroll
        for (int s = 0; s < MS; ++s) end[s] = 16 * s + i < left ? p.k : 0;
        for (int kt = first; kt < last; kt += TI) {
            // Past the wave's last tile that one is loaded again, and counts as zeros (x) times codes of scale 1
            // (finite).
            v4i codes[TI][NT];
            uint32_t words[TI][NT];
            bf16x8 xv[TI][MS][Q];
#pragma unroll
            for (int u = 0; u < TI; ++u) {
                const int64_t t = min(kt + u, last - 1);
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    codes[u][j] =
                        __builtin_nontemporal_load(reinterpret_cast<const v4i*>(w[j] + t * p.ld_w * mx4::kTileBytes));
                    words[u][j] = sw[j][t / mx4::kGroupTiles * p.ld_s * mx4::kScaleWords];
                }
            }
            auto load_row = [&](int u, int s, int q) {
                const int64_t k0 = (int64_t)(kt + u) * mx4::kTileK + 32 * b + 8 * q;
                return load_x<VEC>(xr[s], k0, kt + u < last ? end[s] : 0);
            };
            auto load_tile = [&](int u) {
#pragma unroll
                for (int s = 0; s < MS; ++s)
#pragma unroll
                    for (int q = 0; q < Q; ++q) xv[u][s][q] = load_row(u, s, q);
            };
            if constexpr (AHEAD) {
#pragma unroll
                for (int u = 0; u < TI; ++u) load_tile(u);
            }
#pragma unroll
            for (int u = 0; u < TI; ++u) {
                if constexpr (!AHEAD) {
                    if (kt + u >= last) break;
                    if constexpr (Q == 4) load_tile(u);
                }
                float scale[NT];
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    const uint32_t word = kt + u < last ? words[u][j] >> (8 * ((kt + u) % mx4::kGroupTiles)) : 127u;
                    scale[j] = block_scale(word & 255u);
                }
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    if constexpr (Q == 1) {
#pragma unroll
                        for (int s = 0; s < MS; ++s) xv[u][s][0] = load_row(u, s, q);
                    }
#pragma unroll
                    for (int j = 0; j < NT; ++j) {
                        const bf16x8 wv = dequant8((uint32_t)codes[u][j][q], scale[j]);
#pragma unroll
                        for (int s = 0; s < MS; ++s)
                            acc[j][s] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wv, xv[u][s][q % Q], acc[j][s], 0, 0, 0);
                    }
                }
            }
        }
        if (done > 0) __syncthreads();  // the partials of the rows before have been read
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int s = 0; s < MS; ++s) partial[((wave * NT + j) * MS + s) * 64 + lane] = acc[j][s];
        __syncthreads();
        // a lane's result: row l % 16 of x, columns 4 (l / 16)..; GATED: gate for l < 32, up for the same columns
        // 32 lanes on
        constexpr int LANES = GATED ? 32 : 64, PART = NT * MS * 64;
        for (int x = threadIdx.x; x < NT * MS * LANES; x += blockDim.x) {
            const int l = x % LANES, s = x / LANES % MS, j = x / LANES / MS, row = 16 * s + (l & 15);
            if (row >= left) continue;
            const v4f* const from = partial + (j * MS + s) * 64 + l;
            v4f v = from[0];
            for (int k = 1; k < waves; ++k) v += from[k * PART];
            if constexpr (GATED) {
                v4f u = from[32];
                for (int k = 1; k < waves; ++k) u += from[k * PART + 32];
#pragma unroll
                for (int c = 0; c < 4; ++c) v[c] = gate_act(p.act, v[c]) * u[c];
            }
            const int64_t route = routed ? found.list[done + row] : row0 + done + row;
            const int64_t n = (g0 + j) * COLS + 4 * (l >> 4);
            if (n < p.n) store4<F32>(p, route, n, v);
        }
    }
}

template <int MS, int NT, bool GATED, bool F32>
void launch_nt(const Args& p, const Form& f, dim3 grid, hipStream_t stream) {
    const dim3 block(64 * f.waves);
    const size_t lds = (size_t)f.waves * NT * MS * 64 * sizeof(v4f);
    if (p.x_vec)
        hipLaunchKernelGGL((gemv_kernel<MS, NT, GATED, F32, true>), grid, block, lds, stream, p, f.tiles);
    else
        hipLaunchKernelGGL((gemv_kernel<MS, NT, GATED, F32, false>), grid, block, lds, stream, p, f.tiles);
}

template <int MS, bool GATED, bool F32>
void launch_ms(const Args& p, const Form& f, dim3 grid, hipStream_t stream) {
    if (f.nt == 1) launch_nt<MS, 1, GATED, F32>(p, f, grid, stream);
    else if (f.nt == 2) launch_nt<MS, 2, GATED, F32>(p, f, grid, stream);
    else launch_nt<MS, 4, GATED, F32>(p, f, grid, stream);
}

template <bool GATED, bool F32>
void launch_form(const Args& p, hipStream_t stream) {
    const Form f = form(p.tokens, p.ids ? p.topk : 0, p.experts, p.n, p.k, GATED);
    const dim3 grid((unsigned)ceil_div(column_groups(p.n, GATED), f.nt), (unsigned)f.rows);
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
