// mx4_gemm.hip -- FP4 microscaling products for gfx950.
//
// C[m][n] = sum_k a[m][k] 2^(ea(m, k / 32)) * b[n][k] 2^(eb(n, k / 32)) with
// E2M1 codes a, b: v_mfma_scale_f32_16x16x128_f8f6f4 takes one tile (mx4.h)
// of each operand, applies every block's two exponents and adds into FP32
// accumulators. Each output is rounded once, when it is stored.
//
// As in the FP8 GEMM, the MFMA's row operand is B (n) and its column operand
// is A (m), so that a lane holds four consecutive n of one m.
#include "mx4/mx4.h"

#include "fp8q_device.h"

namespace fp8q {
namespace mx4 {
namespace {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));

constexpr int kFp4 = 4;  // the MFMA's operand format code of E2M1

// acc += (B tile) * (A tile)^T; T: which byte of the scale words applies.
template <int T>
__device__ __forceinline__ v4f mfma_tile(v4i b, v4i a, v4f acc, uint32_t sb, uint32_t sa) {
    const v8i bw = __builtin_shufflevector(b, b, 0, 1, 2, 3, 0, 1, 2, 3);
    const v8i aw = __builtin_shufflevector(a, a, 0, 1, 2, 3, 0, 1, 2, 3);
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(bw, aw, acc, kFp4, kFp4, T, (int)sb, T, (int)sa);
}

// Where lane l's 16 bytes (row l % 16, block l / 16) stand in a tile, and its
// word among the tile's scale words.
__device__ __forceinline__ int lane_code_offset(int lane) {
    const int r = lane & 15;
    return r * 64 + ((lane >> 4) ^ (r >> 2)) * 16;
}
__device__ __forceinline__ int lane_scale_word(int lane) { return 4 * (lane & 15) + (lane >> 4); }

// The rows of one output tile: [m0, row_hi) are stored, those from real_end
// on as zeros (padding of an expert's segment).
struct Rows {
    int64_t m0, row_hi, real_end;
    int expert;
};

// Tile `slot` of the grouped order: expert by expert, tiles of BM rows inside
// each segment [off[e], off[e+1]), then tiles of the rows past the last
// segment (no expert, all padding). The experts are found by a scan over the
// wave: lane l takes segment base + l, a running sum gives the tiles before
// it. Every lane of the wave must take part.
template <int BM>
__device__ __forceinline__ bool grouped_rows(const GemmArgs& p, int64_t slot, Rows& t) {
    const int lane = threadIdx.x & 63;
    for (int base = 0; base <= p.groups; base += 64) {
        const int e = base + lane;
        int64_t beg = 0, end = 0;
        if (e <= p.groups) {
            beg = p.group_offsets[e];
            end = e < p.groups ? p.group_offsets[e + 1] : p.m;
        }
        // offsets that break the contract must not move stores outside C
        beg = beg < 0 ? 0 : (beg > p.m ? p.m : beg);
        end = end < beg ? beg : (end > p.m ? p.m : end);
        const int tiles = (int)((end - beg + BM - 1) / BM);
        int incl = tiles;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int u = __shfl_up(incl, d);
            if (lane >= d) incl += u;
        }
        const int chunk = __builtin_amdgcn_readfirstlane(__shfl(incl, 63));
        if (slot < chunk) {
            const int l = __builtin_amdgcn_readfirstlane(__ffsll((unsigned long long)__ballot(incl > slot)) - 1);
            const int before = __shfl(incl - tiles, l);
            const int64_t seg = __shfl((int)beg, l), seg_end = __shfl((int)end, l);
            t.expert = __builtin_amdgcn_readfirstlane(base + l);
            t.m0 = seg + (slot - before) * BM;
            t.row_hi = min(seg_end, t.m0 + BM);
            int64_t real = seg;  // no expert: nothing is real
            if (t.expert < p.groups) {
                real = seg_end;
                if (p.group_rows) {
                    const int64_t rows = max(p.group_rows[t.expert], 0);
                    real = min(seg + rows, seg_end);
                }
            }
            t.real_end = real;
            return true;
        }
        slot -= chunk;
    }
    return false;
}

template <bool F32>
__device__ __forceinline__ void store4(const GemmArgs& p, int64_t m, int64_t n, v4f v) {
    if constexpr (F32) {
        float* const c = static_cast<float*>(p.c) + m * p.ldc + n;
        if (p.c_vec && n + 4 <= p.n) {
            *reinterpret_cast<v4f*>(c) = v;
        } else {
#pragma unroll
            for (int r = 0; r < 4; ++r)
                if (n + r < p.n) c[r] = v[r];
        }
    } else {
        uint16_t* const c = static_cast<uint16_t*>(p.c) + m * p.ldc + n;
        const uint32_t lo = pack_bf16x2(v[0], v[1]), hi = pack_bf16x2(v[2], v[3]);
        if (p.c_vec && n + 4 <= p.n) {
            *reinterpret_cast<uint2*>(c) = make_uint2(lo, hi);
        } else {
            const uint16_t h[4] = {(uint16_t)lo, (uint16_t)(lo >> 16), (uint16_t)hi, (uint16_t)(hi >> 16)};
#pragma unroll
            for (int r = 0; r < 4; ++r)
                if (n + r < p.n) c[r] = h[r];
        }
    }
}

// ------------------------------------------------------------ few rows

// Few rows of A: the weights are streamed from HBM straight to registers. A
// workgroup owns 16 MS x 16 outputs; its waves take K groups in turn (wave w
// the groups w, w + waves, ...) and their FP32 partials are added in wave
// order through LDS, so the result does not depend on timing.
constexpr int kMaxWaves = 16;

template <int MS, bool F32, bool GROUPED>
__global__ __launch_bounds__(64 * kMaxWaves) void gemm_rows_kernel(GemmArgs p, int64_t tiles_n) {
    extern __shared__ v4f partial[];  // [waves][MS][64]
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
    const int64_t tn = (int64_t)blockIdx.x % tiles_n, tm = (int64_t)blockIdx.x / tiles_n;
    Rows t;
    if constexpr (GROUPED) {
        if (!grouped_rows<16 * MS>(p, tm, t)) return;
    } else {
        t = Rows{tm * 16 * MS, min(p.m, (tm + 1) * 16 * MS), p.m, 0};
    }
    v4f acc[MS];
#pragma unroll
    for (int s = 0; s < MS; ++s) acc[s] = v4f{0.f, 0.f, 0.f, 0.f};

    if (t.m0 < t.real_end) {
        const uint8_t* const qa = p.a + lane_code_offset(lane);
        const uint32_t* const sa = p.a_scale + lane_scale_word(lane);
        const uint8_t* const qb = p.b + (GROUPED ? t.expert * p.stride_b : 0) + tn * kTileBytes + lane_code_offset(lane);
        const uint32_t* const sb =
            p.b_scale + (GROUPED ? t.expert * p.stride_bs : 0) + tn * kScaleWords + lane_scale_word(lane);
        // row tiles past the last real row are loaded from it and not stored
        int64_t rt[MS];
#pragma unroll
        for (int s = 0; s < MS; ++s) rt[s] = min(t.m0 / 16 + s, (t.real_end - 1) / 16);
        for (int64_t g = wave; g * kGroupTiles < p.kt; g += waves) {
            const uint32_t swb = sb[g * p.ld_bs * kScaleWords];
            uint32_t swa[MS];
#pragma unroll
            for (int s = 0; s < MS; ++s) swa[s] = sa[(g * p.ld_as + rt[s]) * kScaleWords];
            v4i fb[kGroupTiles], fa[kGroupTiles][MS];
#pragma unroll
            for (int i = 0; i < kGroupTiles; ++i) {
                // past the last K tile the products are skipped below
                const int64_t kt = min(g * kGroupTiles + i, p.kt - 1);
                fb[i] = *reinterpret_cast<const v4i*>(qb + kt * p.ld_b * kTileBytes);
#pragma unroll
                for (int s = 0; s < MS; ++s)
                    fa[i][s] = *reinterpret_cast<const v4i*>(qa + (kt * p.ld_a + rt[s]) * kTileBytes);
            }
#pragma unroll
            for (int s = 0; s < MS; ++s) acc[s] = mfma_tile<0>(fb[0], fa[0][s], acc[s], swb, swa[s]);
            if (g * kGroupTiles + 1 < p.kt) {
#pragma unroll
                for (int s = 0; s < MS; ++s) acc[s] = mfma_tile<1>(fb[1], fa[1][s], acc[s], swb, swa[s]);
            }
            if (g * kGroupTiles + 2 < p.kt) {
#pragma unroll
                for (int s = 0; s < MS; ++s) acc[s] = mfma_tile<2>(fb[2], fa[2][s], acc[s], swb, swa[s]);
            }
            if (g * kGroupTiles + 3 < p.kt) {
#pragma unroll
                for (int s = 0; s < MS; ++s) acc[s] = mfma_tile<3>(fb[3], fa[3][s], acc[s], swb, swa[s]);
            }
        }
    }
#pragma unroll
    for (int s = 0; s < MS; ++s) partial[(wave * MS + s) * 64 + lane] = acc[s];
    __syncthreads();
    for (int i = threadIdx.x; i < MS * 64; i += blockDim.x) {
        v4f v = partial[i];
        for (int w = 1; w < waves; ++w) v += partial[w * MS * 64 + i];
        const int l = i & 63;
        const int64_t m = t.m0 + (i >> 6) * 16 + (l & 15), n = tn * 16 + 4 * (l >> 4);
        if (m >= t.row_hi) continue;
        if (m >= t.real_end) v = v4f{0.f, 0.f, 0.f, 0.f};
        store4<F32>(p, m, n, v);
    }
}

template <int MS, bool GROUPED>
hipError_t dispatch_rows(const GemmArgs& p, int64_t tiles_m, hipStream_t stream) {
    const int64_t tiles_n = (p.n + 15) / 16, kg = (p.kt + kGroupTiles - 1) / kGroupTiles;
    const int64_t rounds = kg > 0 ? (kg + kMaxWaves - 1) / kMaxWaves : 1;
    const int waves = kg > 0 ? (int)((kg + rounds - 1) / rounds) : 1;
    const dim3 grid((unsigned)(tiles_m * tiles_n)), block(64 * waves);
    const size_t lds = (size_t)waves * MS * 64 * sizeof(v4f);
    if (p.out_f32)
        hipLaunchKernelGGL((gemm_rows_kernel<MS, true, GROUPED>), grid, block, lds, stream, p, tiles_n);
    else
        hipLaunchKernelGGL((gemm_rows_kernel<MS, false, GROUPED>), grid, block, lds, stream, p, tiles_n);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_gemm(const GemmArgs& p, hipStream_t stream) {
    if (p.m <= 16) return dispatch_rows<1, false>(p, 1, stream);
    if (p.m <= 32) return dispatch_rows<2, false>(p, 1, stream);
    return dispatch_rows<4, false>(p, (p.m + 63) / 64, stream);
}

hipError_t launch_grouped_gemm(const GemmArgs& p, hipStream_t stream) {
    // at most one ragged tile per segment, and one past the last
    const int64_t avg = p.m / p.groups;
    if (avg <= 16) return dispatch_rows<1, true>(p, p.m / 16 + p.groups + 1, stream);
    if (avg <= 32) return dispatch_rows<2, true>(p, p.m / 32 + p.groups + 1, stream);
    return dispatch_rows<4, true>(p, p.m / 64 + p.groups + 1, stream);
}

}  // namespace mx4
}  // namespace fp8q
