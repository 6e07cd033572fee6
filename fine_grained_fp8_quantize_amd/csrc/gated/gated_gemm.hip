// gated_gemm.hip -- the gated feed-forward products for gfx950.
//
// H = act(A Wg^T) * (A Wu^T), both products as the block-scaled FP8 GEMM makes
// them (gemm.hip). Many rows: its 256 x 256 tile whose B rows alternate by 16
// between gate and up weights of 128 columns (gemm_kernel.h, GATED), so that a
// lane ends with the two products of the same outputs in its registers and H
// is all that has to be written. The 128 columns are one 1x128 tile of H, which
// can be stored as E4M3 without another pass. Few rows: the kernel below.
//
// Tiles, 4096 rows x 2 x 2048 x 7168, H in E4M3 with gate and up kept: 119 us,
// 2.0 PFLOP/s, where the plain product of 4096 columns takes 115; its copies
// from L2 bound it as they do that one (gemm.hip). Experts, 8192 rows at random
// over 32, the same weights each: 311 to 370 us, 1.3 to 1.55 PFLOP/s; 1.4 GB
// come from beyond the L2s, 0.94 of them the weights once. What bounds it is
// that and the last round of the CUs, which few of its tiles may fill (752
// tiles 322 us, 784, one more round, 368).
#include "gated/gated.h"

#include "gemm_kernel.h"

namespace fp8q {
namespace gated {
namespace {

// Few rows of A: the weights are streamed from HBM straight to registers. A
// workgroup owns 16 MS rows by 8 NT columns: the 16 rows of an MFMA's B operand
// are the weights of 8 gate and 8 up columns. Wave w takes the slabs w, w +
// waves, ..., U of them in flight, and promotes each one's products with its
// scales; the waves' FP32 partials are added in wave order through LDS, so the
// result does not depend on timing. 1 row x 2 x 2048 x 7168, 29 MB: 9.4 us, 3.1
// TB/s; 37 rows x 2 x 1000 x 1024: 5.4 us. Launch, one wait for a wave's loads
// (four slabs, all that a wave has) and join are 2.7 us of it (one row, K = 128),
// and the bytes come at 5 TB/s on top (K = 1024: 4.1 us, 2048: 5.1). 16 rows: 12
// us, 64: 22, A being read through the L2 by every workgroup.
struct RowsPiece {
    const uint8_t* b;      // the gate's weights and scales
    const float* b_scale;
    int64_t m0, n0;
    int64_t real_end;      // rows in [real_end, row_hi) are padding: stored as 0
    int64_t row_hi;
};

template <int MS, int NT, int U, bool F32>
__device__ __forceinline__ void gated_rows(const Params& p, const RowsPiece& t, v4f* partial /* [waves][NT][MS][64] */) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
    const int i = lane & 15, g = lane >> 4;
    const int64_t n0 = t.n0, m0 = t.m0;
    const int slabs = (int)(p.k / kSlab);
    // rows and columns past the last ones repeat it: loaded, not stored
    const uint8_t* wrow[NT];
    const float* sb[NT];
#pragma unroll
    for (int c = 0; c < NT; ++c) {
        const int64_t first = n0 + kRowsColumns * c;
        wrow[c] = t.b + (i >= 8 ? p.stride_up : 0) + min(first + (i & 7), p.n - 1) * p.ldb + 16 * g;
        // (an MFMA result's four rows are 4 g..4 g + 3: gate for g < 2)
        sb[c] = t.b_scale + (g >= 2 ? p.stride_ups : 0) + min(first, p.n - 1) / 128 * p.ld_bs;
    }
    const uint8_t* arow[MS];
    const float* sa[MS];
    v4f acc[NT][MS];
#pragma unroll
    for (int s = 0; s < MS; ++s) {
        const int64_t row = min(m0 + 16 * s + i, t.real_end - 1);
        arow[s] = p.a + row * p.lda + 16 * g;
        sa[s] = p.a_scale + row;
#pragma unroll
        for (int c = 0; c < NT; ++c) acc[c][s] = v4f{0.f, 0.f, 0.f, 0.f};
    }
    for (int j0 = wave; j0 < slabs; j0 += U * waves) {
        v4i w[U][NT][2], a[U][MS][2];
        float fb[U][NT], fa[U][MS];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t j = min(j0 + u * waves, slabs - 1);  // past the last slab: skipped below
#pragma unroll
            for (int c = 0; c < NT; ++c) {
                w[u][c][0] = __builtin_nontemporal_load(reinterpret_cast<const v4i*>(wrow[c] + j * kSlab));
                w[u][c][1] = __builtin_nontemporal_load(reinterpret_cast<const v4i*>(wrow[c] + j * kSlab + 64));
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t j = min(j0 + u * waves, slabs - 1);
#pragma unroll
            for (int c = 0; c < NT; ++c) fb[u][c] = sb[c][j];
#pragma unroll
            for (int s = 0; s < MS; ++s) {
                a[u][s][0] = *reinterpret_cast<const v4i*>(arow[s] + j * kSlab);
                a[u][s][1] = *reinterpret_cast<const v4i*>(arow[s] + j * kSlab + 64);
                fa[u][s] = sa[s][j * p.ld_as];
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (j0 + u * waves < slabs) {
#pragma unroll
                for (int c = 0; c < NT; ++c) {
                    const v8i bw = __builtin_shufflevector(w[u][c][0], w[u][c][1], 0, 1, 2, 3, 4, 5, 6, 7);
#pragma unroll
                    for (int s = 0; s < MS; ++s) {
                        const v8i aw = __builtin_shufflevector(a[u][s][0], a[u][s][1], 0, 1, 2, 3, 4, 5, 6, 7);
                        const v4f zero = {0.f, 0.f, 0.f, 0.f};
                        const v4f part = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(bw, aw, zero, 0, 0, 0, 0, 0, 0);
                        const float f = fa[u][s] * fb[u][c];
#pragma unroll
                        for (int r = 0; r < 4; ++r) acc[c][s][r] = __builtin_fmaf(part[r], f, acc[c][s][r]);
                    }
                }
            }
        }
    }
#pragma unroll
    for (int c = 0; c < NT; ++c)
#pragma unroll
        for (int s = 0; s < MS; ++s) partial[((wave * NT + c) * MS + s) * 64 + lane] = acc[c][s];
    __syncthreads();
    for (int x = threadIdx.x; x < NT * MS * 32; x += blockDim.x) {
        const int l = x & 31, s = (x >> 5) % MS, c = (x >> 5) / MS;
        const int64_t m = m0 + 16 * s + (l & 15), n = n0 + kRowsColumns * c + 4 * (l >> 4);
        if (m >= t.row_hi || n >= p.n) continue;
        const v4f* const from = partial + (c * MS + s) * 64 + l;
        v4f gate = from[0], up = from[32];
        for (int w = 1; w < waves; ++w) {
            gate += from[w * NT * MS * 64];
            up += from[w * NT * MS * 64 + 32];
        }
        if (m >= t.real_end) gate = up = v4f{0.f, 0.f, 0.f, 0.f};
        if (p.gate_up != nullptr) {
            uint16_t* const dst = p.gate_up + m * p.ldg + n;
            store4_bf16(dst, gate, n, p.n, p.g_vec);
            store4_bf16(dst + p.n, up, n, p.n, p.u_vec);
        }
        v4f h;
#pragma unroll
        for (int r = 0; r < 4; ++r) h[r] = gate_act(p.act, gate[r]) * up[r];
        if constexpr (F32)
            store4_f32(static_cast<float*>(p.c) + m * p.ldc + n, h, n, p.n, p.h_vec);
        else
            store4_bf16(static_cast<uint16_t*>(p.c) + m * p.ldc + n, h, n, p.n, p.h_vec);
    }
}

template <int MS, int NT, int U, bool F32>
__global__ __launch_bounds__(64 * rows_waves(MS * NT)) void gated_rows_kernel(Params p) {
    extern __shared__ v4f partial[];
    const RowsPiece t = {p.b, p.b_scale, (int64_t)blockIdx.y * 16 * MS, (int64_t)blockIdx.x * kRowsColumns * NT, p.m, p.m};
    gated_rows<MS, NT, U, F32>(p, t, partial);
}

// The experts' form: a workgroup has the 64-row quarter blockIdx.y of the
// layout, whose segments are whole 128 rows, and takes as many 16-row tiles of
// it as hold real rows. A quarter of padding only is written as zeros. (Twice
// the columns for full quarters, as above, is slower here, where the LDS of
// every workgroup has to have room for it: 4 experts of 128 rows, 2 x 512 x
// 7168: 51 us for 40.)
template <bool F32>
__global__ __launch_bounds__(64 * rows_waves(4)) void grouped_rows_kernel(Params p) {
    extern __shared__ v4f partial[];
    RowsPiece t;
    t.m0 = (int64_t)blockIdx.y * 64;
    t.n0 = (int64_t)blockIdx.x * kRowsColumns;
    // the expert: as many as there are segments that end at or before the quarter (every wave counts for itself)
    int e = 0;
    for (int base = 0; base < p.groups; base += 64) {
        const int l = base + (int)(threadIdx.x & 63);
        e += __popcll(__ballot(l < p.groups && p.group_offsets[min(l, p.groups - 1) + 1] <= t.m0));
    }
    e = __builtin_amdgcn_readfirstlane(e);
    if (e >= p.groups) return;
    const int64_t beg = p.group_offsets[e], end = p.group_offsets[e + 1], seg = max(end - beg, (int64_t)0);
    const int64_t real = p.group_rows ? min(max((int64_t)p.group_rows[e], (int64_t)0), seg) : seg;
    t.b = p.b + e * p.stride_b;
    t.b_scale = p.b_scale + e * p.stride_bs;
    t.row_hi = min(t.m0 + 64, min(end, p.m));
    t.real_end = min(beg + real, t.row_hi);
    const int64_t left = t.real_end - t.m0;
    int done = 0;  // rows
    if (left > 32) {
        gated_rows<4, 1, 2, F32>(p, t, partial);
        return;
    }
    if (left > 16) {
        gated_rows<2, 1, 2, F32>(p, t, partial);
        done = 32;
    } else if (left > 0) {
        // (every wave its share of a short K: 4 experts of 16 rows, 2 x 512 x 2048, 12.0 -> 8.3 us)
        if (p.k <= 2 * kSlab * (int64_t)(blockDim.x >> 6))
            gated_rows<1, 1, 2, F32>(p, t, partial);
        else
            gated_rows<1, 1, 4, F32>(p, t, partial);
        done = 16;
    }
    for (int x = threadIdx.x; x < 64 * 2; x += blockDim.x) {
        const int64_t m = t.m0 + (x >> 1), n = t.n0 + 4 * (x & 1);
        if ((x >> 1) < done || m >= t.row_hi || n >= p.n) continue;
        const v4f zero = {0.f, 0.f, 0.f, 0.f};
        if (p.gate_up != nullptr) {
            uint16_t* const dst = p.gate_up + m * p.ldg + n;
            store4_bf16(dst, zero, n, p.n, p.g_vec);
            store4_bf16(dst + p.n, zero, n, p.n, p.u_vec);
        }
        if constexpr (F32)
            store4_f32(static_cast<float*>(p.c) + m * p.ldc + n, zero, n, p.n, p.h_vec);
        else
            store4_bf16(static_cast<uint16_t*>(p.c) + m * p.ldc + n, zero, n, p.n, p.h_vec);
    }
}

// FP32 rows [m][n] to E4M3 codes and scales of 1x128 tiles: 16 lanes per tile.
__global__ __launch_bounds__(256) void quantize_rows_kernel(const float* __restrict__ x, int64_t m, int64_t n,
                                                            uint8_t* __restrict__ q, int64_t ld_q,
                                                            float* __restrict__ scale, int64_t ld_s) {
    const int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x, per = n / 8;
    if (t >= m * per) return;  // whole tiles of 16 lanes
    const int64_t row = t / per, c = (t - row * per) * 8;
    const v4f lo = *reinterpret_cast<const v4f*>(x + row * n + c), hi = *reinterpret_cast<const v4f*>(x + row * n + c + 4);
    uint32_t top = 0;
#pragma unroll
    for (int r = 0; r < 4; ++r)
        top = umax32(top, umax32(__float_as_uint(lo[r]) & 0x7FFFFFFFu, __float_as_uint(hi[r]) & 0x7FFFFFFFu));
    const GroupScale gs = group_scale_f32(__uint_as_float(row16_max(top)));
    *reinterpret_cast<uint2*>(q + row * ld_q + c) = make_uint2(e4m3x4(lo, gs), e4m3x4(hi, gs));
    if (c % 128 == 0) scale[c / 128 * ld_s + row] = gs.s;
}

Params gated_params(const GatedArgs& g) {
    Params p = to_params(g.g);
    p.stride_up = g.stride_up; p.stride_ups = g.stride_ups;
    p.act = g.act;
    p.out_scale = g.out_scale; p.ld_os = g.ld_os;
    p.gate_up = g.gate_up; p.ldg = g.ldg;
    auto vec = [](const void* x, int64_t ld, uintptr_t bytes) {
        return ld % 4 == 0 && reinterpret_cast<uintptr_t>(x) % bytes == 0;
    };
    p.h_vec = vec(p.c, p.ldc, g.g.out_f32 ? 16 : 8);
    p.g_vec = vec(p.gate_up, p.ldg, 8);
    p.u_vec = p.g_vec && p.n % 4 == 0;
    return p;
}

// E4M3 output of the rows kernels: FP32 rows in the workspace, and their codes
// from there.
void to_workspace(Params& p, float* workspace) {
    p.c = workspace;
    p.ldc = p.n;
    p.h_vec = true;
}
void launch_quantize(const GatedArgs& g, const float* workspace, hipStream_t stream) {
    const int64_t blocks = parts_of(g.g.m * g.g.n / 8, 256);
    hipLaunchKernelGGL(quantize_rows_kernel, dim3((unsigned)blocks), dim3(256), 0, stream, workspace, g.g.m, g.g.n,
                       static_cast<uint8_t*>(g.g.c), g.g.ldc, g.out_scale, g.ld_os);
}

template <int MS, int NT, int U>
void launch_rows(const Params& p, RowsForm f, bool f32, hipStream_t stream) {
    const dim3 grid((unsigned)parts_of(p.n, kRowsColumns * NT), (unsigned)parts_of(p.m, 16 * MS)), block(64 * f.waves);
    const size_t lds = (size_t)f.waves * 64 * NT * MS * sizeof(v4f);
    if (f32)
        hipLaunchKernelGGL((gated_rows_kernel<MS, NT, U, true>), grid, block, lds, stream, p);
    else
        hipLaunchKernelGGL((gated_rows_kernel<MS, NT, U, false>), grid, block, lds, stream, p);
}

}  // namespace

hipError_t launch_gated(const GatedArgs& g, float* workspace, hipStream_t stream) {
    Params p = gated_params(g);
    const RowsForm f = rows_form(g.g.m, g.g.n, g.g.k);
    if (f.ms != 0 && (!g.e4m3 || workspace)) {
        if (g.e4m3) to_workspace(p, workspace);
        const bool f32 = g.e4m3 || g.g.out_f32;
        if (f.ms == 1) launch_rows<1, 1, 4>(p, f, f32, stream);
        else if (f.ms == 2) launch_rows<2, 1, 2>(p, f, f32, stream);
        else if (f.nt == 1) launch_rows<4, 1, 2>(p, f, f32, stream);
        else launch_rows<4, 2, 2>(p, f, f32, stream);
        if (g.e4m3) launch_quantize(g, workspace, stream);
        return hipGetLastError();
    }
    const LaunchShape s = tiles_shape(p.m, p.n);
    const dim3 grid((unsigned)s.blocks), block(s.threads);
    if (g.e4m3)
        hipLaunchKernelGGL((gemm_kernel<256, false, false, kDense, false, false, kGatedE4M3>), grid, block, 0, stream, p);
    else if (g.g.out_f32)
        hipLaunchKernelGGL((gemm_kernel<256, false, true, kDense, false, false, kGated>), grid, block, 0, stream, p);
    else
        hipLaunchKernelGGL((gemm_kernel<256, false, false, kDense, false, false, kGated>), grid, block, 0, stream, p);
    return hipGetLastError();
}

hipError_t launch_grouped_gated(const GatedArgs& g, float* workspace, hipStream_t stream) {
    Params p = gated_params(g);
    if (grouped_rows(p.m, p.n, p.group_rows == nullptr) && (!g.e4m3 || workspace)) {
        if (g.e4m3) to_workspace(p, workspace);
        const int waves = grouped_rows_waves(p.k);
        const dim3 grid((unsigned)parts_of(p.n, kRowsColumns), (unsigned)(p.m / 64)), block(64 * waves);
        const size_t lds = (size_t)waves * 64 * 4 * sizeof(v4f);
        if (g.e4m3 || g.g.out_f32)
            hipLaunchKernelGGL((grouped_rows_kernel<true>), grid, block, lds, stream, p);
        else
            hipLaunchKernelGGL((grouped_rows_kernel<false>), grid, block, lds, stream, p);
        if (g.e4m3) launch_quantize(g, workspace, stream);
        return hipGetLastError();
    }
    const LaunchShape s = grouped_shape(p.m, p.n);
    const dim3 grid((unsigned)s.blocks), block(s.threads);
    if (g.e4m3)
        hipLaunchKernelGGL((gemm_kernel<256, false, false, kGroupedM, false, false, kGatedE4M3>), grid, block, 0, stream, p);
    else if (g.g.out_f32)
        hipLaunchKernelGGL((gemm_kernel<256, false, true, kGroupedM, false, false, kGated>), grid, block, 0, stream, p);
    else
        hipLaunchKernelGGL((gemm_kernel<256, false, false, kGroupedM, false, false, kGated>), grid, block, 0, stream, p);
    return hipGetLastError();
}

}  // namespace gated
}  // namespace fp8q
