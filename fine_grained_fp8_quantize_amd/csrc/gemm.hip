// gemm.hip -- block-scaled FP8 GEMM for gfx950 (Fprop, Dgrad, Wgrad, grouped).
//
// C[m][n] = sum_j sA[j][m] * sB(n, j) * P_j[m][n], where P_j is the FP32 sum
// of the FP8 products of 128-element K slab j. This is the pages' promotion
// scheme: partial products of one 128-element interval (page inprokorea.com
// free board, passage on the four-WGMMA accumulation interval) are moved into
// full-precision FP32 accumulators, where the per-group scales are applied
// (page "Deepseek Ai News Expert Interview", passage on copying partial
// results to FP32 registers; page "Is aI Hitting a Wall?", passage on the
// dequantization overhead).
//
// gfx950 mapping: one v_mfma_f32_16x16x128_f8f6f4 consumes exactly one slab
// for a 16x16 subtile and returns P_j in fresh registers (C operand 0); the
// promotion is one v_fma_f32 per output element per slab on the vector ALU,
// overlapped with the next subtile's MFMA. The interval is set by the
// scales: measured on gfx950, chaining the MFMA accumulator across slabs
// gives the same error as promoting each slab, and what precision is lost
// is lost inside the instruction's own 128-product sum.
//
// Tiling: 256 (m) x BN (n) block tiles, BN = 256 or 224, 8 waves (4 along
// m x 2 along n), 64 x BN/2 per wave. BN = 224 makes N = 7168 (Dgrad, Wgrad)
// an exact multiple, so those grids are whole waves of the 256 CUs. Each
// 128-byte K slab of the A and B tiles is copied global -> LDS by the direct
// LDS-DMA load (global_load_lds_dwordx4) -- two stages, or for grouped-over-M
// tiles two A and three B stages -- with 16-byte chunks XOR-swizzled by row.
//
// Modes: one GEMM; grouped over M (MoE Fprop/Dgrad); grouped over K (MoE
// Wgrad); one GEMM of several rounds of whole tiles, run by one looping block
// per CU that copies each next tile's first slab during the last slab of the
// tile before (Dgrad-like shapes: short K, several rounds).
// Two more dense variants accumulate in place across slabs instead
// of promoting: microscaling operands (E8M0 block scales applied by the
// scaled MFMA) and one scale per tensor (applied in the epilogue).
// The MFMA computes the transposed tile: its row operand is B (n), its column
// operand is A (m), so every lane holds four consecutive n of one m -- one A
// scale per lane per m-subtile, and the B block scale is wave-uniform per
// 16-column subtile. Waves whose rows are all past the real rows (grouped
// padding, ragged M) skip their MFMAs.
#include "fp8q.h"
#include "gemm_kernel.h"

#include <algorithm>
#include <mutex>

namespace fp8q {
namespace {

// Sum of the K pieces of each split tile of a grouped GEMM's last round
// (see tail_split), in piece order, stored to C as the GEMM stores a whole
// tile: rows past row_hi untouched, padding rows zero. The work is cut into
// units of 256 output vectors (an eighth of one GEMM wave's 64 x 128 outputs,
// in its fragment order), 64 per tail tile; block b takes units b, b + grid,
// ..., one vector per thread: the blocks get equal shares, every load
// instruction reads 1 KB contiguous per wave, and a unit's partial loads and
// its tile record (written by the tile's first piece) are in flight together.
// When nothing was split the blocks return after the scan.
constexpr int kFixupThreads = 256;
constexpr int kFixupBlocks = 1024;

template <bool OUT_F32>
__global__ __launch_bounds__(kFixupThreads) void grouped_fixup_kernel(Params p) {
    constexpr int BN = 256, WN = BN / 2, NSUB = WN / 16;
    constexpr int kItems = NSUB * kMSub * 64;           // one GEMM wave's partial, in v4f
    constexpr int kUnits = 8 * kItems / kFixupThreads;  // units per tile
    const TailSplit ts = tail_split<BN>(p);
    if (ts.split < 2) return;
    const v4f* const part = reinterpret_cast<const v4f*>(p.split_ws);
    for (int unit = (int)blockIdx.x; unit < ts.tiles * kUnits; unit += (int)gridDim.x) {
        const int r = unit / kUnits;
        const int flat = (unit % kUnits) * kFixupThreads + (int)threadIdx.x;  // in [0, 8 kItems)
        const int w = flat / kItems, item = flat % kItems;
        v4f pv[kMaxSplit];
#pragma unroll
        for (int i = 0; i < kMaxSplit; ++i)
            if (i < ts.split) pv[i] = part[((int64_t)(i * ts.tiles + r) * 8 + w) * kItems + item];
        const TailRecord tr = p.split_records[r];
        const int lane = item & 63, s = (item >> 6) % kMSub, t = (item >> 6) / kMSub;
        const int64_t m = tr.m0 + (w >> 1) * kWaveM + s * 16 + (lane & 15);
        const int64_t n = tr.n0 + (w & 1) * WN + t * 16 + 4 * (lane >> 4);
        // (offsets that break the contract can leave a piece unrun and its
        // record from an earlier call: the stores still stay inside C)
        if (m >= tr.row_hi || m >= p.m || tr.m0 < 0 || tr.n0 < 0) continue;
        v4f v = {0.f, 0.f, 0.f, 0.f};
        if (m < tr.real_end) {
#pragma unroll
            for (int i = 0; i < kMaxSplit; ++i)
                if (i < ts.split) v += pv[i];
        }
        if constexpr (OUT_F32) {
            float* dst = reinterpret_cast<float*>(p.c) + m * p.ldc + n;
            if (n + 3 < p.n) {
                *reinterpret_cast<v4f*>(dst) = v;
            } else {
                for (int q = 0; q < 4; ++q)
                    if (n + q < p.n) dst[q] = v[q];
            }
        } else {
            uint16_t* dst = reinterpret_cast<uint16_t*>(p.c) + m * p.ldc + n;
            const uint32_t lo = pack_bf16x2(v[0], v[1]), hi = pack_bf16x2(v[2], v[3]);
            if (n + 3 < p.n) {
                *reinterpret_cast<uint2*>(dst) = make_uint2(lo, hi);
            } else {
                const uint16_t h[4] = {(uint16_t)lo, (uint16_t)(lo >> 16), (uint16_t)hi, (uint16_t)(hi >> 16)};
                for (int q = 0; q < 4; ++q)
                    if (n + q < p.n) dst[q] = h[q];
            }
        }
    }
}

// blocks: the dense slots rounded up to a multiple of 8.
template <int BN>
hipError_t dispatch_dense(const GemmProblem& g, int64_t blocks, hipStream_t stream) {
    const Params p = to_params(g);
    const dim3 grid((unsigned)blocks), block(kThreads);
    if (g.b_rowscale) {
        if (g.out_f32)
            hipLaunchKernelGGL((gemm_kernel<BN, true, true, kDense>), grid, block, 0, stream, p);
        else
            hipLaunchKernelGGL((gemm_kernel<BN, true, false, kDense>), grid, block, 0, stream, p);
    } else {
        if (g.out_f32)
            hipLaunchKernelGGL((gemm_kernel<BN, false, true, kDense>), grid, block, 0, stream, p);
        else
            hipLaunchKernelGGL((gemm_kernel<BN, false, false, kDense>), grid, block, 0, stream, p);
    }
    return hipGetLastError();
}

// A dense GEMM of several rounds of whole tiles: 256 blocks, one per CU,
// each looping over its tiles (see dense_tile).
template <int BN>
hipError_t dispatch_rounds(const GemmProblem& g, hipStream_t stream) {
    const Params p = to_params(g);
    const dim3 grid(256), block(kThreads);
    if (g.b_rowscale) {
        if (g.out_f32)
            hipLaunchKernelGGL((gemm_kernel<BN, true, true, kDenseRounds>), grid, block, 0, stream, p);
        else
            hipLaunchKernelGGL((gemm_kernel<BN, true, false, kDenseRounds>), grid, block, 0, stream, p);
    } else {
        if (g.out_f32)
            hipLaunchKernelGGL((gemm_kernel<BN, false, true, kDenseRounds>), grid, block, 0, stream, p);
        else
            hipLaunchKernelGGL((gemm_kernel<BN, false, false, kDenseRounds>), grid, block, 0, stream, p);
    }
    return hipGetLastError();
}

// Microscaling dense GEMM (per-row E8M0 scale words on both operands).
template <int BN>
hipError_t dispatch_mx(const GemmProblem& g, int64_t blocks, hipStream_t stream) {
    const Params p = to_params(g);
    const dim3 grid((unsigned)blocks), block(kThreads);
    if (g.out_f32)
        hipLaunchKernelGGL((gemm_kernel<BN, true, true, kDense, true>), grid, block, 0, stream, p);
    else
        hipLaunchKernelGGL((gemm_kernel<BN, true, false, kDense, true>), grid, block, 0, stream, p);
    return hipGetLastError();
}

// Per-tensor scaled dense GEMM (whole-K accumulation in the MFMA).
template <int BN>
hipError_t dispatch_tensor(const GemmProblem& g, int64_t blocks, hipStream_t stream) {
    const Params p = to_params(g);
    const dim3 grid((unsigned)blocks), block(kThreads);
    if (g.out_f32)
        hipLaunchKernelGGL((gemm_kernel<BN, true, true, kDense, false, true>), grid, block, 0, stream, p);
    else
        hipLaunchKernelGGL((gemm_kernel<BN, true, false, kDense, false, true>), grid, block, 0, stream, p);
    return hipGetLastError();
}

// blocks: a multiple of 256 (see grouped_tile). Grouped GEMMs take 128x128
// block scales only.
constexpr int64_t kRecordBytes = kTailRecords * (int64_t)sizeof(TailRecord);
constexpr int64_t kPartBytes = kSplitFloats * (int64_t)sizeof(float);
static_assert(FP8Q_GROUPED_WORKSPACE_BYTES == kRecordBytes + kMaxPieces * kPartBytes,
              "the workspace size in fp8q.h holds every record and partial a call can use");

hipError_t dispatch_grouped(const GemmProblem& g, int64_t blocks, hipStream_t stream) {
    Params p = to_params(g);
    // workspace: the tile records, then as many partial tiles as fit (two at
    // least, or no split)
    const int64_t pieces = g.workspace ? std::min<int64_t>((g.workspace_bytes - kRecordBytes) / kPartBytes, kMaxPieces) : 0;
    if (pieces >= 2) {
        p.split_records = static_cast<TailRecord*>(g.workspace);
        p.split_ws = reinterpret_cast<float*>(static_cast<char*>(g.workspace) + kRecordBytes);
        p.split_pieces = (int32_t)pieces;
    }
    const dim3 grid((unsigned)blocks), block(kThreads);
    if (g.out_f32)
        hipLaunchKernelGGL((gemm_kernel<256, false, true, kGroupedM>), grid, block, 0, stream, p);
    else
        hipLaunchKernelGGL((gemm_kernel<256, false, false, kGroupedM>), grid, block, 0, stream, p);
    if (p.split_ws == nullptr) return hipGetLastError();
    const dim3 fgrid(kFixupBlocks), fblock(kFixupThreads);
    if (g.out_f32)
        hipLaunchKernelGGL((grouped_fixup_kernel<true>), fgrid, fblock, 0, stream, p);
    else
        hipLaunchKernelGGL((grouped_fixup_kernel<false>), fgrid, fblock, 0, stream, p);
    return hipGetLastError();
}

// blocks: a multiple of 256 (see grouped_k_tile). Grouped-over-K GEMMs take
// per-row (128x1) scales on both operands, as Wgrad does.
template <int BN>
hipError_t dispatch_grouped_k(const GemmProblem& g, int64_t blocks, hipStream_t stream) {
    const Params p = to_params(g);
    const dim3 grid((unsigned)blocks), block(kThreads);
    if (g.out_f32)
        hipLaunchKernelGGL((gemm_kernel<BN, true, true, kGroupedK>), grid, block, 0, stream, p);
    else
        hipLaunchKernelGGL((gemm_kernel<BN, true, false, kGroupedK>), grid, block, 0, stream, p);
    return hipGetLastError();
}

// Time of a dense grid in units of one 256-wide tile's work: the number of
// rounds of the 256 CUs times the tile width (all tiles share K and BM).
int64_t grid_cost(int64_t m, int64_t n, int64_t bn) {
    const int64_t tiles = ((m + kBM - 1) / kBM) * ((n + bn - 1) / bn);
    return (tiles + 255) / 256 * bn;
}

}  // namespace

// Several rounds of whole 224-wide tiles, with an even number of slabs: one
// looping block per CU. (Paired on one MI355X, bit-identical output: Dgrad
// 4096 x 7168 x 2048 took 64.2 against 65.4 us, and 8192 x 7168 x 2048 118.9
// against 123.7 us; a 256-wide looping tile, which needs a few more registers
// than the kernel has, gained nothing on 8192 x 4096 x 7168.)
bool use_rounds(const GemmProblem& g) {
    const int64_t tiles = ((g.m + kBM - 1) / kBM) * ((g.n + 223) / 224);
    const int64_t slabs = g.k / kSlab;
    return tiles > 256 && g.m % kBM == 0 && g.n % 224 == 0 && slabs >= 2 && slabs % 2 == 0;
}

hipError_t launch_gemm(const GemmProblem& g, hipStream_t stream) {
    // 224-wide n tiles when the grid then takes less time on the 256 CUs,
    // e.g. N = 7168 = 32 x 224 (Dgrad, Wgrad); otherwise 256-wide.
    if (grid_cost(g.m, g.n, 224) < grid_cost(g.m, g.n, 256)) {
        if (use_rounds(g)) return dispatch_rounds<224>(g, stream);
        const int64_t tiles = ((g.m + kBM - 1) / kBM) * ((g.n + 223) / 224);
        return dispatch_dense<224>(g, (tiles + 7) / 8 * 8, stream);
    }
    const int64_t tiles = ((g.m + kBM - 1) / kBM) * ((g.n + 255) / 256);
    return dispatch_dense<256>(g, (tiles + 7) / 8 * 8, stream);
}

hipError_t launch_grouped_gemm(const GemmProblem& g, hipStream_t stream) {
    // Upper bound on the tile count: every 256-row m-tile of an expert holds at
    // least 128 of its rows, so there are at most m_total / 128 of them.
    const int64_t tiles = (g.m / 128) * ((g.n + 255) / 256);
    return dispatch_grouped(g, (tiles + 255) / 256 * 256, stream);
}

hipError_t launch_grouped_k_gemm(const GemmProblem& g, hipStream_t stream) {
    // Every expert has the same output tiles; 224-wide when that tiles N
    // better (N = 7168), as for a dense GEMM.
    const int bn = grid_cost(g.m, g.n, 224) < grid_cost(g.m, g.n, 256) ? 224 : 256;
    const int64_t per = ((g.m + kBM - 1) / kBM) * ((g.n + bn - 1) / bn);
    const int64_t blocks = (per * g.groups + 255) / 256 * 256;
    return bn == 224 ? dispatch_grouped_k<224>(g, blocks, stream)
                     : dispatch_grouped_k<256>(g, blocks, stream);
}

hipError_t launch_gemm_mx(const GemmProblem& g, hipStream_t stream) {
    if (grid_cost(g.m, g.n, 224) < grid_cost(g.m, g.n, 256)) {
        const int64_t tiles = ((g.m + kBM - 1) / kBM) * ((g.n + 223) / 224);
        return dispatch_mx<224>(g, (tiles + 7) / 8 * 8, stream);
    }
    const int64_t tiles = ((g.m + kBM - 1) / kBM) * ((g.n + 255) / 256);
    return dispatch_mx<256>(g, (tiles + 7) / 8 * 8, stream);
}

hipError_t launch_gemm_tensor(const GemmProblem& g, hipStream_t stream) {
    if (grid_cost(g.m, g.n, 224) < grid_cost(g.m, g.n, 256)) {
        const int64_t tiles = ((g.m + kBM - 1) / kBM) * ((g.n + 223) / 224);
        return dispatch_tensor<224>(g, (tiles + 7) / 8 * 8, stream);
    }
    const int64_t tiles = ((g.m + kBM - 1) / kBM) * ((g.n + 255) / 256);
    return dispatch_tensor<256>(g, (tiles + 7) / 8 * 8, stream);
}

// Scratch of the allocation-free grouped GEMM (fp8_grouped_gemm_noalloc): the
// largest workspace a call uses, one copy on every GPU the library runs on,
// held until the process ends. In host code the array's name is a host-side
// stand-in, not a device address: host code uses only the address that
// hipGetSymbolAddress gives with the device current, kept per device.
__device__ __align__(256) uint8_t scratch[FP8Q_GROUPED_WORKSPACE_BYTES];

constexpr int kMaxScratchDevices = 64;

hipError_t grouped_scratch(void** ptr) {
    static std::mutex mu;
    static void* per_device[kMaxScratchDevices] = {};
    int dev = 0;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) return e;
    if (dev < 0 || dev >= kMaxScratchDevices) return hipErrorInvalidDevice;
    std::lock_guard<std::mutex> lock(mu);
    if (per_device[dev] == nullptr) {
        void* p = nullptr;
        e = hipGetSymbolAddress(&p, HIP_SYMBOL(scratch));
        if (e != hipSuccess) return e;
        per_device[dev] = p;
    }
    *ptr = per_device[dev];
    return hipSuccess;
}

}  // namespace fp8q
