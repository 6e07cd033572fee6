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
#include "mx4/mx4_mfma.h"

#include <type_traits>
#include <utility>

namespace fp8q {
namespace mx4 {
namespace {

typedef int v8i __attribute__((ext_vector_type(8)));

// Lambdas of the kernels: one that is not inlined would put the register
// arrays that it captures into memory.
#define FP8Q_INLINE __attribute__((always_inline))

constexpr int kFp4 = 4;  // the MFMA's operand format code of E2M1

// acc += (B tile) * (A tile)^T; T: which byte of the scale words applies.
template <int T>
__device__ __forceinline__ v4f mfma_tile(v4i b, v4i a, v4f acc, uint32_t sb, uint32_t sa) {
    const v8i bw = __builtin_shufflevector(b, b, 0, 1, 2, 3, 0, 1, 2, 3);
    const v8i aw = __builtin_shufflevector(a, a, 0, 1, 2, 3, 0, 1, 2, 3);
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(bw, aw, acc, kFp4, kFp4, T, (int)sb, T, (int)sa);
}

// Which row of a tile lane l feeds to the MFMA (any order does, as long as
// the outputs are put back in it). ds_read_b128 serves the lanes 0-3, 12-15,
// 20-27 of each half wave together, then the other 16: with lanes i = l % 16 of
// 0-3 and 12-15 on the tile's first eight rows and 4-11 on the last eight,
// both sets touch all 64 banks once (measured: 4 cycles per read; with rows in
// lane order the layout's XOR leaves a two-way conflict, 8 cycles).
__device__ __forceinline__ int lane_row(int i) { return i < 4 ? i : (i < 12 ? i + 4 : i - 8); }

// Where lane l's 16 bytes (row lane_row(l % 16), block l / 16) stand in a
// tile, and its word among the tile's scale words.
__device__ __forceinline__ int lane_code_offset(int lane) {
    const int r = lane_row(lane & 15);
    return r * 64 + ((lane >> 4) ^ (r >> 2)) * 16;
}
__device__ __forceinline__ int lane_scale_word(int lane) { return 4 * lane_row(lane & 15) + (lane >> 4); }
// The m of lane l's results inside a 16 x 16 output tile, and the first of
// its four consecutive n.
__device__ __forceinline__ int lane_m(int lane) { return lane_row(lane & 15); }
__device__ __forceinline__ int lane_n(int lane) { return lane_row(4 * (lane >> 4)); }

// The rows of one output tile: [m0, row_hi) are stored, those from real_end
// on as zeros (padding of an expert's segment).
// (Row and column numbers are 32-bit: the scalar unit has no 64-bit compare,
// and a buffer resource must stay in scalar registers.)
struct Rows {
    int m0, row_hi, real_end;
    int expert;
};

// Expert e's segment [off[e], off[e+1]) is cut into tiles of BM rows; the
// rows past the last segment are one more segment, with no expert and nothing
// real. A tile is of one of three kinds: more than SMALL real rows, some, or
// none (padding). Row tiles of segment e, by kind; a segment has its tiles in
// this order.
struct Segment {
    int beg, end, real, tiles[3];
};
template <int BM, int SMALL>
__device__ __forceinline__ Segment segment(const GemmArgs& p, int e) {
    Segment s = {};
    if (e <= p.groups) {
        s.beg = p.group_offsets[e];
        s.end = e < p.groups ? p.group_offsets[e + 1] : p.m;
        if (e < p.groups) s.real = p.group_rows ? p.group_rows[e] : 0x7FFFFFFF;
    }
    // offsets that break the contract must not move accesses outside A and C:
    // whole row tiles of [0, m)
    s.beg = min(max(s.beg, 0), p.m) & ~15;
    s.end = min(max(s.end, s.beg), p.m);
    s.real = min(max(s.real, 0), s.end - s.beg);
    const int some = (s.real + BM - 1) / BM;
    s.tiles[0] = s.real / BM + (s.real % BM > SMALL ? 1 : 0);
    s.tiles[1] = some - s.tiles[0];
    s.tiles[2] = (s.end - s.beg + BM - 1) / BM - some;
    return s;
}

__device__ __forceinline__ int wave_inclusive_sum(int v) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int u = __shfl_up(v, d);
        if (lane >= d) v += u;
    }
    return v;
}

// Tile `slot` of the grouped order. Inside a kind: expert by expert, inside an
// expert column tile by column tile and then row tile by row tile, so that the
// tiles that share a panel of weights are neighbours. The tiles with few real
// rows come first, then those with many, then the padding: the few-row tiles
// read their weights from HBM for little work, and behind them the others
// start at different times, so that not everybody waits for HBM at once (8192
// rows over 32 experts of uneven sizes, in turn on one card: 177 us; many first
// 188, the two mixed evenly 189). The experts are found by a scan over the
// wave, lane l taking segment base + l. Every lane of the wave must take part.
template <int BM, int SMALL>
__device__ __forceinline__ bool grouped_tile(const GemmArgs& p, int slot, int tiles_n, Rows& t, int& tn) {
    const int lane = threadIdx.x & 63;
    const Segment first64 = segment<BM, SMALL>(p, lane);  // (up to 63 experts: the arrays are read once)
    int kind = 1;
    if constexpr (SMALL > 0) {
        int many = 0, few = 0;
        for (int base = 0; base <= p.groups; base += 64) {
            const Segment s = base == 0 ? first64 : segment<BM, SMALL>(p, base + lane);
            many += __builtin_amdgcn_readlane(wave_inclusive_sum(s.tiles[0]), 63);
            few += __builtin_amdgcn_readlane(wave_inclusive_sum(s.tiles[1]), 63);
        }
        many *= tiles_n;
        few *= tiles_n;
        kind = slot < few ? 1 : (slot < few + many ? 0 : 2);
        slot -= kind == 1 ? 0 : (kind == 0 ? few : few + many);
        kind = __builtin_amdgcn_readfirstlane(kind);
        slot = __builtin_amdgcn_readfirstlane(slot);
    }
    for (int base = 0; base <= p.groups; base += 64) {
        const Segment s = base == 0 ? first64 : segment<BM, SMALL>(p, base + lane);
        const int tiles_m = SMALL == 0   ? s.tiles[0] + s.tiles[1] + s.tiles[2]
                            : kind == 0 ? s.tiles[0]
                            : kind == 1 ? s.tiles[1]
                                        : s.tiles[2];
        const int first = SMALL == 0 || kind == 0 ? 0 : (kind == 1 ? s.tiles[0] : s.tiles[0] + s.tiles[1]);
        const int tiles = tiles_m * tiles_n, incl = wave_inclusive_sum(tiles);
        const int chunk = __builtin_amdgcn_readlane(incl, 63);
        if (slot < chunk) {
            const int l = __builtin_amdgcn_readfirstlane(__ffsll((unsigned long long)__ballot(incl > slot)) - 1);
            const int seg = __builtin_amdgcn_readlane(s.beg, l), seg_end = __builtin_amdgcn_readlane(s.end, l);
            const int seg_tiles = __builtin_amdgcn_readlane(tiles_m, l);
            const int within = slot - __builtin_amdgcn_readlane(incl - tiles, l);
            // (divisions leave the scalar unit)
            tn = __builtin_amdgcn_readfirstlane(within / seg_tiles);
            t.expert = base + l;
            t.m0 = seg + (__builtin_amdgcn_readlane(first, l) + __builtin_amdgcn_readfirstlane(within % seg_tiles)) * BM;
            t.row_hi = min(seg_end, t.m0 + BM);
            t.real_end = seg + __builtin_amdgcn_readlane(s.real, l);
            return true;
        }
        slot -= chunk;
    }
    return false;
}

// Workgroup b runs on XCD b % 8: round r of an XCD's 32 CUs takes the 32
// consecutive slots 256 r + 32 (b % 8) + [0, 32), so that neighbours share an
// L2 and every round is spread evenly over the XCDs. A bijection for grids of
// whole multiples of 256.
__device__ __forceinline__ int round_slot() {
    const int q = (int)(blockIdx.x >> 3);
    return ((q >> 5) << 8) + ((int)(blockIdx.x & 7) << 5) + (q & 31);
}

template <bool F32>
__device__ __forceinline__ void store4(const GemmArgs& p, int m, int n, v4f v) {
    if constexpr (F32) {
        float* const c = static_cast<float*>(p.c) + (int64_t)m * p.ldc + n;
        if (p.c_vec && n + 4 <= p.n) {
            *reinterpret_cast<v4f*>(c) = v;
        } else {
#pragma unroll
            for (int r = 0; r < 4; ++r)
                if (n + r < p.n) c[r] = v[r];
        }
    } else {
        uint16_t* const c = static_cast<uint16_t*>(p.c) + (int64_t)m * p.ldc + n;
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

// Zeros in the padding rows [from, to) of a column tile, 16 bytes per store
// where rows allow it.
template <int BN, bool F32>
__device__ __forceinline__ void zero_rows(const GemmArgs& p, int from, int to, int tn) {
    constexpr int kElems = F32 ? 4 : 8, kPerRow = BN / kElems;
    constexpr int kBytes = F32 ? 4 : 2;
    const int n = tn * BN + (int)threadIdx.x % kPerRow * kElems;
    char* const c = static_cast<char*>(p.c) + (int64_t)n * kBytes;
    for (int m = from + (int)threadIdx.x / kPerRow; m < to; m += (int)blockDim.x / kPerRow) {
        char* const row = c + (int64_t)m * p.ldc * kBytes;
        if (p.c_vec16 && n + kElems <= p.n) {
            *reinterpret_cast<uint4*>(row) = make_uint4(0, 0, 0, 0);
        } else {
            for (int i = 0; i < kElems; ++i) {
                if (n + i >= p.n) break;
                if constexpr (F32) reinterpret_cast<float*>(row)[i] = 0.0f;
                else reinterpret_cast<uint16_t*>(row)[i] = 0;
            }
        }
    }
}

// 16 bytes of weights, read once (non-temporal).
__device__ __forceinline__ v4i load_weights(const uint8_t* p) {
    return __builtin_nontemporal_load(reinterpret_cast<const v4i*>(p));
}

// ------------------------------------------------------------ few rows

// Few rows of A: the weights are streamed from HBM straight to registers. A
// workgroup owns 16 MS x 16 NT outputs; wave w takes the K groups w, w + waves,
// ... : it loads its A tiles of a group once and multiplies them with the
// group's tiles of all NT column tiles, whose loads (4 NT KB per wave) are in
// flight together. The waves' FP32 partials are added in wave order through
// LDS, so the result does not depend on timing.
// Bound by the HBM stream of the weights: 1 x 4096 x 7168: 6.0 us, 2.6 TB/s (each
// of the 14 waves has one K group: a launch, one wait for its loads and the join
// through LDS are most of it); 1 x 16384 x 7168: 13.6 us, 4.6 TB/s.
template <int MS, int NT, bool F32, bool GROUPED>
__global__ __launch_bounds__(64 * max_waves(MS)) void gemm_rows_kernel(GemmArgs p, int tiles_n) {
    extern __shared__ v4f partial[];  // [waves][NT][MS][64]
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
    Rows t;
    int tn;
    if constexpr (GROUPED) {
        if (!grouped_tile<16 * MS, 0>(p, round_slot(), tiles_n, t, tn)) return;
        if (t.m0 >= t.real_end) {
            zero_rows<16 * NT, F32>(p, t.m0, t.row_hi, tn);
            return;
        }
    } else {
        const int tm = blockIdx.x / tiles_n;
        tn = blockIdx.x % tiles_n;
        t = Rows{tm * 16 * MS, min(p.m, (tm + 1) * 16 * MS), p.m, 0};
    }
    v4f acc[NT][MS];
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int s = 0; s < MS; ++s) acc[j][s] = v4f{0.f, 0.f, 0.f, 0.f};

    // row and column tiles past the last one repeat it: loaded, not stored
    int rt[MS], ct[NT];
#pragma unroll
    for (int s = 0; s < MS; ++s) rt[s] = min(t.m0 / 16 + s, (t.real_end - 1) / 16);
#pragma unroll
    for (int j = 0; j < NT; ++j) ct[j] = min(tn * NT + j, (p.n - 1) / 16);
    const uint8_t* const qa = p.a + lane_code_offset(lane);
    const uint32_t* const sa = p.a_scale + lane_scale_word(lane);
    const uint8_t* const qb = p.b + (GROUPED ? t.expert * p.stride_b : 0) + lane_code_offset(lane);
    const uint32_t* const sb = p.b_scale + (GROUPED ? t.expert * p.stride_bs : 0) + lane_scale_word(lane);
    for (int64_t g = wave; g * kGroupTiles < p.kt; g += waves) {
        const int left = p.kt - (int)g * kGroupTiles;  // K tiles from here on
        v4i fb[kGroupTiles][NT], fa[kGroupTiles][MS];
        uint32_t wb[NT], wa[MS];
#pragma unroll
        for (int i = 0; i < kGroupTiles; ++i) {
            // past the last K tile the products are skipped below
            const int64_t kt = g * kGroupTiles + min(i, left - 1);
#pragma unroll
            for (int j = 0; j < NT; ++j) fb[i][j] = load_weights(qb + (kt * p.ld_b + ct[j]) * kTileBytes);
        }
#pragma unroll
        for (int j = 0; j < NT; ++j) wb[j] = sb[(g * p.ld_bs + ct[j]) * kScaleWords];
#pragma unroll
        for (int i = 0; i < kGroupTiles; ++i) {
            const int64_t kt = g * kGroupTiles + min(i, left - 1);
#pragma unroll
            for (int s = 0; s < MS; ++s)
                fa[i][s] = *reinterpret_cast<const v4i*>(qa + (kt * p.ld_a + rt[s]) * kTileBytes);
        }
#pragma unroll
        for (int s = 0; s < MS; ++s) wa[s] = sa[(g * p.ld_as + rt[s]) * kScaleWords];
        auto multiply = [&](auto tile) FP8Q_INLINE {
            constexpr int T = decltype(tile)::value;
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int s = 0; s < MS; ++s) acc[j][s] = mfma_tile<T>(fb[T][j], fa[T][s], acc[j][s], wb[j], wa[s]);
        };
        multiply(std::integral_constant<int, 0>{});
        if (left > 1) multiply(std::integral_constant<int, 1>{});
        if (left > 2) multiply(std::integral_constant<int, 2>{});
        if (left > 3) multiply(std::integral_constant<int, 3>{});
    }
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int s = 0; s < MS; ++s) partial[((wave * NT + j) * MS + s) * 64 + lane] = acc[j][s];
    __syncthreads();
    for (int i = threadIdx.x; i < NT * MS * 64; i += blockDim.x) {
        const int l = i & 63, s = (i >> 6) % MS, j = (i >> 6) / MS;
        const int m = t.m0 + s * 16 + lane_m(l), n = (tn * NT + j) * 16 + lane_n(l);
        if (m >= t.row_hi || n >= p.n) continue;
        v4f v = partial[i];
        for (int w = 1; w < waves; ++w) v += partial[w * NT * MS * 64 + i];
        if (m >= t.real_end) v = v4f{0.f, 0.f, 0.f, 0.f};
        store4<F32>(p, m, n, v);
    }
}

template <int MS, int NT, bool GROUPED>
hipError_t dispatch_rows(const GemmArgs& p, LaunchShape s, hipStream_t stream) {
    const int tiles_n = (p.n + 16 * NT - 1) / (16 * NT);
    const dim3 grid((unsigned)s.blocks), block(s.threads);
    const size_t lds = (size_t)s.threads * NT * MS * sizeof(v4f);
    if (p.out_f32)
        hipLaunchKernelGGL((gemm_rows_kernel<MS, NT, true, GROUPED>), grid, block, lds, stream, p, tiles_n);
    else
        hipLaunchKernelGGL((gemm_rows_kernel<MS, NT, false, GROUPED>), grid, block, lds, stream, p, tiles_n);
    return hipGetLastError();
}

template <bool GROUPED>
hipError_t dispatch_rows(const GemmArgs& p, GemmForm f, LaunchShape s, hipStream_t stream) {
    if (f.ms == 1) {
        if (f.nt == 1) return dispatch_rows<1, 1, GROUPED>(p, s, stream);
        if (f.nt == 2) return dispatch_rows<1, 2, GROUPED>(p, s, stream);
        return dispatch_rows<1, 4, GROUPED>(p, s, stream);
    }
    if (f.ms == 2) {
        if (f.nt == 1) return dispatch_rows<2, 1, GROUPED>(p, s, stream);
        return dispatch_rows<2, 2, GROUPED>(p, s, stream);
    }
    if (f.nt == 1) return dispatch_rows<4, 1, GROUPED>(p, s, stream);
    if (f.nt == 2) return dispatch_rows<4, 2, GROUPED>(p, s, stream);
    return dispatch_rows<4, 4, GROUPED>(p, s, stream);
}

// ------------------------------------------------------------ many rows

// s_waitcnt with vmcnt = N and the other counters left at their maxima
// (lgkmcnt, bits 11:8, at 0: the wave's own LDS reads are done too).
constexpr int waitcnt_vm(int n) { return 0x0070 | (n & 15) | ((n >> 4) << 14); }

// LDS-DMA copy of 1 KB by a wave: 16 bytes from src + voff (lane * 16) + OFF
// to dst + OFF + 16 * lane. src and dst are wave-uniform; the instruction's
// own offset applies to both, so neighbouring copies need no new addresses.
template <int OFF, int POLICY = 0>
__device__ __forceinline__ void copy_1k(const void* src, uint32_t voff, void* dst) {
    asm("" : "+v"(voff));  // (its zero extension is then seen here: scalar base + 32-bit lane offset)
    __builtin_amdgcn_global_load_lds(static_cast<const uint8_t*>(src) + voff, (lds_void*)dst, 16, OFF, POLICY);
}

template <int... Is, class F>
__device__ __forceinline__ void unroll(std::integer_sequence<int, Is...>, F&& f) {
    (f(std::integral_constant<int, Is>{}), ...);
}

// LDS of the tiled kernels: four stages of one K tile (A tiles, then B
// tiles), each an array of its own, so that the compiler can tell a stage being
// filled from the one being read, and one of scale words (64 per row tile,
// rounded up to what the copies fill). TILES: row tiles of A and B together.
constexpr int kStages = 4;

template <int S, int TILES>
__device__ __forceinline__ uint8_t* stage_tiles() {
    __shared__ __attribute__((aligned(1024))) uint8_t tiles[TILES * kTileBytes];
    return tiles;
}
template <int TILES>
__device__ __forceinline__ uint32_t* stage_scales() {
    __shared__ __attribute__((aligned(1024))) uint32_t words[(TILES + 15) / 16 * 16 * kScaleWords];
    return words;
}

// Output tile `slot` of a dense problem: within an XCD (see below) slots walk
// bands of four tile rows, so that the tiles resident together share A and B
// panels in the XCD's L2.
template <int BM, int BN>
__device__ __forceinline__ bool dense_slot(const GemmArgs& p, int slot, int& tm, int& tn) {
    const int tiles_m = (p.m + BM - 1) / BM, tiles_n = (p.n + BN - 1) / BN;
    if (slot >= tiles_m * tiles_n) return false;
    constexpr int G = 4;
    const int band = slot / (G * tiles_n), first = band * G;
    const int gm = min(tiles_m - first, G), within = slot - band * G * tiles_n;
    tm = __builtin_amdgcn_readfirstlane(first + within % gm);  // (divisions leave the scalar unit)
    tn = __builtin_amdgcn_readfirstlane(within / gm);
    return true;
}

// A workgroup of 4 waves (2 x 2) owns 32 TM x 32 TN outputs, a wave 16 TM x
// 16 TN of them: per K tile it reads TM + TN tiles from LDS and issues TM TN
// MFMAs. While the MFMAs of K tile j run from registers, the fragments of j + 1
// are read from LDS, and the copies of j + 2 .. j + 4 are in flight (LDS-DMA,
// 1 KB contiguous per instruction, linear in LDS). One barrier per K tile: it
// says that everybody's copies of tile j + 1 have landed and that everybody
// has read tile j, whose stage the copies of tile j + 4 then overwrite.
// 4096 x 4096 x 7168 with 256 x 256 tiles: 53 to 56 us by card, 4.3 to 4.6
// PFLOP/s; the same MFMAs on random operands with nothing else reach 6.4 to 7.3
// (the clock falls with the load). A K tile's step takes 0.76 us, its MFMAs alone 0.66, its copies alone
// 0.59. 256 x 256 because a step copies 32 KB for its 4096 cycles of MFMA: a tile
// of half the size needs twice the bytes per product from the L2.
// LDS: row tiles that a stage holds (a kernel with tiles of two sizes uses one
// set of stages for both).
template <int TM, int TN, int LDS, bool F32, bool GROUPED>
__device__ __forceinline__ void tile_product(const GemmArgs& p, const Rows& t, int tn) {
    constexpr int BN = 32 * TN;
    constexpr int kATiles = 2 * TM, kBTiles = 2 * TN;
    constexpr int kCopies = (kATiles + kBTiles) / 4;                 // 1 KB copies per wave and K tile
    // 1 KB (4 row tiles) per wave and K group; past the last row tile (24 of
    // them) a copy repeats it into the unused end of the scale stage
    constexpr int kScaleCopies = (kATiles + kBTiles + 15) / 16;
    static_assert(TM <= TN && kCopies <= TN, "the copies and reads of a K tile fit its rows of MFMAs");
    static_assert(kATiles % 4 == 0 && kBTiles % 4 == 0, "every wave makes the same number of copies");
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave >> 1, wn = wave & 1;

    const int n0 = tn * BN;
    const int kt = p.kt;

    v4f acc[TN][TM];
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
        for (int i = 0; i < TM; ++i) acc[j][i] = v4f{0.f, 0.f, 0.f, 0.f};

    if (t.m0 < t.real_end && kt > 0) {
        // Copies: wave w fills tiles [kATiles / 4 * w, + kATiles / 4) of a
        // stage's A part and the same of its B part. At the edge of the matrix
        // (or of an expert's real rows) row tiles past the last one repeat it:
        // loaded, never stored. What differs between the wave's copies is in
        // the lanes' offsets, so a K tile costs one address per operand.
        constexpr int kAW = kATiles / 4, kBW = kBTiles / 4;
        constexpr int kBack = (kAW > kBW ? kAW : kBW) * kTileBytes;  // keeps the offsets positive
        const int a_last = (min(t.real_end, t.row_hi) - 1) / 16 - t.m0 / 16;
        const int b_last = (p.n - 1) / 16 - n0 / 16;
        const uint8_t* ga = p.a + (int64_t)(t.m0 / 16) * kTileBytes - kBack;
        const uint8_t* gb = p.b + (GROUPED ? t.expert * p.stride_b : 0) + (int64_t)(n0 / 16) * kTileBytes - kBack;
        const int64_t step_a = p.ld_a * kTileBytes, step_b = p.ld_b * kTileBytes;
        uint32_t voff[kCopies];
#pragma unroll
        for (int c = 0; c < kCopies; ++c) {
            const int i = c < kAW ? c : c - kAW;
            const int tile = c < kAW ? min(kAW * wave + i, a_last) : min(kBW * wave + i, b_last);
            voff[c] = (tile - i) * kTileBytes + kBack + lane * 16;
        }
        // copy c of the next K tile into `stage`; past the last K tile they
        // repeat it (never used), which keeps the count of copies in flight
        int ahead = 0;
        auto copy_tile = [&](auto stage, auto copy) FP8Q_INLINE {
            constexpr int C = decltype(copy)::value;
            constexpr bool kA = C < kAW;
            uint8_t* const dst = stage_tiles<decltype(stage)::value, LDS>() + (kA ? kAW * wave : kATiles + kBW * wave) * kTileBytes;
            copy_1k<(kA ? C : C - kAW) * kTileBytes, GROUPED && !kA ? 2 : 0>(kA ? ga : gb, voff[C], dst);
        };
        auto next_tile = [&]() FP8Q_INLINE {
            ++ahead;
            ga += ahead < kt ? step_a : 0;
            gb += ahead < kt ? step_b : 0;
        };
        // The scale words of a K group: copy c takes row tiles [4 (4 c + wave),
        // + 4) of the stage, one per 16 lanes, A's first.
        const int kgs = (kt + kGroupTiles - 1) / kGroupTiles;
        int s_ahead = 0;
        const uint32_t* gsa = p.a_scale + (int64_t)(t.m0 / 16) * kScaleWords;
        const uint32_t* gsb = p.b_scale + (GROUPED ? t.expert * p.stride_bs : 0) + (int64_t)(n0 / 16) * kScaleWords;
        uint32_t soff[kScaleCopies];
#pragma unroll
        for (int c = 0; c < kScaleCopies; ++c) {
            const int i = 4 * (4 * c + wave) + (lane >> 4);
            soff[c] = (i < kATiles ? min(i, a_last) : min(i - kATiles, b_last)) * 4 * kScaleWords + (lane & 15) * 16;
        }
        auto copy_scales = [&]() FP8Q_INLINE {
#pragma unroll
            for (int c = 0; c < kScaleCopies; ++c) {
                const int i = 4 * (4 * c + wave);
                copy_1k<0>(i < kATiles ? gsa : gsb, soff[c], stage_scales<LDS>() + i * kScaleWords);
            }
            ++s_ahead;
            gsa += s_ahead < kgs ? p.ld_as * kScaleWords : 0;
            gsb += s_ahead < kgs ? p.ld_bs * kScaleWords : 0;
        };
        const int frag = lane_code_offset(lane), sword = lane_scale_word(lane);
        auto read_a = [&](auto stage, int i) FP8Q_INLINE {
            return *reinterpret_cast<const v4i*>(stage_tiles<decltype(stage)::value, LDS>() + (wm * TM + i) * kTileBytes + frag);
        };
        auto read_b = [&](auto stage, int i) FP8Q_INLINE {
            return *reinterpret_cast<const v4i*>(stage_tiles<decltype(stage)::value, LDS>() +
                                                 (kATiles + wn * TN + i) * kTileBytes + frag);
        };
        v4i fa[2][TM], fb[2][TN];
        uint32_t sa[2][TM], sb[2][TN];  // this K group's scale words, the next one's
        // The next K tile, j: its MFMAs from register set P % 2; fragments of
        // j + 1 into the other; copies of j + 4. P = j mod 4 fixes stages and
        // registers. A wave has its SIMD to itself, so whatever it issues
        // between two MFMAs beyond the 16 cycles of the first leaves the matrix
        // unit idle: reads and copies go one at a time between MFMAs.
        auto step = [&](auto pos) FP8Q_INLINE {
            constexpr int P = decltype(pos)::value;
            using Next = std::integral_constant<int, (P + 1) % kStages>;
            // batches of the two youngest K tiles may still be in flight
            constexpr int kFlying = 2 * kCopies + (P == 1 || P == 2 ? kScaleCopies : 0);
            __builtin_amdgcn_sched_barrier(0);
            __builtin_amdgcn_s_waitcnt(waitcnt_vm(kFlying));
            __builtin_amdgcn_s_barrier();
            __builtin_amdgcn_sched_barrier(0);
            // the next group's scale words: copied in step 0, read in step 3
            const uint32_t* const s = stage_scales<LDS>() + sword;
            unroll(std::make_integer_sequence<int, TN * TM>{}, [&](auto at) FP8Q_INLINE {
                constexpr int N = decltype(at)::value / TM, M = decltype(at)::value % TM;
                mfma_in_place<P>(acc[N][M], fb[P % 2][N], fa[P % 2][M], sb[0][N], sa[0][M]);
                if constexpr (M == 0) fb[(P + 1) % 2][N] = read_b(Next{}, N);
                if constexpr (M == TM / 4 && N < TM) fa[(P + 1) % 2][N] = read_a(Next{}, N);
                if constexpr (M == TM / 2 && N == 0 && P == 0) copy_scales();
                if constexpr (M == 3 * TM / 4 && N < kCopies) copy_tile(pos, std::integral_constant<int, N>{});
                if constexpr (M == TM - 1 && N == TN - 1) next_tile();
                if constexpr (P == 3 && M == TM - 1) {
                    if constexpr (N < TM) sa[1][N] = s[(wm * TM + N) * kScaleWords];
                    sb[1][N] = s[(kATiles + wn * TN + N) * kScaleWords];
                }
                __builtin_amdgcn_sched_barrier(0);
            });
            if constexpr (P == 3) {
#pragma unroll
                for (int i = 0; i < TM; ++i) sa[0][i] = sa[1][i];
#pragma unroll
                for (int i = 0; i < TN; ++i) sb[0][i] = sb[1][i];
            }
        };
        copy_scales();
        unroll(std::make_integer_sequence<int, kStages>{}, [&](auto stage) FP8Q_INLINE {
            unroll(std::make_integer_sequence<int, kCopies>{}, [&](auto c) FP8Q_INLINE { copy_tile(stage, c); });
            next_tile();
        });
        __builtin_amdgcn_s_waitcnt(waitcnt_vm(3 * kCopies));
        __builtin_amdgcn_s_barrier();
#pragma unroll
        for (int i = 0; i < TM; ++i) {
            sa[0][i] = stage_scales<LDS>()[sword + (wm * TM + i) * kScaleWords];
            fa[0][i] = read_a(std::integral_constant<int, 0>{}, i);
        }
#pragma unroll
        for (int i = 0; i < TN; ++i) {
            sb[0][i] = stage_scales<LDS>()[sword + (kATiles + wn * TN + i) * kScaleWords];
            fb[0][i] = read_b(std::integral_constant<int, 0>{}, i);
        }
        int j = 0;
        for (; j + 4 <= kt; j += 4)
            unroll(std::make_integer_sequence<int, 4>{}, [&](auto pos) FP8Q_INLINE { step(pos); });
        const int rest = kt - j;
        if (rest > 0) step(std::integral_constant<int, 0>{});
        if (rest > 1) step(std::integral_constant<int, 1>{});
        if (rest > 2) step(std::integral_constant<int, 2>{});
        // the last copies land before the LDS is used again, here or by
        // another workgroup
        __builtin_amdgcn_s_waitcnt(waitcnt_vm(0));
        mfma_settle(acc);
        __builtin_amdgcn_s_barrier();
    }

    // bf16 rows that need no edge guards go through the wave's own piece of
    // LDS, 16 rows at a time, and leave as whole runs of 32 TN bytes; straight
    // from the accumulators a store would write 32-byte pieces of 16 rows.
    if constexpr (!F32) {
        if (p.c_vec16 && n0 + BN <= p.n) {
            constexpr int kRow = 32 * TN + 16;  // bytes of a staged row, padded against bank conflicts
            static_assert(4 * 16 * kRow <= LDS * kTileBytes, "the four waves' rows fit a stage");
            constexpr int kLanes = 2 * TN;      // lanes per row when it is read back, 16 bytes each
            unroll(std::make_integer_sequence<int, TM>{}, [&](auto at) FP8Q_INLINE {
                constexpr int I = decltype(at)::value;
                uint8_t* const rows = stage_tiles<I % 2, LDS>() + wave * 16 * kRow;
                const int m16 = t.m0 + (wm * TM + I) * 16;
                if (m16 >= t.row_hi) return;
                const bool pad = m16 + lane_m(lane) >= t.real_end;
#pragma unroll
                for (int j = 0; j < TN; ++j) {
                    const v4f v = pad ? v4f{0.f, 0.f, 0.f, 0.f} : acc[j][I];
                    *reinterpret_cast<uint2*>(rows + lane_m(lane) * kRow + (j * 16 + lane_n(lane)) * 2) =
                        make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
                }
                __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
                __builtin_amdgcn_wave_barrier();
#pragma unroll
                for (int q = 0; q < 16 * kLanes / 64; ++q) {
                    const int r = q * (64 / kLanes) + lane / kLanes, at16 = lane % kLanes;
                    const uint4 v = *reinterpret_cast<const uint4*>(rows + r * kRow + at16 * 16);
                    if (m16 + r < t.row_hi)
                        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.c) + (int64_t)(m16 + r) * p.ldc + n0 +
                                                  wn * 16 * TN + at16 * 8) = v;
                }
            });
            return;
        }
    }
#pragma unroll
    for (int i = 0; i < TM; ++i) {
        const int m = t.m0 + (wm * TM + i) * 16 + lane_m(lane);
        if (m >= t.row_hi) continue;
        const bool pad = m >= t.real_end;
#pragma unroll
        for (int j = 0; j < TN; ++j) {
            const int n = n0 + (wn * TN + j) * 16 + lane_n(lane);
            if (n < p.n) store4<F32>(p, m, n, pad ? v4f{0.f, 0.f, 0.f, 0.f} : acc[j][i]);
        }
    }
}

template <int TM, int TN, bool F32>
__global__ __launch_bounds__(256, TM * TN > 16 ? 1 : 2) void gemm_tiles_kernel(GemmArgs p) {
    constexpr int BM = 32 * TM, BN = 32 * TN;
    // Workgroup b runs on XCD b % 8, which takes one run of slots.
    const int slot = (int)((blockIdx.x % 8) * (gridDim.x / 8) + blockIdx.x / 8);
    int tm, tn;
    if (!dense_slot<BM, BN>(p, slot, tm, tn)) return;
    tile_product<TM, TN, 2 * (TM + TN), F32, false>(p, Rows{tm * BM, min(p.m, (tm + 1) * BM), p.m, 0}, tn);
}

// Tiles of 256 x 256, or half as high where no more than 128 rows are real
// (an expert's last rows, or all of a small one's): that takes about 0.6 of
// the time. 8192 rows over 32 experts of 4096 x 7168, uneven: 163 to 181 us by
// card, of which HBM traffic (the weights once, A, C and its padding: 752 MB)
// takes 145 at the rate of a large copy; 64 routes over 32 experts of 2048 x 4096,
// 27 to 30 of which have rows: 25.6 us, 5.2 TB/s (134 MB moved with 29).
template <bool F32>
__global__ __launch_bounds__(256, 1) void grouped_tiles_kernel(GemmArgs p) {
    constexpr int BM = 256, BN = 256;
    Rows t;
    int tn;
    if (!grouped_tile<BM, BM / 2>(p, round_slot(), (p.n + BN - 1) / BN, t, tn)) return;
    const int real = t.real_end - t.m0;
    if (real > BM / 2) {
        tile_product<8, 8, 32, F32, true>(p, t, tn);
    } else {
        const int half = min(t.row_hi, t.m0 + BM / 2);
        if (real > 0) tile_product<4, 8, 32, F32, true>(p, Rows{t.m0, half, t.real_end, t.expert}, tn);
        zero_rows<BN, F32>(p, real > 0 ? half : t.m0, t.row_hi, tn);
    }
}

template <int TM, int TN>
hipError_t dispatch_tiles(const GemmArgs& p, LaunchShape s, hipStream_t stream) {
    const dim3 grid((unsigned)s.blocks), block(s.threads);
    if (p.out_f32)
        hipLaunchKernelGGL((gemm_tiles_kernel<TM, TN, true>), grid, block, 0, stream, p);
    else
        hipLaunchKernelGGL((gemm_tiles_kernel<TM, TN, false>), grid, block, 0, stream, p);
    return hipGetLastError();
}

hipError_t dispatch_grouped_tiles(const GemmArgs& p, LaunchShape s, hipStream_t stream) {
    const dim3 grid((unsigned)s.blocks), block(s.threads);
    if (p.out_f32)
        hipLaunchKernelGGL((grouped_tiles_kernel<true>), grid, block, 0, stream, p);
    else
        hipLaunchKernelGGL((grouped_tiles_kernel<false>), grid, block, 0, stream, p);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_gemm(const GemmArgs& p, hipStream_t stream) {
    const GemmForm f = gemm_form(p.m, p.n, p.scales16);
    const LaunchShape s = gemm_shape(f, p.m, p.n, p.kt);
    if (f.kernel == GemmKernel::kRows) return dispatch_rows<false>(p, f, s, stream);
    return f.ms == 8 ? dispatch_tiles<8, 8>(p, s, stream) : dispatch_tiles<4, 4>(p, s, stream);
}

hipError_t launch_grouped_gemm(const GemmArgs& p, hipStream_t stream) {
    const GemmForm f = grouped_form(p.m, p.n, p.groups, p.scales16);
    const LaunchShape s = grouped_shape(f, p.m, p.n, p.kt, p.groups);
    return f.kernel == GemmKernel::kRows ? dispatch_rows<true>(p, f, s, stream) : dispatch_grouped_tiles(p, s, stream);
}

}  // namespace mx4
}  // namespace fp8q
