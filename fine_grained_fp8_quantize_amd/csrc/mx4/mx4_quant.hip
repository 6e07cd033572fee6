// mx4_quant.hip -- FP4 microscaling quantization and read-back for gfx950.
//
// For every 32 consecutive elements along K: amax = max |x|,
// e = clamp(floor(log2 amax) - 2, -127, 127) (2: exponent of E2M1's largest
// value, 6 = 1.5 * 2^2), code = E2M1(x / 2^e) to nearest, ties to the even
// code, saturating to +-6. With bf16 input the biased exponent byte is
// max(E - 2, 0) for amax's exponent field E (a zero, subnormal or smallest
// normal amax clamps to byte 0 = 2^-127), and x / 2^e is exact, so the
// hardware conversion v_cvt_scalef32_pk_fp4_bf16 is the definition itself
// (checked on gfx950 for every bf16 value at every scale, both signs). A
// block with an infinity or NaN gets exponent byte 255 and zero codes: it
// reads back as NaN, and products with it are NaN.
//
// All four kernels are bound by HBM: 2 bytes read and 0.53 written per
// element when quantizing, the reverse for the read-back. The tile layout
// (mx4.h) is built in LDS, so that the global accesses on both sides are
// whole lines.
#include "mx4/mx4.h"

#include "fp8q_device.h"

namespace fp8q {
namespace mx4 {
namespace {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

// Wave-private LDS staging: the wave's own stores before its own loads.
__device__ __forceinline__ void wave_lds_fence() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// E8M0 byte of a block whose largest magnitude has these bf16 bits.
__device__ __forceinline__ uint32_t block_byte(uint32_t amax_bits) {
    const uint32_t ex = amax_bits >> 7;
    return ex == 255u ? 255u : (ex > 2u ? ex - 2u : 0u);
}

// 2^(byte - 127) as a float (2^-127 is subnormal).
__device__ __forceinline__ float block_scale(uint32_t byte) {
    return __uint_as_float(byte == 0u ? 0x00400000u : byte << 23);
}

// Eight bf16 (four words, two each) -> eight E2M1 codes, element 0 in the
// low nibble.
__device__ __forceinline__ uint32_t pack_e2m1x8(uint32_t w0, uint32_t w1, uint32_t w2, uint32_t w3, float scale) {
    uint32_t c = 0;
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2, w0), scale, 0);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2, w1), scale, 1);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2, w2), scale, 2);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2, w3), scale, 3);
    return c;
}

// Eight consecutive bf16 from element `at` on of up to N rows (`have` of them
// exist), zeros past `end`. Whether a lane reads 16 bytes, single elements or
// nothing is decided once for all rows: inside each row's load the branch would
// wait for the row before (8192 x 2040, whose last lanes read nothing: 17.0
// against 10.2 us).
template <bool VEC, int N>
__device__ __forceinline__ void load_rows(uint4 (&v)[N], const uint16_t* first, int64_t ld, int64_t have, int64_t at,
                                          int64_t end) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = make_uint4(0, 0, 0, 0);
    if (VEC && at + 8 <= end) {
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (i < have) v[i] = load_nt16(first + i * ld + at);
    } else if (at < end) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if (i >= have) continue;
            uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (at + k < end) w[k >> 1] |= (uint32_t)first[i * ld + at + k] << (16 * (k & 1));
            v[i] = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
}

// Codes and exponent byte of one lane's eight elements; the block's amax is
// taken over the quad of lanes that holds it.
__device__ __forceinline__ uint32_t quant_quad(uint4 v, uint32_t& byte) {
    const uint32_t mask = 0x7FFF7FFFu;
    const uint32_t m = pk_max_u16(pk_max_u16(v.x & mask, v.y & mask), pk_max_u16(v.z & mask, v.w & mask));
    byte = block_byte(quad_max(umax32(m & 0xFFFFu, m >> 16)));
    const uint32_t c = pack_e2m1x8(v.x, v.y, v.z, v.w, block_scale(byte));
    return byte == 255u ? 0u : c;
}

__device__ __forceinline__ void store_nt16(void* p, uint4 v) {
    typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
    __builtin_nontemporal_store(u32x4{v.x, v.y, v.z, v.w}, reinterpret_cast<u32x4*>(p));
}

constexpr int kMaxTopk = 8;
// One wave's staging: four tiles, 16 words apart so that the four tiles'
// equal places fall into different banks.
constexpr int kStageTile = kTileBytes / 4 + 16;

// A wave quantizes 16 rows x 512 k (one K group of one row tile): lane l
// holds elements [8 l, 8 l + 8) of each row, so a load instruction reads 1 KB
// of one row; 16 loads are in flight per wave. 4096 x 7168: 15.4 us, 4.8 TB/s
// read and written; 8192 x 2040: 10.2 us, 4.2 TB/s.
template <bool VEC>
__global__ __launch_bounds__(64 * kQuantWaves) void quant_rows_kernel(QuantArgs p, int64_t rt, int64_t kg, int64_t units) {
    __shared__ __attribute__((aligned(16))) uint32_t codes[kQuantWaves][kGroupTiles * kStageTile];
    __shared__ __attribute__((aligned(16))) uint8_t bytes[kQuantWaves][kScaleWords * 4];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t unit = (int64_t)blockIdx.x * kQuantWaves + wave;
    if (unit >= units) return;  // whole wave; no workgroup barrier below
    const int64_t g = unit % kg, tile = unit / kg % rt, e = unit / kg / rt;
    const uint16_t* const x = p.x + e * p.stride_x;
    const int t = lane >> 4, b = (lane >> 2) & 3;

    uint4 v[kTileRows];
    load_rows<VEC>(v, x + tile * kTileRows * p.ld_x, p.ld_x, p.rows - tile * kTileRows, g * kGroupK + 8 * lane, p.cols);
#pragma unroll
    for (int r = 0; r < kTileRows; ++r) {
        uint32_t byte;
        const uint32_t c = quant_quad(v[r], byte);
        codes[wave][t * kStageTile + r * 16 + (b ^ ((r >> 2) & 3)) * 4 + (lane & 3)] = c;
        if ((lane & 3) == 0) bytes[wave][(4 * r + b) * 4 + t] = (uint8_t)byte;
    }
    wave_lds_fence();
    const int64_t kts = (p.cols + kTileK - 1) / kTileK;
#pragma unroll
    for (int i = 0; i < kGroupTiles; ++i) {
        const int64_t kt = g * kGroupTiles + i;
        if (kt < kts)
            store_nt16(p.q + e * p.stride_q + (kt * p.ld_q + tile) * kTileBytes + lane * 16,
                       *reinterpret_cast<const uint4*>(&codes[wave][i * kStageTile + lane * 4]));
    }
    p.scale[e * p.stride_s + (g * p.ld_s + tile) * kScaleWords + lane] =
        reinterpret_cast<const uint32_t*>(bytes[wave])[lane];
}

// Max over each quad of lanes of both 16-bit halves.
__device__ __forceinline__ uint32_t quad_max_u16x2(uint32_t v) {
    v = pk_max_u16(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xF, 0xF, false));
    v = pk_max_u16(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xF, 0xF, false));
    return v;
}

// The transposed operand: blocks of 32 consecutive rows of x, one matrix row
// per column of x. A workgroup takes 256 rows (tokens: two K tiles, half a
// group) x 128 columns (channels); wave w takes 32 tokens (block w % 4 of K tile
// w / 4), lane l tokens [8 (l % 4), +8) and channels [8 (l / 4), +8): a load
// instruction reads 256 bytes of each of 4 tokens, and a block's amax is a quad
// maximum. (64 channels, 128 bytes of 8 tokens: a tenth slower where rows do
// not start on 128-byte lines, as each piece then touches two.) 4096 x 7168: 17.0
// us, 4.4 TB/s; 8192 x 2040: 11.2 us, 3.8 TB/s.
// LDS words of a tile and of its upper eight rows: the 16 (tile, half) pairs
// that one store instruction touches start 4 banks apart.
constexpr int kColsTile = kTileBytes / 4 + 8;
constexpr int kColsHalf = kTileBytes / 8 + 4;

template <bool VEC>
__global__ __launch_bounds__(kColsThreads) void quant_cols_kernel(QuantArgs p, int64_t ct, int64_t halves, int64_t units) {
    constexpr int kTiles = kColsChannels / kTileRows;
    __shared__ __attribute__((aligned(16))) uint32_t codes[kColsKTiles * kTiles * kColsTile];
    __shared__ __attribute__((aligned(16))) uint8_t bytes[kTiles * kScaleWords * kColsKTiles];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    // Workgroup b runs on XCD b % 8. Where rows do not start on 128-byte lines,
    // neighbours share lines, and every XCD takes one run of units (8192 x 2040:
    // 11.0 against 12.7 us, 4096 x 7160: 17.9 against 20.1); where they do, the
    // plain order spreads the reads better (8192 x 2048: 11.7 against 12.2).
    const int64_t unit = p.ld_x % 64 != 0 ? (int64_t)(blockIdx.x % 8) * (gridDim.x / 8) + blockIdx.x / 8 : blockIdx.x;
    if (unit >= units) return;
    const int64_t c = unit % ct, hf = unit / ct % halves, e = unit / ct / halves;
    const int64_t kt0 = hf * kColsKTiles;  // first K tile
    const uint16_t* const x = p.x + e * p.stride_x;
    const int t = wave >> 2, b = wave & 3, j = lane & 3, chunk = lane >> 2;
    const int64_t col = c * kColsChannels + 8 * chunk;
    const int64_t tok = kt0 * kTileK + wave * 32 + 8 * j;

    uint4 v[8];
    load_rows<VEC>(v, x + tok * p.ld_x, p.ld_x, p.rows - tok, col, p.cols);
#pragma unroll
    for (int w = 0; w < 4; ++w) {  // word w: channels 2w and 2w + 1
        uint32_t u[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) u[i] = w == 0 ? v[i].x : w == 1 ? v[i].y : w == 2 ? v[i].z : v[i].w;
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = pk_max_u16(m, u[i] & 0x7FFF7FFFu);
        m = quad_max_u16x2(m);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t byte = block_byte(h == 0 ? m & 0xFFFFu : m >> 16);
            const uint32_t sel = h == 0 ? 0x05040100u : 0x07060302u;  // the low or high half of two tokens
            uint32_t code = pack_e2m1x8(__builtin_amdgcn_perm(u[1], u[0], sel), __builtin_amdgcn_perm(u[3], u[2], sel),
                                        __builtin_amdgcn_perm(u[5], u[4], sel), __builtin_amdgcn_perm(u[7], u[6], sel),
                                        block_scale(byte));
            if (byte == 255u) code = 0;
            const int ch = 8 * chunk + 2 * w + h, r = ch & 15;
            codes[(t * kTiles + (ch >> 4)) * kColsTile + (r >> 3) * kColsHalf + (r & 7) * 16 +
                  (b ^ ((r >> 2) & 3)) * 4 + j] = code;
            if (j == w) bytes[((ch >> 4) * kScaleWords + 4 * r + b) * kColsKTiles + t] = (uint8_t)byte;
        }
    }
    __syncthreads();
    const int64_t kts = (p.rows + kTileK - 1) / kTileK, rts = (p.cols + kTileRows - 1) / kTileRows;
#pragma unroll
    for (int i = 0; i < kColsKTiles * kTiles / (kColsThreads / 64); ++i) {
        const int at = i * (kColsThreads / 64) + wave;  // K tile at / kTiles, row tile at % kTiles
        const int64_t kt = kt0 + at / kTiles, rt = c * kTiles + at % kTiles;
        if (kt < kts && rt < rts)
            *reinterpret_cast<uint4*>(p.q + e * p.stride_q + (kt * p.ld_q + rt) * kTileBytes + lane * 16) =
                *reinterpret_cast<const uint4*>(&codes[at * kColsTile + (lane >> 5) * kColsHalf + (lane & 31) * 4]);
    }
    // two of the four bytes of each scale word
    static_assert(kTiles == kColsThreads / 64, "one row tile per wave");
    if (c * kTiles + wave < rts)
        reinterpret_cast<uint16_t*>(p.scale + e * p.stride_s +
                                    (hf / 2 * p.ld_s + c * kTiles + wave) * kScaleWords + lane)[hf & 1] =
            reinterpret_cast<const uint16_t*>(bytes)[wave * kScaleWords + lane];
}

// Quantize each token once and store its codes to every row its routes name.
// A wave takes 16 tokens x 512 k as quant_rows_kernel does; a row's share of a
// tile is 64 contiguous bytes, so a store instruction writes 4 tokens x 4 K
// tiles x 64 bytes, and one store of scale words serves 16 tokens. 8192 tokens x
// 7168, 8192 routes: 34.4 us, 4.4 TB/s.
template <bool VEC>
__global__ __launch_bounds__(64 * kQuantWaves) void quant_scatter_kernel(ScatterArgs p, int64_t kg, int64_t units) {
    __shared__ __attribute__((aligned(16))) uint32_t codes[kQuantWaves][kGroupTiles * kStageTile];
    __shared__ __attribute__((aligned(16))) uint8_t bytes[kQuantWaves][kScaleWords * 4];
    __shared__ int32_t routes[kQuantWaves][kTileRows * kMaxTopk];  // of the wave's 16 tokens, -1 for none
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t unit = (int64_t)blockIdx.x * kQuantWaves + wave;
    if (unit >= units) return;  // whole wave; no workgroup barrier below
    const int64_t g = unit % kg, first = unit / kg * kTileRows;
    const int t = lane >> 4, b = (lane >> 2) & 3;
#pragma unroll
    for (int i = 0; i < kTileRows * kMaxTopk / 64; ++i) {
        const int at = i * 64 + lane;
        int64_t dst = -1;
        if (at < kTileRows * p.topk && first * p.topk + at < p.tokens * p.topk) dst = p.dst[first * p.topk + at];
        routes[wave][at] = dst < 0 || dst >= p.m_total ? -1 : (int32_t)dst;
    }

    uint4 v[kTileRows];
    load_rows<VEC>(v, p.x + first * p.ld_x, p.ld_x, p.tokens - first, g * kGroupK + 8 * lane, p.cols);
#pragma unroll
    for (int r = 0; r < kTileRows; ++r) {
        uint32_t byte;
        const uint32_t c = quant_quad(v[r], byte);
        codes[wave][t * kStageTile + r * 16 + b * 4 + (lane & 3)] = c;
        if ((lane & 3) == 0) bytes[wave][(4 * r + b) * 4 + t] = (uint8_t)byte;
    }
    wave_lds_fence();
    const int64_t kts = (p.cols + kTileK - 1) / kTileK;
    // lane: token 4 i + l / 16, K tile (l / 4) % 4, block l % 4
    const int kt_rel = (lane >> 2) & 3, blk = lane & 3;
    const int64_t kt = g * kGroupTiles + kt_rel;
    uint4 w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        w[i] = *reinterpret_cast<const uint4*>(&codes[wave][kt_rel * kStageTile + (4 * i + (lane >> 4)) * 16 + blk * 4]);
    const uint32_t word = reinterpret_cast<const uint32_t*>(bytes[wave])[lane];
    for (int k = 0; k < p.topk; ++k) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int dst = routes[wave][(4 * i + (lane >> 4)) * p.topk + k];
            if (dst < 0 || kt >= kts) continue;
            const int r = dst & 15;
            *reinterpret_cast<uint4*>(p.q + (kt * p.ld_q + (dst >> 4)) * kTileBytes + r * 64 +
                                      (blk ^ ((r >> 2) & 3)) * 16) = w[i];
        }
        const int dst = routes[wave][(lane >> 2) * p.topk + k];
        if (dst >= 0) p.scale[(g * p.ld_s + (dst >> 4)) * kScaleWords + (dst & 15) * 4 + (lane & 3)] = word;
    }
}

// Codes back to values: a wave reads the four tiles of a K group (1 KB loads)
// and writes 16 rows of 512 elements, 1 KB (bf16) or 2 KB (fp32) per row. 4096 x
// 7168 to bf16: 13.3 us, 5.6 TB/s.
template <bool F32, bool VEC>
__global__ __launch_bounds__(64 * kQuantWaves) void dequant_kernel(DequantArgs p, int64_t kg, int64_t units) {
    __shared__ __attribute__((aligned(16))) uint32_t codes[kQuantWaves][kGroupTiles * kStageTile];
    __shared__ __attribute__((aligned(16))) uint8_t bytes[kQuantWaves][kScaleWords * 4];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t unit = (int64_t)blockIdx.x * kQuantWaves + wave;
    if (unit >= units) return;  // whole wave; no workgroup barrier below
    const int64_t g = unit % kg, tile = unit / kg;
    const int64_t kts = (p.cols + kTileK - 1) / kTileK;
#pragma unroll
    for (int i = 0; i < kGroupTiles; ++i) {
        const int64_t kt = g * kGroupTiles + i;
        if (kt < kts)
            *reinterpret_cast<uint4*>(&codes[wave][i * kStageTile + lane * 4]) =
                load_nt16(p.q + (kt * p.ld_q + tile) * kTileBytes + lane * 16);
    }
    reinterpret_cast<uint32_t*>(bytes[wave])[lane] = p.scale[(g * p.ld_s + tile) * kScaleWords + lane];
    wave_lds_fence();
    const int t = lane >> 4, b = (lane >> 2) & 3;
    const int64_t k = g * kGroupK + 8 * lane;
    if (k >= p.cols) return;
#pragma unroll
    for (int r = 0; r < kTileRows; ++r) {
        const int64_t row = tile * kTileRows + r;
        if (row >= p.rows) continue;
        const uint32_t c = codes[wave][t * kStageTile + r * 16 + (b ^ ((r >> 2) & 3)) * 4 + (lane & 3)];
        const uint32_t byte = bytes[wave][(4 * r + b) * 4 + t];
        const float s = block_scale(byte);
        uint32_t w[4];
        w[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 0));
        w[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 1));
        w[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 2));
        w[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 3));
        if constexpr (F32) {
            float* const y = static_cast<float*>(p.y) + row * p.ld_y + k;
            const float f[8] = {bf16_lo(w[0]), bf16_hi(w[0]), bf16_lo(w[1]), bf16_hi(w[1]),
                                bf16_lo(w[2]), bf16_hi(w[2]), bf16_lo(w[3]), bf16_hi(w[3])};
            if (VEC && k + 8 <= p.cols) {
                reinterpret_cast<float4*>(y)[0] = make_float4(f[0], f[1], f[2], f[3]);
                reinterpret_cast<float4*>(y)[1] = make_float4(f[4], f[5], f[6], f[7]);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (k + i < p.cols) y[i] = f[i];
            }
        } else {
            uint16_t* const y = static_cast<uint16_t*>(p.y) + row * p.ld_y + k;
            if (VEC && k + 8 <= p.cols) {
                *reinterpret_cast<uint4*>(y) = make_uint4(w[0], w[1], w[2], w[3]);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (k + i < p.cols) y[i] = (uint16_t)(w[i >> 1] >> (16 * (i & 1)));
            }
        }
    }
}

}  // namespace

hipError_t launch_quant_rows(const QuantArgs& p, hipStream_t stream) {
    const int64_t rt = ceil_div(p.rows, kTileRows), kg = ceil_div(p.cols, kGroupK);
    const int64_t units = quant_rows_units(p.groups, p.rows, p.cols);
    const LaunchShape s = quant_rows_shape(p.groups, p.rows, p.cols);
    const dim3 grid((unsigned)s.blocks), block(s.threads);
    if (p.vec)
        hipLaunchKernelGGL((quant_rows_kernel<true>), grid, block, 0, stream, p, rt, kg, units);
    else
        hipLaunchKernelGGL((quant_rows_kernel<false>), grid, block, 0, stream, p, rt, kg, units);
    return hipGetLastError();
}

hipError_t launch_quant_cols(const QuantArgs& p, hipStream_t stream) {
    const int64_t ct = ceil_div(p.cols, kColsChannels), halves = quant_cols_halves(p.rows);
    const int64_t units = quant_cols_units(p.groups, p.rows, p.cols);
    const LaunchShape s = quant_cols_shape(p.groups, p.rows, p.cols);
    const dim3 grid((unsigned)s.blocks), block(s.threads);
    if (p.vec)
        hipLaunchKernelGGL((quant_cols_kernel<true>), grid, block, 0, stream, p, ct, halves, units);
    else
        hipLaunchKernelGGL((quant_cols_kernel<false>), grid, block, 0, stream, p, ct, halves, units);
    return hipGetLastError();
}

hipError_t launch_quant_scatter(const ScatterArgs& p, hipStream_t stream) {
    const int64_t kg = ceil_div(p.cols, kGroupK), units = quant_rows_units(1, p.tokens, p.cols);
    const LaunchShape s = quant_rows_shape(1, p.tokens, p.cols);
    const dim3 grid((unsigned)s.blocks), block(s.threads);
    if (p.vec)
        hipLaunchKernelGGL((quant_scatter_kernel<true>), grid, block, 0, stream, p, kg, units);
    else
        hipLaunchKernelGGL((quant_scatter_kernel<false>), grid, block, 0, stream, p, kg, units);
    return hipGetLastError();
}

hipError_t launch_dequant(const DequantArgs& p, hipStream_t stream) {
    const int64_t kg = ceil_div(p.cols, kGroupK), units = quant_rows_units(1, p.rows, p.cols);
    const LaunchShape s = quant_rows_shape(1, p.rows, p.cols);
    const dim3 grid((unsigned)s.blocks), block(s.threads);
    if (p.f32) {
        if (p.vec)
            hipLaunchKernelGGL((dequant_kernel<true, true>), grid, block, 0, stream, p, kg, units);
        else
            hipLaunchKernelGGL((dequant_kernel<true, false>), grid, block, 0, stream, p, kg, units);
    } else {
        if (p.vec)
            hipLaunchKernelGGL((dequant_kernel<false, true>), grid, block, 0, stream, p, kg, units);
        else
            hipLaunchKernelGGL((dequant_kernel<false, false>), grid, block, 0, stream, p, kg, units);
    }
    return hipGetLastError();
}

}  // namespace mx4
}  // namespace fp8q
