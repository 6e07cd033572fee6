// mx4.h -- the FP4 microscaling (MXFP4) kernels of libfp8q: tile layout and
// host-side launchers (internal; arguments are already validated by
// mx4_api.cpp).
//
// An FP4 matrix [rows][k] is held in tiles of 16 rows x 128 k, 1 KB each,
// K tiles outermost: tile (kt, rt) at byte (kt * ld + rt) * 1024. Row r of a
// tile is 64 contiguous bytes, its four 32-element blocks of 16 bytes each;
// block b stands at position b ^ ((r >> 2) & 3) of the row. The scale words
// of four K tiles (a K group) and one row tile are 64 contiguous uint32:
// word 4 r + b holds in byte t the E8M0 exponent of block b of row r in K
// tile 4 kg + t.
//
// Why this layout. One tile is exactly what a wave feeds to one operand of
// v_mfma_scale_f32_16x16x128_f8f6f4 (a lane: 16 bytes, one block of one
// row), so every copy of it, to LDS or straight to registers, is 1 KB
// contiguous: on MI355X such copies run at 47-49 B/clk per CU from L2, where
// 8 rows x 128 B at a row pitch run at 29-32. A row's 64 bytes repeat the LDS
// banks every four rows; the XOR moves a block of rows four apart to
// different banks, so that a tile is read from LDS without bank conflicts (in
// the lane order of mx4_gemm.hip). With K tiles outermost the tiles that a
// workgroup reads together are one contiguous run, spread over all L2
// channels. A lane's scale word serves four K tiles: the MFMA's op_sel picks
// the byte.
#pragma once

#include <hip/hip_runtime_api.h>
#include <stdint.h>

#include "mx4/mx4_launch.hpp"

namespace fp8q {
namespace mx4 {

struct QuantArgs {
    const uint16_t* x;
    int64_t rows, cols, ld_x, stride_x;  // of x; stride between matrices, in elements
    uint8_t* q;
    int64_t ld_q, stride_q;              // row tiles between K tiles; bytes between matrices
    uint32_t* scale;
    int64_t ld_s, stride_s;              // row tiles between K groups; words between matrices
    int64_t groups;
    bool vec;                            // 16-byte loads of x are aligned
};

struct ScatterArgs {
    const uint16_t* x;
    int64_t tokens, cols, ld_x;
    int topk;
    const int32_t* dst;
    int64_t m_total;
    uint8_t* q;
    int64_t ld_q;
    uint32_t* scale;
    int64_t ld_s;
    bool vec;
};

struct DequantArgs {
    const uint8_t* q;
    int64_t ld_q;
    const uint32_t* scale;
    int64_t ld_s;
    int64_t rows, cols;
    void* y;
    int64_t ld_y;
    bool f32;
    bool vec;  // 16-byte stores to y are aligned
};

hipError_t launch_quant_rows(const QuantArgs& p, hipStream_t stream);
hipError_t launch_quant_cols(const QuantArgs& p, hipStream_t stream);
hipError_t launch_quant_scatter(const ScatterArgs& p, hipStream_t stream);
hipError_t launch_dequant(const DequantArgs& p, hipStream_t stream);

struct GemmArgs {
    int32_t m, n;
    int32_t kt;  // K tiles
    const uint8_t* a;
    int64_t ld_a;  // row tiles between K tiles
    const uint32_t* a_scale;
    int64_t ld_as;  // row tiles between K groups
    const uint8_t* b;
    int64_t ld_b;
    const uint32_t* b_scale;
    int64_t ld_bs;
    void* c;
    int64_t ldc;
    bool out_f32;
    bool c_vec;    // four adjacent outputs of a row may be stored together
    bool c_vec16;  // rows start on 16-byte boundaries
    bool scales16;  // all scale arrays start on 16-byte boundaries
    // grouped problems only: expert e owns rows [off[e], off[e+1]) of A and C
    int32_t groups;
    const int32_t* group_offsets;
    const int32_t* group_rows;
    int64_t stride_b;   // bytes between experts
    int64_t stride_bs;  // words between experts
};

hipError_t launch_gemm(const GemmArgs& p, hipStream_t stream);
hipError_t launch_grouped_gemm(const GemmArgs& p, hipStream_t stream);

}  // namespace mx4
}  // namespace fp8q
