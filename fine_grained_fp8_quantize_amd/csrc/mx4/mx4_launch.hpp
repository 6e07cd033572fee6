// mx4_launch.hpp -- which FP4 kernel takes a problem, and the launch's size
// (internal, host code only; it needs no HIP header, so that the rules can be
// tested alone). Every rule depends on sizes alone.
#pragma once

#include "launch_shape.hpp"

namespace fp8q {
namespace mx4 {

constexpr int kTileRows = 16;
constexpr int kTileK = 128;
constexpr int kTileBytes = 1024;
constexpr int kGroupTiles = 4;              // K tiles that share scale words
constexpr int kGroupK = kTileK * kGroupTiles;
constexpr int kScaleWords = 64;             // per row tile and K group

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// ------------------------------------------------------------- quantizers

constexpr int kQuantWaves = 4;      // a wave takes 16 rows x 512 k
constexpr int kColsThreads = 512;   // the transposing quantizer: 256 tokens
constexpr int kColsKTiles = 2;      // (two K tiles, half a group) by 128
constexpr int kColsChannels = 128;  // channels per workgroup

inline int64_t quant_rows_units(int64_t groups, int64_t rows, int64_t cols) {
    return groups * ceil_div(rows, kTileRows) * ceil_div(cols, kGroupK);
}
inline LaunchShape quant_rows_shape(int64_t groups, int64_t rows, int64_t cols) {
    return {ceil_div(quant_rows_units(groups, rows, cols), kQuantWaves), 64 * kQuantWaves};
}
// (both halves of the last K group, whose scale bytes must all be written)
inline int64_t quant_cols_halves(int64_t rows) { return 2 * ceil_div(rows, kGroupK); }
inline int64_t quant_cols_units(int64_t groups, int64_t rows, int64_t cols) {
    return groups * ceil_div(cols, kColsChannels) * quant_cols_halves(rows);
}
inline LaunchShape quant_cols_shape(int64_t groups, int64_t rows, int64_t cols) {
    return {ceil_div(quant_cols_units(groups, rows, cols), 8) * 8, kColsThreads};
}

// --------------------------------------------------------------- products

enum class GemmKernel { kRows, kTiles, kGroupedTiles };

// kRows: ms row tiles by nt column tiles of 16 per workgroup, K split over its
// waves. kTiles: 32 ms x 32 nt outputs per workgroup. kGroupedTiles: 256 x 256.
struct GemmForm {
    GemmKernel kernel;
    int ms, nt;
};

// With four row tiles a wave needs up to 200 registers: eight waves.
constexpr int max_waves(int ms) { return ms >= 4 ? 8 : 16; }

// Waves of a kRows workgroup: every wave the same number of K groups, as far
// as they divide.
inline int rows_waves(int ms, int64_t kt) {
    const int64_t kg = ceil_div(kt, kGroupTiles);
    if (kg <= 0) return 1;
    return (int)ceil_div(kg, ceil_div(kg, max_waves(ms)));
}

// Column tiles per workgroup: the fewest with which the workgroups are one round
// of the 256 CUs, and at most four; a workgroup with more of them reads A less
// often but runs longer (one row, K = 7168, 1 / 2 / 4 column tiles: n = 4096: 6.2 /
// 7.3 / 9.5 us; 8192: 9.5 / 8.5 / 10.7; 16384: 18.7 / 15.3 / 13.6; 64 rows: n =
// 8192: 15.5 / 13.3 / 18.0; 48 rows, K = 4096, n = 10000: 13.2 / 14.1 / 11.8).
// `busy`: row tiles that are likely to have work.
inline GemmForm rows_form(int ms, int64_t busy, int64_t n) {
    const int64_t tiles = busy * ceil_div(n, 16);
    // (two row tiles by four columns do not fit 128 registers)
    return {GemmKernel::kRows, ms, tiles > 512 && ms != 2 ? 4 : (tiles > 256 ? 2 : 1)};
}

// Rounds of the 256 CUs that tiles of size x size take.
inline int64_t rounds_of(int64_t m, int64_t n, int64_t size) {
    return ceil_div(ceil_div(m, size) * ceil_div(n, size), 256);
}

// scales16: both scale arrays (every expert's) start on 16-byte boundaries. The
// tile kernels copy scale words to LDS 16 bytes at a time; scales that are
// aligned to their 4-byte words only go to the rows kernel, which reads words.
inline GemmForm gemm_form(int64_t m, int64_t n, bool scales16) {
    if (m <= 16) return rows_form(1, 1, n);
    if (m <= 32) return rows_form(2, 1, n);
    // Pieces of 64 x 64 with K split over a workgroup's waves, while they are
    // less than one round of the CUs: a whole K sum per wave is the longer way
    // (64 x 4096 x 7168: 10.3 against 14.7 us with 128 x 128 tiles; 256 x 4096 x
    // 7168, 256 pieces: 17.0 against 15.0).
    const int64_t rows64 = ceil_div(m, 64);
    if (!scales16 || rows64 * ceil_div(n, 64) <= 192) return rows_form(4, rows64, n);
    // 256 x 256 tiles or 128 x 128 ones, by the time of a round of the 256 CUs:
    // a tile of the first kind takes about as long as 3.2 of the second one
    // after the other on a CU (two share it). (4096 x 4096 x 7168: 59 against
    // 69 us; 2048 x 4096 x 7168: 42 against 36; 1024 x 4096 x 7168: 40 against 20.)
    const int size = 16 * rounds_of(m, n, 256) <= 5 * rounds_of(m, n, 128) ? 8 : 4;
    return {GemmKernel::kTiles, size, size};
}

inline GemmForm grouped_form(int64_t m_total, int64_t n, int64_t groups, bool scales16) {
    // How many rows an expert has is not known here; m_total bounds their sum.
    const int64_t avg = m_total / groups, columns = ceil_div(n, 256);
    // Tiles of 256 columns once the experts alone give three tiles for four CUs
    // (27 experts with 2 rows, 2048 x 4096, 216 tiles: 27 us, 28 without LDS);
    // otherwise narrow pieces with K split over the waves. Fewer rows than
    // experts (avg = 0) belong to one expert in 16 at the most, segments being
    // whole row tiles, and take the narrow pieces.
    if (scales16 && groups * ceil_div(avg, 256) * columns >= 192) return {GemmKernel::kGroupedTiles, 8, 8};
    // Row tiles of 16, 32 or 64 rows, or 256 x 256 tiles again when there are
    // rows for them (8 experts, 2048 x 4096, us for each of the four: 16 rows an
    // expert: 9.9 / 10.2 / 13.4 / 19.8; 32: 12.7 / 11.2 / 13.6 / 20.7; 48: 16.8 /
    // 16.2 / 13.8 / 21.5; 64: 20.4 / 17.1 / 14.8 / 22.6; 128: 35.1 / 28.6 / 24.4 /
    // 25.0; 256: 65.3 / 52.2 / 42.4 / 31.7).
    if (avg <= 20) return rows_form(1, groups, n);
    if (avg <= 40) return rows_form(2, groups, n);
    const int64_t rows64 = m_total / 64 + groups + 1;
    if (!scales16 || rows64 * ceil_div(n, 64) <= 768) return rows_form(4, rows64, n);
    return {GemmKernel::kGroupedTiles, 8, 8};
}

inline LaunchShape gemm_shape(GemmForm f, int64_t m, int64_t n, int64_t kt) {
    if (f.kernel == GemmKernel::kRows)
        return {ceil_div(m, 16 * f.ms) * ceil_div(n, 16 * f.nt), 64 * rows_waves(f.ms, kt)};
    return {ceil_div(ceil_div(m, 32 * f.ms) * ceil_div(n, 32 * f.nt), 8) * 8, 256};
}

// (at most one ragged row tile per segment, and one past the last)
inline LaunchShape grouped_shape(GemmForm f, int64_t m_total, int64_t n, int64_t kt, int64_t groups) {
    const bool rows = f.kernel == GemmKernel::kRows;
    const int64_t bm = rows ? 16 * f.ms : 256, bn = rows ? 16 * f.nt : 256;
    return {ceil_div((m_total / bm + groups + 1) * ceil_div(n, bn), 256) * 256, rows ? 64 * rows_waves(f.ms, kt) : 256};
}

}  // namespace mx4
}  // namespace fp8q
