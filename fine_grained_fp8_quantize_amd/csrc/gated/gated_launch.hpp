// gated_launch.hpp -- which gated kernel takes a problem, and the launches'
// sizes (internal, host code only; it needs no HIP header, so that the rules
// can be tested alone). Every rule depends on sizes alone.
#pragma once

#include "launch_shape.hpp"

namespace fp8q {
namespace gated {

inline int64_t parts_of(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Few rows: 16 ms rows by 8 nt columns (nt times 8 gate and 8 up weight rows)
// per workgroup, K split over its waves, four slabs of a wave in flight with
// one row tile and two with more.
struct RowsForm {
    int ms;  // 0: the tile kernel
    int nt;
    int waves;
};
constexpr int kRowsColumns = 8;
// The most workgroups that rows_form and grouped_rows choose a rows kernel for: a
// tile's share of the limit is 8 pieces, so that rows of many tiles take the
// rows kernel only where n is so small that a tile has no more of them (n up to
// 16, experts' 128-row segments up to 32), and the 2^20 rows that either rule
// allows end that: 32 columns of that many are 2^16, a 64th of what a launch may
// hold.
constexpr int64_t kRowsMostPieces = 1 << 16;
// (eight accumulators and more take more than 128 registers)
constexpr int rows_waves(int accumulators) { return accumulators >= 8 ? 8 : 16; }

// Tiles of 256 rows by 128 columns.
inline int64_t tiles_of(int64_t m, int64_t n) { return parts_of(m, 256) * parts_of(n, 128); }

inline RowsForm rows_form(int64_t m, int64_t n, int64_t k) {
    const int ms = m <= 16 ? 1 : (m <= 32 ? 2 : 4);
    const int64_t wgs = parts_of(m, 16 * ms) * parts_of(n, kRowsColumns);
    // Against the tile kernel, which takes as long for one row of tiles as for 256 of them (us, rows kernel and tiles:
    // 2048 columns, K = 7168, 64 rows: 22 / 73; 256: 50 / 97; 512, 2048 pieces of 64 x 8: 94 / 95; 1024: 205 / 94;
    // 1000 columns, K = 1024, 1024 rows, 2000 pieces: 18.4 / 19.4; K = 7168, 16384 columns, 2048 pieces, 1 row: 56 / 81,
    // 16: 75 / 81, 32: 102 / 83; 24576 columns, 1 row: 82 / 86, 16: 111 / 87).
    // (A launch has fewer than 2^16 workgroups along the rows.)
    if (wgs > (ms == 2 ? 1536 : 2048) * parts_of(tiles_of(m, n), 256) || m > 1 << 20) return {0, 0, 0};
    // Twice the columns, so that A is read half as often, once one column group each makes more than one round of the
    // CUs (64 rows x 2048: 21.8 us with one, 30.1 with two; 128: 40.5 / 29.8; 256: 77 / 50).
    const int nt = ms == 4 && wgs > 256 ? 2 : 1;
    const int64_t slabs = k >= 128 ? k / 128 : 1, at_once = (int64_t)rows_waves(ms * nt) * (ms == 1 ? 4 : 2);
    const int64_t steps = parts_of(slabs, at_once);
    return {ms, nt, (int)parts_of(slabs, steps * (ms == 1 ? 4 : 2))};
}

inline LaunchShape tiles_shape(int64_t m, int64_t n) { return {parts_of(tiles_of(m, n), 8) * 8, 512}; }
// Experts with few columns or few rows set aside: quarters of 64 rows by 8
// columns, by the same rule. How many of the rows are real only the GPU knows:
// segments of 128 rows with 2 / 16 / 32 / 64 / 128 real ones (us, rows kernel
// and, one round of them whatever the rows, tiles: 4 experts, 2 x 512 x 7168,
// 512 pieces: 12 / 14 / 18 / 23 / 40 and 68 to 75; 1024 columns, 1024 pieces: 20 /
// 25 / 30 / 42 / 76; 2048 columns, 2048 pieces: 37 / 46 / 57 / 81 / 153; 32
// experts, 256 columns: 39 / 49 / 61 / 84 / 149; 4 experts, 512 columns, K =
// 2048: 7 / 8 / 10 / 14 / 14 and 27 to 29). Mostly full segments near the limit
// are the price of the few rows that decoding has in them. `full`: the host
// knows that all rows are real (no group_rows). Then half the pieces (us, rows
// kernel and tiles, K = 7168 / 2048 / 512: 4 experts of 128 rows, 768 pieces:
// 58 and 66 / 20 and 26 / 8 and 14; 1024: 76 and 68 / 24 and 27 / 9 and 14, of
// one expert of 512 rows 75 and 85 / 23 and 33 / 8 and 17; 1536: 115 and 68 / 35
// and 27 / 12 and 14; 2048: 154 and 70 / 46 and 28 / 15 and 15).
inline bool grouped_rows(int64_t m_total, int64_t n, bool full = false) {
    const int64_t wgs = m_total / 64 * parts_of(n, kRowsColumns);
    return wgs <= (full ? 1024 : 2048) * parts_of(m_total / 128 * parts_of(n, 128), 256) && m_total <= 1 << 20;
}
inline int grouped_rows_waves(int64_t k) {
    const int64_t slabs = k >= 128 ? k / 128 : 1, steps = parts_of(slabs, 32);
    return (int)parts_of(slabs, 2 * steps);
}
// (every 256-row tile of an expert holds at least 128 of its rows)
inline LaunchShape grouped_shape(int64_t m_total, int64_t n) {
    return {parts_of(m_total / 128 * parts_of(n, 128), 256) * 256, 512};
}

// Bytes of FP32 scratch that E4M3 output goes through: the 128 columns of a
// scale belong to 16 workgroups of the rows kernel.
inline int64_t workspace_bytes(int64_t m, int64_t n, int64_t k) { return rows_form(m, n, k).ms ? m * n * 4 : 0; }

inline int64_t grouped_workspace_bytes(int64_t m_total, int64_t n) {
    return grouped_rows(m_total, n) ? m_total * n * 4 : 0;
}

// Gradient: 8 columns of a row per thread, or panels of 128 x 128.
constexpr int kBackwardThreads = 256;
constexpr int kPanelThreads = 512;
inline LaunchShape backward_shape(int64_t m, int64_t n) {
    return {parts_of(m * parts_of(n, 8), kBackwardThreads), kBackwardThreads};
}
inline LaunchShape panel_shape(int64_t m, int64_t n) { return {(m / 128) * (n / 128), kPanelThreads}; }

}  // namespace gated
}  // namespace fp8q
