// gated_launch.hpp -- which gated kernel takes a problem, and the launches'
// sizes (internal, host code only; it needs no HIP header, so that the rules
// can be tested alone). Every rule depends on sizes alone.
#pragma once

#include "launch_shape.hpp"

namespace fp8q {
namespace gated {

inline int64_t parts_of(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Few rows: 16 ms rows by 8 columns (8 gate and 8 up weight rows) per
// workgroup, K split over its waves, `unroll` slabs of a wave in flight.
struct RowsForm {
    int ms;  // 0: the tile kernel
    int unroll;
    int waves;
};
constexpr int kRowsColumns = 8;
constexpr int kRowsMost = 64;

inline RowsForm rows_form(int64_t m, int64_t k) {
    if (m > kRowsMost) return {0, 0, 0};
    const int ms = m <= 16 ? 1 : (m <= 32 ? 2 : 4), unroll = ms == 1 ? 4 : 2;
    const int64_t slabs = k / 128, steps = parts_of(slabs > 0 ? slabs : 1, 16 * unroll);
    return {ms, unroll, (int)parts_of(slabs > 0 ? slabs : 1, steps * unroll)};
}
inline LaunchShape rows_shape(RowsForm f, int64_t n) { return {parts_of(n, kRowsColumns), 64 * f.waves}; }

// Tiles of 256 rows by 128 columns.
inline LaunchShape tiles_shape(int64_t m, int64_t n) {
    return {parts_of(parts_of(m, 256) * parts_of(n, 128), 8) * 8, 512};
}
// (every 256-row tile of an expert holds at least 128 of its rows)
inline LaunchShape grouped_shape(int64_t m_total, int64_t n) {
    return {parts_of(m_total / 128 * parts_of(n, 128), 256) * 256, 512};
}

// Bytes of FP32 scratch that E4M3 output goes through: the 128 columns of a
// scale belong to 16 workgroups of the rows kernel.
inline int64_t workspace_bytes(int64_t m, int64_t n, int64_t k) { return rows_form(m, k).ms ? m * n * 4 : 0; }

// Gradient: 8 columns of a row per thread, or panels of 128 x 128.
constexpr int kBackwardThreads = 256;
constexpr int kPanelThreads = 512;
inline LaunchShape backward_shape(int64_t m, int64_t n) {
    return {parts_of(m * parts_of(n, 8), kBackwardThreads), kBackwardThreads};
}
inline LaunchShape panel_shape(int64_t m, int64_t n) { return {(m / 128) * (n / 128), kPanelThreads}; }

}  // namespace gated
}  // namespace fp8q
