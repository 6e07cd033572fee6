// gemv_launch.hpp -- launch sizes of the products of few rows with FP4 weights
// (internal, host code only; it needs no HIP header, so that the rules can be
// tested alone). Every rule depends on sizes alone.
#pragma once

#include "mx4/mx4_launch.hpp"

namespace fp8q {
namespace gemv {

using mx4::ceil_div;

constexpr int kMaxExperts = 1024;
constexpr int kMaxRoutes = 4096;
constexpr int kMaxTopk = 32;
// Waves of a workgroup: more than one row tile takes more than 128 registers.
constexpr int max_waves(int ms) { return ms == 1 ? 16 : 8; }

// A gated group is 8 gate and 8 up columns.
inline int64_t column_groups(int64_t n, bool gated) { return ceil_div(n, gated ? 8 : 16); }

// 16 ms rows by nt column groups per workgroup; wave w takes `tiles` K tiles.
struct Form {
    int ms, nt;
    int waves;
    int tiles;
    int64_t rows;  // workgroups along the rows (topk > 0: along the experts)
};

// topk: 0 without ids.
inline Form form(int64_t tokens, int64_t topk, int64_t experts, int64_t n, int64_t k, bool gated) {
    Form f;
    f.ms = tokens <= 16 ? 1 : (tokens <= 32 ? 2 : 4);
    const int64_t routes = tokens * topk;
    f.rows = topk > 0 ? (routes < experts ? routes : experts) + 1 : ceil_div(tokens, 16 * f.ms);
    const int64_t kt = k > 0 ? ceil_div(k, mx4::kTileK) : 1;
    // Column groups per workgroup: as few as make one round of the 256 CUs, and at most four. Every CU streams at a
    // rate of its own, so that 257 workgroups take as long as 512, and fewer, wider ones read x less often (us for 1 /
    // 2 / 4 groups: 5 rows, 2050 gated columns, K = 7168, 257 groups: 13.0 / 10.7 / 12.7; 1 row, 7168 x 2048, 448
    // groups: 5.6 / 5.1 / 5.9; 1 row, 16384 x 7168, 1024 groups: 21.6 / 18.4 / 14.7; 1 row, 2048 gated columns, 256
    // groups: 8.2 / 10.2 / 12.6; 64 routes over 32 experts, 2048 gated columns, about 7000 groups: 142 / 94 / 86).
    const int64_t groups = column_groups(n, gated) * (topk > 0 ? f.rows - 1 : f.rows);
    f.nt = groups <= 256 ? 1 : (groups <= 512 ? 2 : 4);
    // Waves: as many as have a step of loads each; four where there are several rounds of workgroups, which then hide
    // each other's start and end (experts' 7168 x 2048, 28 of them: 41 us with 4 waves, 54 with 8; 16384 x 7168: 15
    // with 8, 20 with 4).
    const int64_t wgs = ceil_div(column_groups(n, gated), f.nt) * f.rows;
    int waves = wgs > 512 ? 4 : (f.nt == 4 ? 8 : max_waves(f.ms));
    const int64_t steps = ceil_div(kt, 4 / f.nt);
    if (steps < waves) waves = (int)steps;
    f.tiles = (int)ceil_div(kt, waves);
    f.waves = (int)ceil_div(kt, f.tiles);
    return f;
}

}  // namespace gemv
}  // namespace fp8q
