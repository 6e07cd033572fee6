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
constexpr int kMaxWaves = 16;  // 8 where four row tiles take the registers

// 16 ms rows by `cols` columns per workgroup; wave w takes `tiles` K tiles.
struct Form {
    int ms;
    int waves;
    int tiles;
};

inline Form form(int64_t rows, int64_t k) {
    const int ms = rows <= 16 ? 1 : (rows <= 32 ? 2 : 4);
    const int64_t kt = k > 0 ? ceil_div(k, mx4::kTileK) : 1, tiles = ceil_div(kt, ms == 4 ? 8 : kMaxWaves);
    return {ms, (int)ceil_div(kt, tiles), (int)tiles};
}

// A gated workgroup has 8 gate and 8 up columns.
inline int64_t column_groups(int64_t n, bool gated) { return ceil_div(n, gated ? 8 : 16); }

}  // namespace gemv
}  // namespace fp8q
