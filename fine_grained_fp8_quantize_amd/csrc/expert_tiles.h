// expert_tiles.h -- which of an expert's rows a 256-row tile of the gated
// products takes (internal; constexpr, so device and host code may call it; it
// needs no HIP header, so that the split can be tested alone).
#pragma once

namespace fp8q {

// Rows [first, first + rows) of the segment.
struct TileSpan {
    int first;
    int rows;
};

// The segment's 64-row quarters dealt out evenly to its tiles = ceil(seg / 256)
// m-tiles: tile mt begins at quarter floor(mt * quarters / tiles). The product
// passes 32 bits in segments of 6 million rows; with quarters = 4 tiles - short,
// short 0..3, it is 4 mt - ceil(mt * short / tiles), which does not.
constexpr int even_quarter(int mt, int short_of, int tiles) {
    return 4 * mt - (mt * short_of + tiles - 1) / tiles;
}
constexpr TileSpan even_span(int seg, int tiles, int mt) {
    const int short_of = 4 * tiles - (seg + 63) / 64;
    const int first = even_quarter(mt, short_of, tiles), next = even_quarter(mt + 1, short_of, tiles);
    return {64 * first, 64 * (next - first)};
}

}  // namespace fp8q
