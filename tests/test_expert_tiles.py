"""How the gated products deal an expert's rows out to their 256-row tiles, built
by g++ from the header that the kernel uses: the tiles of a segment partition it,
one to four 64-row quarters each, at any segment that 32-bit offsets can hold."""
from __future__ import annotations

import ctypes
import os
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "fine_grained_fp8_quantize_amd", "csrc")

SOURCE = r"""
#include <cstdint>
#include "expert_tiles.h"
// tiles of a segment that are not where the even split in 64 bits has them, or hold no or more than four quarters
extern "C" int64_t wrong_tiles(int64_t seg) {
    const int64_t tiles = (seg + 255) / 256, quarters = (seg + 63) / 64;
    int64_t at = 0, wrong = 0;
    for (int64_t mt = 0; mt < tiles; ++mt) {
        const fp8q::TileSpan s = fp8q::even_span((int)seg, (int)tiles, (int)mt);
        const int64_t first = mt * quarters / tiles, next = (mt + 1) * quarters / tiles;
        wrong += s.first != 64 * first || s.rows != 64 * (next - first) || s.first != at || s.rows < 64 || s.rows > 256;
        at = (int64_t)s.first + s.rows;
    }
    return wrong + (at != 64 * quarters);
}
"""


@pytest.fixture(scope="module")
def wrong(tmp_path_factory):
    d = tmp_path_factory.mktemp("tiles")
    (d / "tiles.cpp").write_text(SOURCE)
    made = subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-fsanitize=signed-integer-overflow",
                           "-fsanitize-undefined-trap-on-error", "-fPIC", "-shared", "-I", CSRC, str(d / "tiles.cpp"), "-o",
                           str(d / "tiles.so")], capture_output=True, text=True)
    assert made.returncode == 0, made.stdout + made.stderr
    fn = ctypes.CDLL(str(d / "tiles.so")).wrong_tiles
    fn.argtypes, fn.restype = [ctypes.c_int64], ctypes.c_int64
    return fn


def test_short_segments(wrong):
    assert [seg for seg in range(128, 128 * 400, 128) if wrong(seg)] == []


@pytest.mark.parametrize("seg", [5931648, 5931776, 5931904, 5932032, 6000000, 1 << 23, (1 << 27) + 128, (1 << 29) - 128,
                                 1 << 30, (1 << 31) - 256])
def test_segments_of_millions_of_rows(wrong, seg):
    assert seg % 128 == 0 and wrong(seg) == 0
