"""How large the launches of the gated products' rows kernels get, by the rules
that the launchers use: their sizes are not looked at in the calls."""
from __future__ import annotations

import ctypes
import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "fine_grained_fp8_quantize_amd", "csrc")

pytestmark = pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")

SOURCE = r"""
#include "gated/gated_launch.hpp"
using namespace fp8q;
using namespace fp8q::gated;
static int64_t most = 0;
static int bad(int64_t across, int64_t down, int waves) {
    if (across * down > most) most = across * down;
    return waves < 1 || waves > 16 || across * down > kRowsMostPieces || down > 65535 ||
           !launchable({across * down, 64 * waves});
}
extern "C" int dense(int64_t m, int64_t n, int64_t k) {
    const RowsForm f = rows_form(m, n, k);
    return f.ms ? bad(parts_of(n, kRowsColumns * f.nt), parts_of(m, 16 * f.ms), f.waves) : 0;
}
extern "C" int grouped(int64_t m, int64_t n, int64_t k) {
    return grouped_rows(m, n) ? bad(parts_of(n, kRowsColumns), m / 64, grouped_rows_waves(k)) : 0;
}
extern "C" int segments(int64_t m, int64_t n, int full) { return grouped_rows(m, n, full != 0); }
extern "C" int64_t largest() { return most; }
// every n up to `to`, and both ends of the steps of m, at one K
extern "C" int sweep(int64_t to, int64_t k) {
    int wrong = 0;
    for (int64_t n = 1; n <= to; ++n)
        for (int64_t m = 128; m <= (1 << 20) + 65536; m += m < 65536 ? 128 : 16384)
            for (int64_t d = -1; d <= 1; ++d) {
                wrong += dense(m + d, n, k);
                if (d == 0) wrong += grouped(m, n, k);
            }
    return wrong;
}
"""


@pytest.fixture(scope="module")
def rules(tmp_path_factory):
    d = tmp_path_factory.mktemp("bounds")
    (d / "bounds.cpp").write_text(SOURCE)
    made = subprocess.run(["g++", "-std=c++17", "-O2", "-Wall", "-fPIC", "-shared", "-I", CSRC, str(d / "bounds.cpp"), "-o",
                           str(d / "bounds.so")], capture_output=True, text=True)
    assert made.returncode == 0, made.stdout + made.stderr
    L = ctypes.CDLL(str(d / "bounds.so"))
    L.sweep.argtypes = [ctypes.c_int64] * 2
    L.dense.argtypes = L.grouped.argtypes = [ctypes.c_int64] * 3
    L.segments.argtypes = [ctypes.c_int64, ctypes.c_int64, ctypes.c_int]
    L.largest.restype = ctypes.c_int64
    return L


def test_the_rows_kernels_launches(rules):
    for k in (0, 128, 7168):
        assert rules.sweep(700, k) == 0
    for k in (0, 128, 7168, 1 << 20):
        for n in (1 << 10, 1 << 14, 16385, 24576, 1 << 15, 65537, 1 << 20, (1 << 31) - 1, 1 << 40):
            for m in (1, 16, 17, 32, 33, 64, 65, 128, 1000, 1 << 14, 1 << 20):
                assert rules.dense(m, n, k) == 0 and rules.grouped(-(-m // 128) * 128, n, k) == 0
    assert rules.largest() == 1 << 16  # the bound is met: experts' 2^20 rows of 25 to 32 columns


def test_full_segments_take_tiles_earlier(rules):
    """Where the host knows that all rows are real, the rows kernel has half the pieces."""
    for m, n, some, full in ((512, 512, 1, 1), (512, 1024, 1, 1), (512, 1536, 1, 0), (512, 2048, 1, 0), (4096, 256, 1, 0),
                             (1024, 2048, 0, 0)):
        assert (rules.segments(m, n, 0), rules.segments(m, n, 1)) == (some, full), (m, n)
