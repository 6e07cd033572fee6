"""The launch rules of the gated products and the weight-only products, built by
g++ from the headers that the launchers use: every kernel form that a launcher
can start is one that the rules choose, at sizes that the GPU tests run."""
from __future__ import annotations

import ctypes
import os
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "fine_grained_fp8_quantize_amd", "csrc")

SOURCE = r"""
#include "gated/gated_launch.hpp"
#include "gemv/gemv_launch.hpp"
extern "C" void rows_form(int64_t m, int64_t n, int64_t k, int* out) {
    const fp8q::gated::RowsForm f = fp8q::gated::rows_form(m, n, k);
    out[0] = f.ms; out[1] = f.nt; out[2] = f.waves;
}
extern "C" void grouped_form(int64_t m, int64_t n, int64_t k, int* out) {
    out[0] = fp8q::gated::grouped_rows(m, n); out[1] = fp8q::gated::grouped_rows_waves(k);
}
extern "C" void gemv_form(int64_t t, int64_t topk, int64_t e, int64_t n, int64_t k, int gated, int* out) {
    const fp8q::gemv::Form f = fp8q::gemv::form(t, topk, e, n, k, gated != 0);
    out[0] = f.ms; out[1] = f.nt; out[2] = f.waves; out[3] = f.tiles; out[4] = (int)f.rows;
}
"""


@pytest.fixture(scope="module")
def rules(tmp_path_factory):
    d = tmp_path_factory.mktemp("rules")
    (d / "rules.cpp").write_text(SOURCE)
    made = subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-fPIC", "-shared", "-I", CSRC, str(d / "rules.cpp"), "-o",
                           str(d / "rules.so")], capture_output=True, text=True)
    assert made.returncode == 0, made.stdout + made.stderr
    L = ctypes.CDLL(str(d / "rules.so"))

    def call(name, *args, size=5):
        out = (ctypes.c_int * size)()
        getattr(L, name)(*[ctypes.c_int64(a) for a in args[:5]], *args[5:], out)
        return list(out)

    return call


def test_gated_forms(rules):
    """(rows of a tile / 16, column groups): what launch_gated can start."""
    import test_gpu_gated as gpu
    want = {(1, 1), (2, 1), (4, 1), (4, 2), (0, 0)}
    assert {tuple(rules("rows_form", *s, size=3)[:2]) for s in gpu.SHAPES} == want
    for m in (1, 16, 17, 32, 33, 64, 65, 256, 1000, 5000, 1 << 20, 1 << 23, 1 << 30):
        for n in (1, 8, 128, 1000, 2048, 1 << 20):
            for k in (0, 128, 1024, 7168, 1 << 20):
                ms, nt, waves = rules("rows_form", m, n, k, size=3)
                assert (ms, nt) in want
                assert ms == 0 or m <= 16 * ms * 65535
                if ms:
                    assert 1 <= waves <= (8 if ms * nt >= 8 else 16) and waves * nt * ms <= 64  # KB of LDS


def test_grouped_forms(rules):
    import test_gpu_gated as gpu
    seen = set()
    for rows, more in gpu.EXPERTS:
        m = sum(-(-r // 128) * 128 for r in rows) + more
        for n, k in gpu.COLUMNS:
            seen.add((rules("grouped_form", m, n, k, size=2)[0], n % 128 == 0))
    assert seen == {(0, False), (0, True), (1, False), (1, True)}
    for m in (128, 1024, 8192, 1 << 20, 1 << 23, 1 << 30):
        for n in (1, 8, 128, 2048, 1 << 20):
            for k in (0, 128, 1024, 7168, 1 << 20):
                rows, waves = rules("grouped_form", m, n, k, size=2)
                assert not rows or (m <= 64 * 65535 and 1 <= waves <= 16)  # 4 KB of LDS per wave


def test_gemv_forms(rules):
    import test_gpu_gemv as gpu
    seen = set()
    for m, n, k in gpu.SHAPES:
        seen.add(tuple(rules("gemv_form", m, 0, 1, n, k, 0)[:2]))
    assert seen == {(ms, nt) for ms in (1, 2, 4) for nt in (1, 2, 4)}
    for t in (1, 16, 17, 33, 200, 4096):
        for topk in (0, 1, 8):
            for n in (1, 16, 2048, 7168, 1 << 17):
                for k in (0, 1, 128, 2048, 7168, 1 << 18):
                    ms, nt, waves, tiles, rows = rules("gemv_form", t, topk, 32, n, k, 1)
                    assert ms in (1, 2, 4) and nt in (1, 2, 4) and 1 <= waves <= (16 if ms == 1 else 8)
                    assert waves * tiles * 128 >= k and (waves - 1) * tiles * 128 < max(k, 1)
                    assert waves * nt * ms <= 128  # KB of LDS, beside 8 for the routes
