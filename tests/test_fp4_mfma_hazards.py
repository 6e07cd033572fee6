"""The FP4 tile kernels issue their matrix instructions from inline assembly,
so the compiler puts no wait states around them. Here the kernels are compiled
to assembly and looked over: nothing touches a result before it is there."""
from __future__ import annotations

import os
import re
import subprocess

import pytest

import mfma_hazards
from fine_grained_fp8_quantize_amd import build

HERE = os.path.dirname(os.path.abspath(__file__))

pytestmark = pytest.mark.skipif(not os.path.exists(build.HIPCC), reason="needs hipcc")


def listing(source, out, *flags):
    cmd = [build.HIPCC, *(f for f in build.FLAGS if f not in ("-shared", "-fPIC")), "-I", build.INCLUDE, "-I", build.CSRC,
           *flags, "--cuda-device-only", "-S", source, "-o", str(out)]
    made = subprocess.run(cmd, capture_output=True, text=True)
    assert made.returncode == 0, made.stdout + made.stderr
    return out.read_text()


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    return listing(os.path.join(build.CSRC, "mx4", "mx4_gemm.hip"), tmp_path_factory.mktemp("isa") / "mx4_gemm.s")


def test_the_tile_kernels(kernels):
    report = mfma_hazards.check(kernels)
    assert len(report) == 6 and all("tiles_kernel" in name for name in report)
    for name, (count, found) in report.items():
        assert count >= 64 and not found, (name, found[:5])


def test_a_read_behind_a_product_would_be_seen(kernels):
    """The same listing with one more instruction per kernel, a read too early."""
    planted, n = re.subn(r"(\tv_mfma_scale\S+ a\[(\d+):\d+\][^\n]*\n\s*;;#ASMEND\n)", r"\1\tv_accvgpr_read_b32 v0, a\2\n",
                         kernels)
    assert n >= 6 and all(found for _, found in mfma_hazards.check(planted).values())


def test_results_cannot_be_read_ahead_of_the_wait(tmp_path):
    report = mfma_hazards.check(listing(os.path.join(HERE, "host", "settle_probe.hip"), tmp_path / "probe.s"))
    (count, found), = report.values()
    assert count == 1 and not found, found


def kernel(*lines):
    text = "_Zk:\n" + "\n".join(lines) + "\n\ts_endpgm\n.Lfunc_end0:\n"
    text = re.sub(r"^MFMA(.*)$", r"\t;;#ASMSTART\n\tv_mfma_scale_f32_16x16x128_f8f6f4\1\n\t;;#ASMEND", text, flags=re.M)
    return mfma_hazards.check(text)["_Zk"][1]


def test_the_check_itself():
    mfma = "MFMA a[0:3], v[0:3], v[4:7], a[0:3], v8, v9"
    assert kernel(mfma, "\tv_accvgpr_read_b32 v1, a2")
    assert kernel(mfma, "\ts_nop 10", "\tv_accvgpr_read_b32 v1, a2")
    assert not kernel(mfma, "\ts_nop 11", "\tv_accvgpr_read_b32 v1, a2")
    assert not kernel(mfma, "\tv_accvgpr_read_b32 v1, a4")
    assert not kernel(mfma, mfma)
    assert kernel(mfma, "\tv_accvgpr_write_b32 a3, v1")
    assert kernel("\tv_mov_b32_e32 v9, 0", "\ts_nop 0", mfma) and not kernel("\tv_mov_b32_e32 v9, 0", "\ts_nop 1", mfma)
    # over branches, backward ones too
    assert kernel(mfma, "\ts_cbranch_scc1 .LBB0_1", "\ts_nop 15", ".LBB0_1:", "\tv_accvgpr_read_b32 v1, a2")
    assert kernel("\ts_nop 15", ".LBB0_1:", "\tv_accvgpr_read_b32 v1, a2", "\ts_nop 15", mfma, "\ts_cbranch_scc1 .LBB0_1")
    assert not kernel(mfma, "\ts_branch .LBB0_2", ".LBB0_1:", "\tv_accvgpr_read_b32 v1, a2", ".LBB0_2:", "\ts_nop 15")
