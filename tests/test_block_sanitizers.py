"""The entry points of the gated block, the weight-only products and the
optimizer under AddressSanitizer and UndefinedBehaviorSanitizer: their host code
and api.cpp built by g++ with launcher stubs, and their ABI suites run against
that build in a child process."""
from __future__ import annotations

import os
import shutil
import subprocess
import sys

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(ROOT, "fine_grained_fp8_quantize_amd", "csrc")
SAN = ["-fsanitize=address,undefined", "-fno-sanitize-recover=undefined", "-fno-omit-frame-pointer", "-g", "-O1"]


@pytest.mark.skipif(shutil.which("gcc") is None or shutil.which("g++") is None, reason="needs gcc and g++")
def test_abi_suites_under_asan_ubsan(tmp_path):
    lib = str(tmp_path / "libfp8q_host_asan.so")
    sources = [os.path.join(CSRC, s) for s in ("api.cpp", "gated/gated_api.cpp", "gemv/gemv_api.cpp",
                                               "adamw/adamw_api.cpp")]
    stubs = [os.path.join(HERE, "sanitize", s) for s in ("launch_stubs.cpp", "block_stubs.cpp")]
    made = subprocess.run(["g++", *SAN, "-std=c++17", "-fPIC", "-shared", "-Wall", "-D__HIP_PLATFORM_AMD__",
                           "-I", "/opt/rocm/include", "-I", os.path.join(ROOT, "include"), "-I", CSRC, *sources, *stubs,
                           "-o", lib, "-L", "/opt/rocm/lib", "-Wl,-rpath,/opt/rocm/lib", "-lamdhip64"],
                          capture_output=True, text=True)
    assert made.returncode == 0, made.stdout + made.stderr
    asan = subprocess.run(["gcc", "-print-file-name=libasan.so"], capture_output=True, text=True, check=True).stdout.strip()
    env = dict(os.environ, LD_PRELOAD=asan, FP8Q_LIBRARY=lib,
               ASAN_OPTIONS="detect_leaks=0:detect_odr_violation=0:alloc_dealloc_mismatch=0:abort_on_error=1:"
                            "verify_asan_link_order=0",
               UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    env["PYTHONPATH"] = os.pathsep.join([ROOT, HERE] + [p for p in env.get("PYTHONPATH", "").split(os.pathsep) if p])
    res = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-p", "no:cacheprovider", "-m", "not gpu",
                          *(os.path.join(HERE, t) for t in ("test_gated_abi.py", "test_gemv_abi.py", "test_adamw_abi.py"))],
                         cwd=ROOT, env=env, capture_output=True, text=True, timeout=1200)
    tail = (res.stdout + res.stderr)[-4000:]
    assert res.returncode == 0, tail
    assert "passed" in res.stdout and "ERROR: AddressSanitizer" not in tail and "runtime error" not in tail, tail
