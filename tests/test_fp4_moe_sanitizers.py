"""The FP4 and MoE entry points' host code under AddressSanitizer and
UndefinedBehaviorSanitizer: api.cpp, mx4_api.cpp and moe_api.cpp built by g++
with launcher stubs, and the two ABI suites run against that build in a child
process. The workspace size is the kernels' own plan, so its test is left out."""
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
    sources = [os.path.join(CSRC, s) for s in ("api.cpp", "mx4/mx4_api.cpp", "moe/moe_api.cpp")]
    stubs = [os.path.join(HERE, "sanitize", s) for s in ("launch_stubs.cpp", "mx4_moe_stubs.cpp")]
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
    probe = subprocess.run([sys.executable, "-c", "import fine_grained_fp8_quantize_amd as fq; fq._load();"
                            "maps = open('/proc/self/maps').read();"
                            "assert 'libasan' in maps and 'libfp8q_host_asan.so' in maps"],
                           cwd=ROOT, env=env, capture_output=True, text=True, timeout=300)
    assert probe.returncode == 0, probe.stdout + probe.stderr
    res = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-p", "no:cacheprovider", "-m", "not gpu",
                          "-k", "not workspace_bytes", os.path.join(HERE, "test_fp4_abi.py"),
                          os.path.join(HERE, "test_moe_abi.py")],
                         cwd=ROOT, env=env, capture_output=True, text=True, timeout=1200)
    tail = (res.stdout + res.stderr)[-4000:]
    assert res.returncode == 0, tail
    assert "passed" in res.stdout and "ERROR: AddressSanitizer" not in tail and "runtime error" not in tail, tail
