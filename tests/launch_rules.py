"""The launch rules of the FP4 and MoE kernels, built by g++ from the headers
that the launchers use (``tests/host/launch_rules.cpp``)."""
from __future__ import annotations

import ctypes
import functools
import os
import subprocess
import tempfile

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "fine_grained_fp8_quantize_amd", "csrc")


@functools.lru_cache(maxsize=None)
def lib() -> ctypes.CDLL:
    with tempfile.TemporaryDirectory() as d:
        so = os.path.join(d, "launch_rules.so")
        made = subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-fPIC", "-shared", "-I", CSRC,
                               os.path.join(HERE, "host", "launch_rules.cpp"), "-o", so], capture_output=True, text=True)
        assert made.returncode == 0, made.stdout + made.stderr
        L = ctypes.CDLL(so)
    L.launch_fits.argtypes = [ctypes.c_int64, ctypes.c_int]
    L.moe_backward_tokens.restype = ctypes.c_int64
    return L


def shape(name: str, *args: int) -> tuple[int, int]:
    """Blocks and threads per block of launch rule ``name``."""
    blocks, threads = ctypes.c_int64(), ctypes.c_int()
    getattr(lib(), name)(*[ctypes.c_int64(a) for a in args], ctypes.byref(blocks), ctypes.byref(threads))
    return blocks.value, threads.value
