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


KERNELS = ("rows", "tiles", "grouped tiles")


def gemm_form(m: int, n: int, scales16: bool = True) -> tuple[str, int, int]:
    """Kernel of a dense FP4 product, and its tile's parameters."""
    out = (ctypes.c_int * 3)()
    lib().fp4_gemm_form(ctypes.c_int64(m), ctypes.c_int64(n), int(scales16), out)
    return KERNELS[out[0]], out[1], out[2]


def grouped_form(m_total: int, n: int, groups: int, scales16: bool = True) -> tuple[str, int, int]:
    """Kernel of a grouped FP4 product, and its tile's parameters."""
    out = (ctypes.c_int * 3)()
    lib().fp4_grouped_form(ctypes.c_int64(m_total), ctypes.c_int64(n), ctypes.c_int64(groups), int(scales16), out)
    return KERNELS[out[0]], out[1], out[2]
