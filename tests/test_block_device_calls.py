"""The gated, weight-only and optimizer calls make their C calls with their
tensors' GPU as the current device and on the stream they were given, whichever
is current: each entry point called, with a library that notes it."""
from __future__ import annotations

import contextlib

import pytest
import torch

import fine_grained_fp8_quantize_amd as fq
from fine_grained_fp8_quantize_amd import _adamw, _gated, _gemv

DEV = 3
BF, F32, U8, I32 = torch.bfloat16, torch.float32, torch.uint8, torch.int32


class Library:
    """Functions of any name; those that launch end with the stream."""

    def __init__(self, at):
        self.at, self.calls = at, []

    def __getattr__(self, name):
        if name.endswith("_bytes"):
            return lambda *args: 0
        return lambda *args: self.calls.append((name, self.at[0], args[-1])) or 0


def _z(*shape, dt=BF):
    return torch.zeros(shape, dtype=dt)


def _gated_gemm(**kw):
    return fq.fp8_gated_gemm(_z(4, 128, dt=U8), _z(1, 4, dt=F32), _z(2, 128, 128, dt=U8), _z(2, 1, 1, dt=F32), out=_z(4, 128), **kw)


def _grouped(**kw):
    return fq.fp8_grouped_gated_gemm(_z(2, dt=I32), None, _z(128, 128, dt=U8), _z(1, 128, dt=F32), _z(1, 2, 128, 128, dt=U8),
                                     _z(1, 2, 1, 1, dt=F32), out=_z(128, 128), **kw)


def _backward(**kw):
    return fq.fp8_gated_backward(_z(4, 8), _z(4, 16), out_dtype=BF, out=_z(4, 16), **kw)


def _gemv_call(**kw):
    return fq.fp4_gemv_mx(_z(2, 128), _z(1, 1, 1024, dt=U8), _z(1, 1, 64, dt=I32), out=_z(2, 16), **kw)


def _gated_gemv(**kw):
    return fq.fp4_gated_gemv_mx(_z(2, 128), _z(2, 1, 1, 1024, dt=U8), _z(2, 1, 1, 64, dt=I32), out=_z(2, 16), **kw)


def _step(**kw):
    t = [[_z(4, dt=F32)] for _ in range(4)]
    return fq.adamw_step(fq.adamw_plan(*t[:3]), t[3], 1, 1e-3, **kw)


@pytest.mark.parametrize("call,name", [(_gated_gemm, "fp8_gated_gemm"), (_grouped, "fp8_grouped_gated_gemm"),
                                       (_backward, "fp8_gated_backward"), (_gemv_call, "fp4_gemv_mx"),
                                       (_gated_gemv, "fp4_gated_gemv_mx"), (_step, "adamw_step")])
@pytest.mark.parametrize("current", [0, DEV])
def test_launches_on_the_tensors_gpu(monkeypatch, call, name, current):
    at = [current]
    library = Library(at)

    @contextlib.contextmanager
    def device(d):
        before, at[0] = at[0], d
        yield
        at[0] = before

    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: at[0])
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 100 + d)
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(_adamw, "_device_of", lambda t: DEV)
    for module in (_adamw, _gated, _gemv):
        monkeypatch.setattr(module, "_on_gpu", lambda *ts: DEV)
        monkeypatch.setattr(module, "_library", lambda: library)
    call()
    call(stream=type("Stream", (), {"cuda_stream": 77})())
    assert library.calls == [(name, DEV, 100 + DEV), (name, DEV, 77)] and at[0] == current
