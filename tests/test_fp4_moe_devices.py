"""The FP4 and MoE calls launch on their tensors' GPU, also where another one is
the current device: the default stream has the same handle on every GPU, and a
launch on it goes to the current device."""
from __future__ import annotations

import contextlib
import inspect

import pytest
import torch

from fine_grained_fp8_quantize_amd import _moe, _mx4


@pytest.mark.parametrize("dev,current", [(0, 0), (1, 0), (0, 3), (2, 2)])
@pytest.mark.parametrize("given", [False, True])
def test_the_device_of_a_launch(monkeypatch, dev, current, given):
    at = [current]

    @contextlib.contextmanager
    def device(d):
        before, at[0] = at[0], d
        yield
        at[0] = before

    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: at[0])
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 0)
    monkeypatch.setattr(torch.cuda, "device", device)
    stream = type("Stream", (), {"cuda_stream": 77})() if given else None
    calls = []

    def fn(*args):
        calls.append((at[0], args))
        return 5

    assert _mx4._call(fn, dev, stream, 1, 2) == 5
    assert calls == [(dev, (1, 2, 77 if given else 0))] and at[0] == current


def test_every_entry_point_goes_through_it():
    for module, names in ((_mx4, ("fp4_quantize_mx", "fp4_quantize_mx_scatter", "fp4_dequantize_mx", "fp4_gemm_mx",
                                  "fp4_grouped_gemm_mx")),
                          (_moe, ("moe_dispatch", "moe_balance_loss", "moe_balance_loss_backward"))):
        for name in names:
            text = inspect.getsource(getattr(module, name))
            assert "st = _call(" in text and "_raw_stream" not in text, name
