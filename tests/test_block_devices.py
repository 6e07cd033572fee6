"""Every entry point of the gated block, the weight-only products and the
optimizer launches on its tensors' GPU, whichever is current."""
from __future__ import annotations

import inspect

import pytest

from fine_grained_fp8_quantize_amd import _adamw, _gated, _gemv


@pytest.mark.parametrize("module,names", [
    (_gated, ("fp8_gated_gemm", "fp8_grouped_gated_gemm", "fp8_gated_backward")), (_gemv, ("_gemv",)),
    (_adamw, ("adamw_step",))])
def test_every_entry_point_goes_through_the_device_guard(module, names):
    for name in names:
        text = inspect.getsource(getattr(module, name))
        assert "st = _call(" in text and "_raw_stream" not in text, name
