"""Which stream and device a norm, activation or few-row call runs on: a stream
of another device is refused before anything else is looked at, and the
tensors' device is current while the library runs."""
from __future__ import annotations

from types import SimpleNamespace

import pytest
import torch


def on(index):
    return SimpleNamespace(device=torch.device("cuda", index))


def calls(t):
    import gemm_pt_block_gb300 as mx

    return {
        "norm": lambda s: mx.mxfp4_rmsnorm_quantize(t, None, stream=s),
        "norm backward": lambda s: mx.mxfp4_rmsnorm_backward(t, t, None, t, stream=s),
        "swiglu": lambda s: mx.mxfp4_swiglu_quantize(t, t, stream=s),
        "swiglu backward": lambda s: mx.mxfp4_swiglu_backward(t, t, t, stream=s),
        "gemv": lambda s: mx.mxfp4_gemv(t, t, t, 1, 32, stream=s),
    }


@pytest.mark.parametrize("name", ["norm", "norm backward", "swiglu", "swiglu backward", "gemv"])
def test_a_stream_of_another_device_is_refused(name):
    with pytest.raises(ValueError, match="stream must be one of the tensors' device cuda:1"):
        calls(on(1))[name](on(0))


def test_every_entry_makes_the_tensors_device_current():
    """(What a second device would show, read from the source: each entry point
    holds the guard from where it knows the device.)"""
    import os
    import re

    import gemm_pt_block_gb300 as mx

    with open(os.path.join(os.path.dirname(mx.__file__), "csrc", "binding.cpp")) as f:
        text = f.read()
    entries = re.findall(r"^PyObject\* (\w+)\(PyObject\* const\* a\) \{\n(.*?)^\}", text, re.S | re.M)
    assert [e for e, _ in entries] == ["norm", "norm_backward", "swiglu", "swiglu_backward", "gemv"]
    for name, body in entries:
        guard, first = body.find("const OnDevice current("), min(
            i for i in (body.find("empty("), body.find("quantized("), body.find("call(")) if i >= 0)
        assert 0 <= guard < first, name


@pytest.mark.gpu
def test_a_stream_of_the_same_device_runs():
    import gemm_pt_block_gb300 as mx

    x = torch.randn((4, 64), device="cuda")
    want = mx.mxfp4_swiglu_quantize(x, x, y_dtype=torch.float32)[2]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = mx.mxfp4_swiglu_quantize(x, x, y_dtype=torch.float32, stream=side)[2]
    side.synchronize()
    assert torch.equal(got, want)
    assert mx.mxfp4_rmsnorm_quantize(x, None, y_dtype=torch.float32, stream=torch.cuda.default_stream())[2].shape == x.shape
