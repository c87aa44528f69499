"""When the Python extension is built anew, and what is said when it does not
load (no GPU needed)."""
from __future__ import annotations

import os
import sys

import pytest
import torch


def test_the_extension_is_stale_for_another_pytorch(monkeypatch, tmp_path):
    from gemm_pt_block_gb300 import build as b

    so, stamp, src = (str(tmp_path / n) for n in ("x.so", "for.txt", "x.cpp"))
    monkeypatch.setattr(b, "BINDING", so)
    monkeypatch.setattr(b, "BINDING_FOR", stamp)
    for i, name in enumerate((src, so)):
        open(name, "w").close()
        os.utime(name, (1000 + i, 1000 + i))
    assert b._binding_stale([src])                          # by no one knows what
    with open(stamp, "w") as f:
        f.write(b._built_for())
    assert not b._binding_stale([src])
    monkeypatch.setattr(torch, "__version__", "1.0.0")
    assert b._binding_stale([src])
    monkeypatch.undo()
    monkeypatch.setattr(b, "BINDING", so)
    monkeypatch.setattr(b, "BINDING_FOR", stamp)
    os.utime(src, (2000, 2000))
    assert b._binding_stale([src])
    os.remove(so)
    os.utime(src, (1000, 1000))
    assert b._binding_stale([src])


def test_build_leaves_the_extension_for_this_pytorch():
    from gemm_pt_block_gb300 import build as b

    b.build()
    with open(b.BINDING_FOR) as f:
        assert f.read() == b._built_for() and torch.__version__ in b._built_for()


def test_a_failed_load_says_why(monkeypatch):
    import gemm_pt_block_gb300 as mx
    from gemm_pt_block_gb300 import binding

    monkeypatch.setattr(binding, "_ext", None)
    monkeypatch.delattr(mx, "_binding", raising=False)
    monkeypatch.setitem(sys.modules, "gemm_pt_block_gb300._binding", None)
    with pytest.raises(RuntimeError, match="does not load .*_binding.*build"):
        mx.mxfp4_swiglu_quantize(torch.zeros(1, 32), torch.zeros(1, 32))
