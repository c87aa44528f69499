"""Workspaces of the attention over the 8-bit cache: how many bytes a call asks
for, and that a kernel never sees one that the call did not ask for. The
library's own objects run on a runtime that launches nothing (no GPU needed);
what the first launch is given is read there."""
from __future__ import annotations

import ctypes
import os
import subprocess

import pytest

from test_cache_abi import G, call
from test_launch_errors import CUDA, HERE


@pytest.fixture(scope="module")
def L(tmp_path_factory):
    from gemm_pt_block_gb300 import binding
    from gemm_pt_block_gb300 import build as b

    b.build()
    tmp = tmp_path_factory.mktemp("fake")
    so, fields = str(tmp / "libmxfp4_args.so"), str(tmp / "launch_fields.o")
    fake = os.path.join(HERE, "fake_cudart")
    for cmd in ([b.nvcc(), *b.ARCH, "-std=c++17", "-Xcompiler", "-fPIC", "-c", os.path.join(fake, "launch_fields.cu"), "-o", fields],
                [os.environ.get("CXX", "g++"), "-O1", "-std=c++17", "-fPIC", "-shared", f"-I{CUDA}/include",
                 os.path.join(fake, "launch_args.cpp"), fields,
                 *[os.path.join(b.BUILD, u.replace(".cu", ".o")) for u in b.UNITS], "-Wl,-Bsymbolic", "-o", so]):
        r = subprocess.run(cmd, capture_output=True, text=True)
        assert r.returncode == 0, r.stdout + r.stderr
    lib = binding.load_library(so)
    lib.fake_workspace.restype = ctypes.c_void_p
    lib.fake_workspace_bytes.restype = ctypes.c_uint64
    return lib


# Tables of at most one unit of work (fewer tokens than 64 at 64 channels, 32 above), one row a sequence or several.
ONE_UNIT = [dict(P=16, max_pages=3, ld_table=3), dict(P=32, max_pages=1, ld_table=1), dict(max_pages=0, ld_table=0),
            dict(P=16, max_pages=1, ld_table=1, D=128, qh=128, qt=512, oh=128, ot=512),
            dict(P=16, max_pages=1, ld_table=1, D=256, qh=256, qt=1024, oh=256, ot=1024, starts=None, tokens=3),
            dict(P=16, max_pages=1, ld_table=1, sequences=60000)]


@pytest.mark.parametrize("kw", ONE_UNIT, ids=str)
def test_a_call_that_needs_none_uses_none(L, kw):
    assert call(L, "size", **kw) == 0
    for given in (dict(ws=None, ws_bytes=0), dict(ws=G, ws_bytes=0), dict(ws=G, ws_bytes=16)):
        L.fake_fail_at(-1)
        assert call(L, "attention", **kw, **given) == 0
        assert L.fake_launches() == 1
        assert L.fake_workspace() is None and L.fake_workspace_bytes() == 0


@pytest.mark.parametrize("kw", [dict(max_pages=1024, ld_table=1024), dict(P=16, max_pages=4, ld_table=4),
                                dict(max_pages=1024, ld_table=1024, window=9)], ids=str)
def test_a_call_that_needs_one_gets_it(L, kw):
    need = call(L, "size", **{k: v for k, v in kw.items() if k != "window"})
    assert need > 0
    L.fake_fail_at(-1)
    assert call(L, "attention", **kw, ws_bytes=need) == 0
    assert L.fake_launches() == 2
    assert L.fake_workspace() == G and 0 < L.fake_workspace_bytes() <= need
    if "window" not in kw:
        assert call(L, "attention", **kw, ws_bytes=need - 1) == 1
        assert call(L, "attention", **kw, ws=None, ws_bytes=0) == 1
