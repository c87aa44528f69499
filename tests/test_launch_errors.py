"""A launch that fails is reported by the call that made it, whichever of its
kernels it was. The library's own objects run on a runtime that launches
nothing and lets a chosen launch fail (no GPU needed)."""
from __future__ import annotations

import ctypes
import os
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CUDA = os.environ.get("CUDA_HOME", "/usr/local/cuda")
G = ctypes.c_void_p(1 << 20)
NONE, BF16, F32 = None, 0, 1
ERR_CUDA = 5


@pytest.fixture(scope="module")
def L(tmp_path_factory):
    from gemm_pt_block_gb300 import binding
    from gemm_pt_block_gb300 import build as b

    b.build()
    so = str(tmp_path_factory.mktemp("fake") / "libmxfp4_fake.so")
    cmd = [os.environ.get("CXX", "g++"), "-O1", "-std=c++17", "-fPIC", "-shared", f"-I{CUDA}/include",
           os.path.join(HERE, "fake_cudart", "fake_cudart.cpp"),
           *[os.path.join(b.BUILD, u.replace(".cu", ".o")) for u in b.UNITS], "-Wl,-Bsymbolic", "-o", so]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr
    return binding.load_library(so)


def norm_gradient(L, rows, cols, dt, dw, dh=False):
    ws = L.mxfp4_rmsnorm_backward_workspace_size(rows, cols)
    return L.mxfp4_rmsnorm_backward(G, dt, cols, G, dt, cols, G, F32, G, G if dh else NONE, cols, rows, cols, G, cols,
                                    G if dw else NONE, G if dw else NONE, ws, NONE)


def norm(L, rows, cols, dt):
    return L.mxfp4_rmsnorm_quantize(G, dt, rows, cols, cols, NONE, cols, G, F32, 1e-6, NONE, cols, G, dt, cols, G, NONE,
                                    NONE, NONE, NONE)


def swiglu(L, rows, cols, dt):
    return L.mxfp4_swiglu_quantize(G, cols, G, cols, dt, rows, cols, G, dt, cols, NONE, NONE, NONE, NONE)


def swiglu_gradient(L, rows, cols, dt):
    return L.mxfp4_swiglu_backward(G, dt, cols, G, cols, G, cols, dt, rows, cols, G, cols, G, cols, NONE)


def gemv(L, M, N, K, nv, ws):
    block = 3 if nv else 0
    n = L.mxfp4_gemv_workspace_size(0, block, M, N, K) if ws else 0
    return L.mxfp4_gemv_ex(G, 0, K, NONE, G, G, block, 0, 0, M, N, K, G, F32, N, G if ws else NONE, n, NONE)


CALLS = [
    (1, norm_gradient, (5, 64, BF16, False)), (2, norm_gradient, (5, 64, BF16, True)),
    (2, norm_gradient, (9, 512, F32, True, True)),
    (1, norm_gradient, (300, 4096, BF16, False)), (2, norm_gradient, (300, 4096, BF16, True, True)),
    (2, norm_gradient, (700, 8192, F32, True)),
    (1, norm_gradient, (3, 32768, F32, False, True)), (3, norm_gradient, (3, 32768, F32, True, True)),
    (1, norm, (7, 96, BF16)), (1, norm, (200, 8192, F32)), (1, norm, (2, 65536, F32)),
    (1, swiglu, (40, 1056, BF16)), (1, swiglu_gradient, (40, 1056, F32)),
    (1, gemv, (1, 1000, 1024, False, False)), (1, gemv, (20, 200, 544, True, False)),
    (2, gemv, (12, 1024, 1024, False, True)), (2, gemv, (12, 1024, 1024, True, True)), (1, gemv, (12, 96, 544, False, False)),
]


@pytest.mark.parametrize("launches,call,args", CALLS)
def test_every_failed_launch_is_reported(L, launches, call, args):
    L.fake_fail_at(-1)
    assert call(L, *args) == 0
    assert L.fake_launches() == launches
    for n in range(launches):
        L.fake_fail_at(n)
        assert call(L, *args) == ERR_CUDA, f"launch {n} failed unnoticed"
        assert L.fake_launches() == n + 1, "launched on after a failure"
        assert b"fake error" in L.mxfp4_last_error()


def test_an_earlier_callers_error_is_not_this_calls(L):
    L.fake_fail_at(0)
    assert norm(L, 7, 96, BF16) == ERR_CUDA
    L.fake_fail_at(-1)
    assert norm(L, 7, 96, BF16) == 0
