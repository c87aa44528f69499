"""The norm, activation and few-row calls from several host threads at once,
each on its own stream: the same bits as one after the other. In a fresh
process, so that the concurrent calls are its first ones (kernel attributes and
the table of the library's functions are filled under contention)."""
from __future__ import annotations

import os
import subprocess
import sys
import threading

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def work(mx, torch, i):
    g = torch.Generator(device="cuda").manual_seed(i)
    x = torch.randn((24 + i, 4096), device="cuda", generator=g).to(torch.bfloat16)
    q = torch.randint(0, 256, (4096, 2048), dtype=torch.uint8, device="cuda", generator=g)
    out = []
    for nv in (False, True):
        s = torch.randint(110, 126, (4096, 4096 // (16 if nv else 32)), dtype=torch.uint8, device="cuda", generator=g)
        w = mx.QuantParams(mx.BLOCK_1X16 if nv else mx.BLOCK_1X32)
        ws = torch.empty(1 << 22, dtype=torch.uint8, device="cuda")
        for rows in (1, 12, 24):
            for space in (False, ws):
                out.append(mx.mxfp4_gemv(x[:rows], q, s, 4096, 4096, w, workspace=space))
    p = mx.QuantParams(elem_format=mx.FORMAT_E4M3)
    one = torch.ones(4096, device="cuda")
    q8, s8, y, h, rstd = mx.mxfp4_rmsnorm_quantize(x, one, p, residual=x, y_dtype=torch.float32, with_rstd=True)
    out += [q8, s8, y, h, rstd, *mx.mxfp4_rmsnorm_backward(x, h, one, rstd)]
    out += [t for t in mx.mxfp4_swiglu_quantize(x, h, p, y_dtype=torch.bfloat16)]
    return out + list(mx.mxfp4_swiglu_backward(x, x, h))


def main() -> int:
    import torch

    import gemm_pt_block_gb300 as mx

    n = 4
    torch.empty(1, device="cuda")
    results, errors = [None] * n, []
    start = threading.Barrier(n)

    def run(i):
        try:
            s = torch.cuda.Stream()
            start.wait()
            with torch.cuda.stream(s):
                for _ in range(5):
                    results[i] = work(mx, torch, i)
            s.synchronize()
        except Exception as e:  # reported below
            errors.append(f"thread {i}: {e!r}")

    threads = [threading.Thread(target=run, args=(i,)) for i in range(n)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    if errors:
        print("\n".join(errors))
        return 1
    for i in range(n):
        for k, (a, b) in enumerate(zip(results[i], work(mx, torch, i))):
            if not torch.equal(a, b):
                print(f"thread {i}, output {k} differs from the serial run")
                return 1
    print("OK" if mx.device_status() == 0 else "device error")
    return 0


@pytest.mark.gpu
def test_concurrent_threads_match_serial():
    env = dict(os.environ, PYTHONPATH=os.pathsep.join([ROOT, os.environ.get("PYTHONPATH", "")]))
    r = subprocess.run([sys.executable, os.path.abspath(__file__)], capture_output=True, text=True,
                       timeout=300, env=env, cwd=ROOT)
    assert r.returncode == 0 and "OK" in r.stdout, r.stdout + r.stderr


if __name__ == "__main__":
    sys.exit(main())
