"""Host-side refusals of the calls on the 8-bit cache (no GPU needed: every
call fails validation before any pointer is used), and failed launches."""
from __future__ import annotations

import ctypes
from types import SimpleNamespace

import pytest
import torch

from test_launch_errors import ERR_CUDA, L as fake  # noqa: F401  (a fixture: the library on a runtime that launches nothing)

G = 1 << 20
OFF = G + 2
OFF8 = G + 8


@pytest.fixture(scope="module")
def L():
    from gemm_pt_block_gb300 import build as b

    b.build()
    import gemm_pt_block_gb300 as mx

    return mx.lib()


def call(L, what, codes=G, scales=G, pages=9, heads=2, P=32, D=64, table=G, ld_table=4, max_pages=4, lens=G, starts=G,
         sequences=3, tokens=5, k=G, kd=0, kt=128, kh=64, v=G, vd=0, vt=128, vh=64, q=G, qd=0, qt=256, qh=64, q_heads=4,
         scale=0.1, softcap=0.0, slopes=None, window=0, out=G, od=0, ot=256, oh=64, lse=None, ws=G, ws_bytes=1 << 40,
         cache=True, batch=True, params=True):
    from gemm_pt_block_gb300 import binding as B

    R = ctypes.byref
    c = R(B._CCache(codes, scales, pages, heads, P, D)) if cache else None
    b = R(B._CBatch(table, ld_table, max_pages, lens, starts, sequences, tokens)) if batch else None
    if what in ("append", "read"):
        return getattr(L, "mxfp8_cache_" + what)(c, b, R(B._CHeads(k, kd, kt, kh)) if k != "none" else None,
                                                 R(B._CHeads(v, vd, vt, vh)), None)
    p = R(B._CAttention(scale, softcap, slopes, window)) if params else None
    if what == "size":
        return L.mxfp8_cache_attention_workspace_size(c, b, q_heads)
    return L.mxfp8_cache_attention(c, b, R(B._CHeads(q, qd, qt, qh)), q_heads, p, R(B._CHeads(out, od, ot, oh)), lse, ws,
                                   ws_bytes, None)


COMMON = [
    (1, dict(cache=False)), (1, dict(batch=False)), (2, dict(P=8)), (2, dict(P=48)), (2, dict(P=256)), (2, dict(D=32)),
    (2, dict(D=80)), (2, dict(D=512)), (2, dict(heads=0)), (2, dict(heads=-1)), (2, dict(heads=32768)),
    (2, dict(pages=-1)), (2, dict(pages=1 << 29)), (2, dict(sequences=-1)), (2, dict(sequences=65536)),
    (2, dict(tokens=-1)), (2, dict(tokens=1 << 24)), (2, dict(max_pages=-1)), (2, dict(max_pages=1 << 25, ld_table=1 << 25)),
    (2, dict(ld_table=3)), (2, dict(ld_table=(1 << 40) + 1)), (1, dict(codes=None)), (1, dict(scales=None)),
    (1, dict(table=None)), (3, dict(codes=OFF8)), (3, dict(table=OFF)), (3, dict(starts=OFF)),
]


@pytest.mark.parametrize("what", ["append", "read", "attention"])
@pytest.mark.parametrize("status,kw", COMMON, ids=str)
def test_refusals_of_caches_and_batches(L, what, status, kw):
    assert call(L, what, **kw) == status
    assert len(L.mxfp4_last_error()) > 0


@pytest.mark.parametrize("what", ["append", "read"])
@pytest.mark.parametrize("status,kw", [
    (1, dict(k="none")), (1, dict(k=None)), (1, dict(v=None)), (1, dict(kd=2)), (1, dict(vd=1)), (2, dict(kh=56)),
    (2, dict(kt=-128)), (2, dict(vt=(1 << 40) + 8)), (2, dict(vh=(1 << 40) + 8)), (3, dict(k=OFF8)), (3, dict(v=OFF8)),
    (3, dict(kt=132)), (3, dict(vh=68, vt=256)),
], ids=str)
def test_refusals_of_keys_and_values(L, what, status, kw):
    assert call(L, what, **kw) == status


def test_refusals_of_one_call(L):
    assert call(L, "append", lens=None) == 1 and call(L, "append", lens=OFF) == 3
    assert call(L, "append", starts=None) == 2                       # 5 rows of 3 sequences
    assert call(L, "read", starts=None, tokens=3) == 1
    assert call(L, "read", kt=64) == 2                                # rows over one another
    assert call(L, "read", kt=64, kh=256) == 2                        # heads over rows: 5 rows of 64 need 320


@pytest.mark.parametrize("status,kw", [
    (1, dict(lens=None)), (2, dict(starts=None)), (1, dict(params=False)), (2, dict(q_heads=0)), (2, dict(q_heads=3)),
    (2, dict(q_heads=65536)), (2, dict(q_heads=1024, tokens=1 << 21)), (1, dict(q=None)), (1, dict(out=None)), (1, dict(qd=1)), (1, dict(od=2)),
    (1, dict(scale=float("nan"))), (1, dict(scale=float("inf"))), (1, dict(softcap=-1.0)), (1, dict(softcap=float("nan"))),
    (1, dict(softcap=float("inf"))), (1, dict(window=-1)), (3, dict(slopes=OFF)), (3, dict(lse=OFF)), (3, dict(ws=OFF8)),
    (2, dict(qh=32)), (2, dict(qt=-8)), (3, dict(qt=260)), (3, dict(q=OFF8)), (2, dict(ot=128)), (2, dict(ot=0)),
    (3, dict(oh=68, ot=512)), (3, dict(out=OFF8)),
], ids=str)
def test_refusals_of_attention(L, status, kw):
    assert call(L, "attention", **kw) == status


def test_workspace_size(L):
    assert call(L, "size", codes=None, scales=None, table=None, lens=None) == call(L, "size")
    for kw in (dict(P=8), dict(q_heads=3), dict(sequences=-1), dict(cache=False), dict(heads=0)):
        assert call(L, "size", **kw) == 0


def test_attention_needs_its_workspace(L):
    need = call(L, "size", max_pages=1024, ld_table=1024)
    if need:
        assert call(L, "attention", max_pages=1024, ld_table=1024, ws_bytes=need - 1) == 1
        assert call(L, "attention", max_pages=1024, ld_table=1024, ws=None, ws_bytes=0) == 1


LAUNCHES = [("append", {}), ("append", dict(kd=1, vd=1, starts=None, tokens=3)), ("read", {}), ("read", dict(kd=1, vd=1)),
            ("attention", {}), ("attention", dict(max_pages=4096, ld_table=4096, od=1, D=256, kt=512)),
            ("attention", dict(q_heads=64, qt=4096, ot=4096, max_pages=300, ld_table=300)),
            ("attention", dict(D=96, P=16, qh=96, qt=384, oh=96, ot=384, slopes=G, window=9, softcap=2.0, lse=G))]


@pytest.mark.parametrize("what,kw", LAUNCHES, ids=str)
def test_every_failed_launch_is_reported(fake, what, kw):  # noqa: F811
    if kw.get("D") == 256:
        kw = dict(kw, qh=256, qt=1024, oh=256, ot=1024)
    fake.fake_fail_at(-1)
    assert call(fake, what, **kw) == 0
    launches = fake.fake_launches()
    assert launches >= 1
    for n in range(launches):
        fake.fake_fail_at(n)
        assert call(fake, what, **kw) == ERR_CUDA, f"launch {n} failed unnoticed"
        assert fake.fake_launches() == n + 1, "launched on after a failure"


@pytest.mark.parametrize("what", ["append", "read", "attention"])
def test_nothing_to_do_launches_nothing(fake, what):  # noqa: F811
    fake.fake_fail_at(-1)
    for kw in (dict(tokens=0), dict(sequences=0), dict(tokens=0, sequences=0, starts=G)):
        assert call(fake, what, **kw) == 0
    assert fake.fake_launches() == 0


def test_a_stream_of_another_device_is_refused():
    import gemm_pt_block_gb300 as mx

    t = SimpleNamespace(device=torch.device("cuda", 1))
    s = SimpleNamespace(device=torch.device("cuda", 0))
    for f in (lambda: mx.mxfp8_cache_append(t, t, t, t, t, t, stream=s), lambda: mx.mxfp8_cache_read(t, t, t, t, 1, stream=s),
              lambda: mx.mxfp8_cache_attention(t, t, t, t, t, stream=s)):
        with pytest.raises(ValueError, match="stream must be one of the tensors' device cuda:1"):
            f()


def test_every_entry_makes_the_tensors_device_current():
    """(Read from the source: each entry holds the guard before it allocates or calls.)"""
    import os
    import re

    import gemm_pt_block_gb300 as mx

    with open(os.path.join(os.path.dirname(mx.__file__), "csrc", "cache_binding.cpp")) as f:
        text = f.read()
    entries = re.findall(r"^PyObject\* (\w+)\(PyObject\* const\* a\) \{\n(.*?)^\}", text, re.S | re.M)
    assert [e for e, _ in entries] == ["append", "read", "attention"]
    for name, body in entries:
        first = min(i for i in (body.find("empty("), body.find("call(")) if i >= 0)
        assert 0 <= body.find("const OnDevice current(") < first, name


def test_cpu_tensors_are_refused():
    import gemm_pt_block_gb300 as mx

    codes, scales = torch.zeros((2, 2, 1, 16, 64), dtype=torch.uint8), torch.zeros((2, 2, 1), dtype=torch.uint8)
    table, lens = torch.zeros((1, 2), dtype=torch.int32), torch.ones(1, dtype=torch.int32)
    k = torch.zeros((1, 1, 64))
    with pytest.raises(ValueError, match="codes must be a CUDA tensor"):
        mx.mxfp8_cache_append(k, k, codes, scales, table, lens)
    with pytest.raises(ValueError, match="codes must be a CUDA tensor"):
        mx.mxfp8_cache_read(codes, scales, table, lens, 1)
    with pytest.raises(ValueError, match="codes must be a CUDA tensor"):
        mx.mxfp8_cache_attention(k.bfloat16(), codes, scales, table, lens)
    with pytest.raises(TypeError, match="must be a tensor"):
        mx.mxfp8_cache_append(k, k, None, scales, table, lens)


def test_a_failed_load_says_why(monkeypatch):
    import sys

    import gemm_pt_block_gb300 as mx
    from gemm_pt_block_gb300 import binding

    monkeypatch.setattr(binding, "_cache_ext", None)
    monkeypatch.delattr(mx, "_cache_binding", raising=False)
    monkeypatch.setitem(sys.modules, "gemm_pt_block_gb300._cache_binding", None)
    with pytest.raises(RuntimeError, match="does not load .*_cache_binding.*build"):
        mx.mxfp8_cache_read(torch.zeros(1), torch.zeros(1), torch.zeros(1), torch.zeros(1), 1)


def test_the_block_refuses_sizes_off_the_tiles():
    import gemm_pt_block_gb300 as mx

    for kw in (dict(dim=200, heads=2, head_dim=128), dict(dim=256, heads=3, kv_heads=2), dict(dim=256, heads=3, head_dim=64),
               dict(dim=256, heads=2, kv_heads=0, head_dim=64)):
        with pytest.raises(ValueError):
            mx.Mxfp4Attention(**kw)
    block = mx.Mxfp4Attention(256, 4, 2, 64)
    with pytest.raises(RuntimeError, match="quantize_weights"):
        block.decode(torch.zeros(1, 256), None, None, None)
    assert set(block.state_dict()) == {"norm", "qkv.weight", "out.weight"}


def test_waits_are_whole_warps():
    """The attention kernel's waits, read from the source: every loop that waits on a barrier has a limit, and
    code of whole warps goes on or leaves together."""
    import os
    import re

    import gemm_pt_block_gb300 as mx

    with open(os.path.join(os.path.dirname(mx.__file__), "csrc", "cache.cu")) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    tries = [m.start() for m in re.finditer(r"mbar_try_wait(_sleep)?\(", text)]
    assert len(tries) == 5
    for at in tries:
        around = text[max(0, at - 400):at + 700]
        assert "kWaitLimitNs" in around
    for name in ("wait_bar_warp", "wait_bars"):
        body = text[text.index(f"bool {name}("):]
        body = body[:body.index("\n}")]
        assert "__all_sync" in body and "kWaitLimitNs" in body


def test_a_window_bounds_the_work(fake):  # noqa: F811
    """A table that would be too wide without one: its workspace is known, and suffices."""
    fake.fake_fail_at(-1)
    wide = dict(tokens=1 << 20, max_pages=1 << 20, ld_table=1 << 20)
    need = call(fake, "size", **wide)
    assert need > 0 and call(fake, "attention", **wide) == 2
    assert call(fake, "attention", window=100, ws_bytes=need, **wide) == 0
