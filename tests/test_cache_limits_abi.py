"""The work that one call of the attention over the 8-bit cache may have, as
include/mxfp4.h counts it: calls just below the limit are taken, just above it
refused. (The library's own objects on a runtime that launches nothing.)"""
from __future__ import annotations

import pytest

from test_cache_abi import call
from test_launch_errors import L as fake  # noqa: F401  (a fixture)

LIMIT = 15 << 27


def units(tokens, sequences, heads, q_heads, D, P, max_pages, window=0):
    group, chunk = q_heads // heads, 64 if D == 64 else 32
    span = max_pages * P + 1
    if window:
        span = min(span, window + (group + 6) // group + 1 + chunk)
    tiles = heads * (tokens * group // 8 + sequences)
    return tiles * (-(-span // chunk) + (sequences > 1))


CASES = [
    # tokens, sequences, heads, q_heads, D, P, window
    (4096, 4096, 32, 32, 128, 64, 0), (1, 1, 32767, 32767, 128, 16, 0), (4096, 4096, 32, 32, 64, 64, 0),
    (4096, 4096, 8, 64, 128, 64, 0), (300000, 3, 8, 64, 96, 32, 0), (1000, 2, 4, 4, 256, 128, 0),
]


@pytest.mark.parametrize("tokens,sequences,heads,q_heads,D,P,window", CASES)
def test_the_widest_table_that_is_taken(fake, tokens, sequences, heads, q_heads, D, P, window):  # noqa: F811
    kw = dict(tokens=tokens, sequences=sequences, heads=heads, q_heads=q_heads, D=D, P=P, window=window, pages=1,
              kt=heads * D, kh=D, qt=q_heads * D, qh=D, ot=q_heads * D, oh=D)
    lo, hi = 0, (1 << 30) // P
    while lo + 1 < hi:                                      # the last width below the limit
        mid = (lo + hi) // 2
        lo, hi = (mid, hi) if units(tokens, sequences, heads, q_heads, D, P, mid, window) < LIMIT else (lo, mid)
    fake.fake_fail_at(-1)
    assert call(fake, "attention", max_pages=lo, ld_table=lo, **kw) == 0
    if hi < (1 << 30) // P:
        assert fake.fake_launches() == 2
        assert call(fake, "attention", max_pages=hi, ld_table=hi, **kw) == 2
        assert b"too many tokens" in fake.mxfp4_last_error()
        assert call(fake, "attention", max_pages=hi, ld_table=hi, **dict(kw, window=100)) == 0


@pytest.mark.parametrize("D,group", [(64, 1), (128, 1), (128, 7), (256, 8)])
def test_the_widest_window_that_is_taken(fake, D, group):  # noqa: F811
    tokens, sequences, heads = 1 << 16, 1000, 8
    kw = dict(tokens=tokens, sequences=sequences, heads=heads, q_heads=group * heads, D=D, P=128, pages=1, kt=heads * D, kh=D,
              qt=group * heads * D, qh=D, ot=group * heads * D, oh=D, max_pages=1 << 22, ld_table=1 << 22)
    lo, hi = 1, 1 << 29
    while lo + 1 < hi:
        mid = (lo + hi) // 2
        lo, hi = (mid, hi) if units(tokens, sequences, heads, group * heads, D, 128, 1 << 22, mid) < LIMIT else (lo, mid)
    fake.fake_fail_at(-1)
    assert call(fake, "attention", window=lo, **kw) == 0
    assert call(fake, "attention", window=hi, **kw) == 2


@pytest.mark.parametrize("status,scale,softcap", [
    (1, 1e30, 1e-30), (1, -1e30, 1e-30), (1, 1e10, 1e-21), (1, 2.0, 1e-30), (0, 0.5, 1e-30), (0, -0.5, 1e-30), (0, 1e30, 1.5), (0, 1e-30, 1e30),
    (0, 0.0, 1e-30), (0, 0.125, 50.0), (0, 1e30, 0.0), (1, 0.125, 1e-31), (1, 0.125, 2e30), (1, 2e30, 0.0), (1, -2e30, 0.0),
])
def test_scales_and_caps(fake, status, scale, softcap):  # noqa: F811
    fake.fake_fail_at(-1)
    assert call(fake, "attention", scale=scale, softcap=softcap) == status
    assert fake.fake_launches() == (2 if status == 0 else 0)


def test_the_case_of_many_sequences_of_one_row_a_head():
    """Nine times the work of the rows alone: at group 1 each sequence's tile holds one row of eight."""
    assert units(4096, 4096, 32, 32, 128, 64, 1 << 14) >= LIMIT
    assert 4096 * 32 * (1 << 20) // 256 < LIMIT
