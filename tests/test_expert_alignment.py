"""Arrays of 32-bit numbers that do not begin at a multiple of 4 bytes are refused, as scales and row numbers are."""
from __future__ import annotations

import ctypes

import pytest

import register_tiled_matrix_amd as rt
from register_tiled_matrix_amd._f8 import RowsStruct

AT, OFF = 0x1000, 0x1002  # never dereferenced


@pytest.fixture(scope="module")
def lib():
    import os

    if not os.path.exists(rt.lib_path()):
        from register_tiled_matrix_amd import build
        build.build()
    return rt.load()


def rows(**kw):
    return ctypes.byref(RowsStruct(**{**dict(slots=AT, position=AT, offsets=AT, counts=AT, tokens=4, k=2, experts=3, align=1, rows=8), **kw}))


@pytest.mark.parametrize("part", ["slots", "position", "offsets", "counts"])
def test_rows(lib, part):
    r = rows(**{part: OFF})
    assert lib.regtile_order_experts(AT, r, None, 0, None) == -2
    assert lib.regtile_combine_experts(r, 1, 8, AT, 8, None, AT, 8, None) == -1
    assert lib.regtile_combine_experts_grad(r, 1, 8, AT, 8, AT, 8, None, AT, 8, None, None) == -1


def test_arguments(lib):
    assert lib.regtile_order_experts(OFF, rows(), None, 0, None) == -1
    route = dict(score=0, dtype=1, tokens=3, experts=16, k=4, groups=1, top=1, best=1, renorm=1, scale=1.0, x=AT, ldl=16, bias=0, chosen=AT, w=AT)
    for name, want in (("bias", -13), ("chosen", -14), ("w", -15)):
        assert lib.regtile_route_experts(*{**route, name: OFF}.values(), None) == want
    grad = dict(score=0, dtype=1, tokens=3, experts=16, k=4, renorm=1, scale=1.0, x=AT, ldl=16, chosen=AT, dw=AT, dx=AT, ldd=16)
    for name, want in (("chosen", -10), ("dw", -11)):
        assert lib.regtile_route_experts_grad(*{**grad, name: OFF}.values(), None) == want
    assert lib.regtile_combine_experts(rows(), 1, 8, AT, 8, OFF, AT, 8, None) == -6
    assert lib.regtile_combine_experts_grad(rows(), 1, 8, AT, 8, AT, 8, OFF, AT, 8, AT, None) == -8
    assert lib.regtile_combine_experts_grad(rows(), 1, 8, AT, 8, AT, 8, AT, AT, 8, OFF, None) == -11
