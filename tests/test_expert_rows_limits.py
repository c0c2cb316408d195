"""Sizes of experts' rows that pass 2^31 - 1 are refused by every call that takes them: no call below gets past its argument
checks, whatever `rows` and the arrays hold."""
from __future__ import annotations

import ctypes

import pytest

import register_tiled_matrix_amd as rt
from register_tiled_matrix_amd._f8 import MatrixStruct, RowsStruct

DUMMY = 0x1000  # never dereferenced
TOO_MANY = [dict(tokens=1024, k=1, experts=1024, align=1 << 22), dict(tokens=2**31 - 1, k=1, experts=1, align=128),
            dict(tokens=2**30, k=4, experts=8, align=1), dict(tokens=2**31 - 1, k=2**31 - 1, experts=2**31 - 1, align=128)]


@pytest.fixture(scope="module")
def lib():
    import os

    if not os.path.exists(rt.lib_path()):
        from register_tiled_matrix_amd import build
        build.build()
    return rt.load()


def matrix(rows, cols, **kw):
    m = dict(codes=DUMMY, ld=max(cols, 1), scales=DUMMY, scale_row=1, scale_col=1, codes_stack=0, scales_stack=0, rows=rows, cols=cols, stack=1,
             type=0, block_rows=1)
    return MatrixStruct(**{**m, **kw})


@pytest.mark.parametrize("sizes", TOO_MANY, ids=lambda s: "x".join(map(str, s.values())))
@pytest.mark.parametrize("at", [None, DUMMY])
@pytest.mark.parametrize("rows", [-1, 0, 2**31 - 1])
def test_sizes_past_the_limit_are_refused(lib, sizes, at, rows):
    assert lib.regtile_expert_rows_size(*sizes.values()) == -1
    r = RowsStruct(slots=at, position=at, offsets=DUMMY, counts=DUMMY, rows=rows, **sizes)
    b, n = ctypes.byref, sizes["experts"]
    assert lib.regtile_order_experts(DUMMY, b(r), DUMMY, 2**40, None) == -2
    stack = matrix(300, 200, block_rows=128, stack=n, scale_col=3)
    for gather, a_rows in ((0, max(rows, 0)), (1, sizes["tokens"])):
        A = matrix(a_rows, 200)
        assert lib.regtile_gemm_f8_experts(b(r), gather, 1, 1.0, b(A), b(stack), 0.0, 1, DUMMY, 300, None, 0, None) == -1
        assert lib.regtile_gemm_f8_experts_workspace(b(r), gather, 1, b(A), b(stack), 1) == 0
    A = matrix(64, max(rows, 0))
    assert lib.regtile_gemm_f8_experts_dw(b(r), 1.0, b(A), b(A), 0.0, 0, DUMMY, 64, 4096, None, 0, None) == -1
    assert lib.regtile_gemm_f8_experts_dw_workspace(b(r), b(A), b(A), 0) == 0
    assert lib.regtile_combine_experts(b(r), 1, 8, DUMMY, 8, None, DUMMY, 8, None) == -1
    assert lib.regtile_combine_experts_grad(b(r), 1, 8, DUMMY, 8, DUMMY, 8, None, DUMMY, 8, None, None) == -1
