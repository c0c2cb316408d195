"""The workspace queries of the block-scaled products, without a GPU."""
from __future__ import annotations

import os

import pytest

import mx_reference as mx
import register_tiled_matrix_amd as rt


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not os.path.exists(rt.lib_path()):
        from register_tiled_matrix_amd import build
        build.build()
    rt.load()


def test_workspace_of_exactly_these_operands():
    """The query follows the kernel that takes the call: nothing where that one splits nothing, the parts of its
    own tiles where it does."""
    at = 0x10000

    def parts(M, N, K, order="nt", fmt=rt.MX_INT8, A=at, Q=at, S=at, lda=None, ldq=None, lds=None, ldc=None):
        ta, tb = int(order[0] == "t"), int(order[1] == "t")
        w, g = mx.widths(fmt, K if tb else N)
        n = rt.regtile_gemm_mx_workspace_ex(fmt, ta, tb, M, N, K, A, lda or (M if ta else K), Q, ldq or w, S, lds or g, ldc or N)
        assert n % (M * N * 4) == 0
        most = rt.regtile_gemm_mx_workspace(ta, tb, M, N, K, lda or (M if ta else K), ldc or N)
        assert n <= most
        return n // (M * N * 4), most // (M * N * 4)

    # rows of tokens: the token kernels split nothing; 33 to 64 unaligned ones run on 128-wide tiles
    assert parts(16, 8192, 8192) == (0, 0)
    assert parts(48, 2880, 4096) == (0, 8)
    assert parts(48, 2880, 2880) == (5, 5)           # 90 scale bytes a row
    assert parts(48, 2880, 4096, S=at + 1)[0] == 8
    # few rows in the other orders
    assert parts(16, 8192, 8192, "nn")[0] == 8 and parts(64, 4096, 4096, "nn")[0] == 8
    assert parts(64, 4096, 16384, "tn")[0] == 16
    # more rows: 64-wide tiles (256 of them here) split nothing, the 128-wide ones (64) of unaligned rows do
    for fmt in (rt.MX_FP4, rt.MX_INT8):
        assert parts(256, 4096, 4096, fmt=fmt)[0] == 0
        assert parts(256, 4096, 4096, fmt=fmt, Q=at + 8)[0] == 8
        assert parts(256, 4096, 2880, fmt=fmt)[0] == 5 and parts(128, 2880, 2880, fmt=fmt)[0] == 5
    # register-staged tiles: none
    assert parts(100, 1500, 2001) == (0, 0)
    assert parts(100, 1500, 2048, A=at + 8)[0] == 0
    # parts of an equal number of slabs: 65 of 128 k (fp4, codes in LDS) in 16 would leave 3 without any
    assert parts(512, 512, 65 * 128, fmt=rt.MX_FP4, Q=at + 16)[0] == parts(512, 512, 65 * 128, fmt=rt.MX_FP4)[0]
    assert parts(8, 512, 65 * 128, "nn")[0] == 15    # 130 of 64
    # parts of at least 512 k
    assert parts(512, 512, 1023, "tn")[1] == 0 and parts(512, 512, 1024, "tn")[0] == 2
    for wrong in ((2, 0, 1, 4), (0, 2, 1, 4), (0, 0, -1, 4), (0, 0, 1, 0)):
        assert rt.regtile_gemm_mx_workspace_ex(*wrong, 512, 8192, 0, 8192, 0, 8192, 0, 256, 512) == 0
