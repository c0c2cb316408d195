"""The block-scaled entry points without a GPU: argument checks of the C ABI and the binding, and
the reference encoder against itself."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import mx_reference as mx
import register_tiled_matrix_amd as rt

DUMMY = 0x1000  # never dereferenced: every call below returns before any HIP call


@pytest.fixture(scope="module", autouse=True)
def _built():
    import os

    if not os.path.exists(rt.lib_path()):
        from register_tiled_matrix_amd import build
        build.build()
    rt.load()


@pytest.mark.parametrize("fn", ["regtile_gemm_bf16_mx", "regtile_gemm_f16_mx"])
def test_gemm_arguments(fn):
    f = getattr(rt, fn)
    base = dict(format=rt.MX_FP4, ta=0, tb=1, M=4, N=5, K=65, alpha=1.0, A=DUMMY, lda=65, Q=DUMMY, ldq=33, S=DUMMY,
                lds=3, beta=0.0, C=DUMMY, ldc=5, work=0, work_bytes=0)

    def call(**kw):
        return f(*{**base, **kw}.values(), 0)

    assert call(format=2) == -1 and call(format=-1) == -1
    assert call(ta=2) == -2 and call(tb=-1) == -3
    assert call(M=-1) == -4 and call(N=-1) == -5 and call(K=-1) == -6
    assert call(A=0) == -8 and call(lda=64) == -9
    assert call(ta=1, lda=3) == -9          # A stored K x M
    assert call(Q=0) == -10
    assert call(ldq=32) == -11              # 65 columns of fp4: 33 bytes
    assert call(format=rt.MX_INT8, ldq=64) == -11
    assert call(S=0) == -12 and call(lds=2) == -13
    assert call(C=0) == -15 and call(ldc=4) == -16
    assert call(work=DUMMY + 8, work_bytes=64) == -17
    assert call(work=DUMMY, work_bytes=-1) == -18 and call(work_bytes=16) == -18
    # B stored K x N: its rows are N columns wide
    assert call(tb=0, ldq=2) == -11 and call(tb=0, N=33, ldc=33, ldq=17, lds=1) == -13
    # nothing is read or launched where there is no output
    assert call(M=0, A=0, Q=0, S=0, C=0) == 0 and rt.last_kernel() == "quick-return"
    assert call(N=0, A=0, Q=0, S=0, C=0, ldc=1) == 0
    # the largest sizes whose checks pass or fail without overflow
    big = 2**31 - 1
    assert call(K=big, lda=big, ldq=2**30 - 1) == -11
    assert call(K=big, lda=big, ldq=2**30, lds=2**26 - 1) == -13


def test_conversion_arguments():
    q = dict(format=rt.MX_INT8, dtype=1, rows=4, cols=33, X=DUMMY, ldx=33, Q=DUMMY, ldq=33, S=DUMMY, lds=2)
    d = dict(format=rt.MX_INT8, dtype=1, rows=4, cols=33, Q=DUMMY, ldq=33, S=DUMMY, lds=2, X=DUMMY, ldx=33)
    for f, base, at in ((rt.regtile_quantize_mx, q, {"X": 5, "ldx": 6, "Q": 7, "ldq": 8, "S": 9, "lds": 10}),
                        (rt.regtile_dequantize_mx, d, {"Q": 5, "ldq": 6, "S": 7, "lds": 8, "X": 9, "ldx": 10})):
        def call(**kw):
            return f(*{**base, **kw}.values(), 0)

        assert call(format=3) == -1 and call(dtype=3) == -2 and call(dtype=-1) == -2
        assert call(rows=-1) == -3 and call(cols=-1) == -4
        for name, pos in at.items():
            assert call(**{name: 0}) == -pos, name
        assert call(ldx=32) == -at["ldx"] and call(ldq=32) == -at["ldq"] and call(lds=1) == -at["lds"]
        assert call(format=rt.MX_FP4, ldq=16) == -at["ldq"]
        assert call(X=DUMMY + 1) == -at["X"] and call(dtype=0, X=DUMMY + 2) == -at["X"]
        assert call(rows=0, X=0, Q=0, S=0) == 0 and call(cols=0, X=0, Q=0, S=0) == 0
        assert rt.last_kernel() == "quick-return"


def _mat(fmt, rows, cols, **kw):
    w, g = mx.widths(fmt, cols)
    return rt.MXMatrix(fmt, torch.zeros(rows, w, dtype=torch.uint8), torch.zeros(rows, g, dtype=torch.uint8), cols, **kw)


def test_matrix_checks():
    m = _mat(rt.MX_FP4, 3, 33)
    assert m.shape == (3, 33) and m.t().shape == (33, 3) and m.t().t().shape == (3, 33)
    assert m.t().codes is m.codes and "transposed" in repr(m.t())
    z = torch.zeros
    u8 = torch.uint8
    with pytest.raises(ValueError, match="format"):
        rt.MXMatrix(2, z(3, 17, dtype=u8), z(3, 2, dtype=u8), 33)
    with pytest.raises(ValueError, match="bytes wide"):
        rt.MXMatrix(rt.MX_FP4, z(3, 16, dtype=u8), z(3, 2, dtype=u8), 33)
    with pytest.raises(ValueError, match="scales must be"):
        rt.MXMatrix(rt.MX_FP4, z(3, 17, dtype=u8), z(3, 1, dtype=u8), 33)
    with pytest.raises(ValueError, match="scales must be"):
        rt.MXMatrix(rt.MX_FP4, z(3, 17, dtype=u8), z(2, 2, dtype=u8), 33)
    with pytest.raises(ValueError, match="uint8"):
        rt.MXMatrix(rt.MX_FP4, z(3, 17, dtype=torch.int8), z(3, 2, dtype=u8), 33)
    with pytest.raises(ValueError, match="uint8"):
        rt.MXMatrix(rt.MX_INT8, z(3, 33, dtype=u8), z(3, 2), 33)
    with pytest.raises(ValueError, match="unit column stride"):
        rt.MXMatrix(rt.MX_INT8, z(33, 3, dtype=u8).t(), z(3, 2, dtype=u8), 33)
    with pytest.raises(ValueError, match="overlap"):
        rt.MXMatrix(rt.MX_INT8, z(1, 33, dtype=u8).expand(3, 33), z(3, 2, dtype=u8), 33)
    assert rt.MXMatrix(rt.MX_INT8, z(3, 33, dtype=torch.int8), z(3, 2, dtype=u8), 33).shape == (3, 33)


def test_binding_refuses_host_tensors_and_wrong_types():
    B = _mat(rt.MX_INT8, 4, 64)
    a = torch.zeros(2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="device"):
        rt.gemm_bf16_mx(a, B.t())
    with pytest.raises(ValueError, match="takes"):
        rt.gemm_f16_mx(a, B.t())
    with pytest.raises(ValueError, match="MXMatrix"):
        rt.gemm_bf16_mx(a, a.t())
    with pytest.raises(ValueError, match="device"):
        rt.quantize_mx(a)
    with pytest.raises(ValueError, match="device"):
        rt.dequantize_mx(B)
    with pytest.raises(ValueError, match="float32"):
        rt.quantize_mx(a.double())
    with pytest.raises(ValueError, match="format"):
        rt.quantize_mx(a, format=7)


def test_reference_encoder_on_known_groups():
    x = np.array([[6.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -0.24, 7.9, -7.0]])
    codes, E = mx.encode(x, mx.FP4)
    assert E.tolist() == [[127]]
    v = mx.decode(codes, E, mx.FP4, 11)[0]
    assert v.tolist() == [6.0, 0.0, 1.0, 1.0, 2.0, 2.0, 4.0, 4.0, 0.0, 6.0, -6.0]
    codes, E = mx.encode(np.array([[1.0, -1.9999, 2**-6, 2**-7, 3 * 2**-7, np.inf]])[:, :5], mx.INT8)
    assert E.tolist() == [[127]] and codes.view(np.int8).tolist() == [[64, -127, 1, 0, 2]]
    _, E = mx.encode(np.array([[1.0, np.inf]]), mx.INT8)
    assert E.tolist() == [[255]]
    _, E = mx.encode(np.zeros((1, 40)), mx.FP4)
    assert E.tolist() == [[0, 0]]


def test_workspace_sizes():
    f = rt.regtile_gemm_mx_workspace
    # few tiles and a long K: whole parts of M x N floats
    n = f(1, 0, 1024, 1024, 16384, 1024, 1024)
    assert n > 0 and n % (1024 * 1024 * 4) == 0
    assert f(0, 1, 8192, 8192, 8192, 8192, 8192) == 0   # the tiles fill the chip
    assert f(0, 1, 128, 128, 64, 64, 128) == 0          # nothing to split
    assert f(0, 1, 0, 128, 64, 64, 128) == 0 and f(2, 1, 128, 128, 64, 64, 128) == 0


def test_quantize_refuses_an_out_that_is_no_matrix():
    class OnDevice:  # what the checks look at, without a device
        dtype, is_cuda, device = torch.float32, True, torch.device("cuda", 0)
        shape = (2, 32)

        def dim(self):
            return 2

        def stride(self):
            return (32, 1)

    with pytest.raises(ValueError, match="out must be"):
        rt.quantize_mx(OnDevice(), rt.MX_INT8, out=torch.empty(2, 32, dtype=torch.uint8))
