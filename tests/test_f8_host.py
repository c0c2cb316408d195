"""8-bit float matrices and a mixture of experts without a GPU: argument checks of the C ABI and the binding,
and the reference against torch and against itself."""
from __future__ import annotations

import ctypes

import numpy as np
import pytest
import torch

import f8_reference as f8
import register_tiled_matrix_amd as rt
from register_tiled_matrix_amd._f8 import MatrixStruct, RowsStruct

DUMMY = 0x1000  # never dereferenced: every call below returns before any HIP call
TYPES = {f8.E4M3: torch.float8_e4m3fn, f8.E5M2: torch.float8_e5m2}


@pytest.fixture(scope="module")
def lib():
    import os

    if not os.path.exists(rt.lib_path()):
        from register_tiled_matrix_amd import build
        build.build()
    return rt.load()


def matrix(rows=4, cols=200, block_rows=1, **kw):
    m = dict(codes=DUMMY, ld=cols, scales=DUMMY, scale_row=1, scale_col=rows, codes_stack=0, scales_stack=0, rows=rows, cols=cols,
             stack=1, type=0, block_rows=block_rows)
    return MatrixStruct(**{**m, **kw})


BAD = [dict(rows=-1), dict(cols=-1), dict(type=2), dict(type=-1), dict(block_rows=2), dict(ld=199), dict(ld=2**31), dict(codes=0),
       dict(scales=0), dict(scales=DUMMY + 2), dict(scale_row=-1), dict(scale_col=-1), dict(stack=0), dict(codes_stack=-1)]


def test_conversion_arguments(lib):
    def q(Q=None, **kw):
        a = {**dict(dtype=1, transpose=0, rows=4, cols=200, X=DUMMY, ldx=200, index=0), **kw}
        return lib.regtile_quantize_f8(*a.values(), ctypes.byref(matrix() if Q is None else Q), 0)

    assert q(dtype=3) == -1 and q(dtype=-1) == -1 and q(transpose=2) == -2 and q(rows=-1) == -3 and q(cols=-1) == -4
    assert q(X=0) == -5 and q(X=DUMMY + 1) == -5 and q(dtype=0, X=DUMMY + 2) == -5 and q(ldx=199) == -6 and q(index=DUMMY + 2) == -7
    for bad in BAD:
        assert q(matrix(**bad)) == -8, bad
    assert q(matrix(cols=201)) == -8 and q(matrix(rows=5)) == -8                  # another shape than X's
    assert q(matrix(rows=200, cols=5, ld=5), transpose=1) == -8
    assert q(matrix(rows=200, cols=4, ld=4, block_rows=128), transpose=1) == -8   # blocks of 1 x 128 only
    assert q(matrix(rows=0), rows=0, X=0) == 0 and rt.last_kernel() == "quick-return"
    assert lib.regtile_quantize_f8(1, 0, 4, 200, DUMMY, 200, None, None, None) == -8

    def d(Q=None, dtype=1, X=DUMMY, ldx=200):
        return lib.regtile_dequantize_f8(ctypes.byref(matrix() if Q is None else Q), dtype, X, ldx, None)

    for bad in BAD:
        assert d(matrix(**bad)) == -1, bad
    assert d(dtype=3) == -2 and d(X=0) == -3 and d(X=DUMMY + 1) == -3 and d(ldx=199) == -4
    assert d(matrix(cols=0), X=0) == 0


def test_gemm_arguments(lib):
    W = matrix(rows=300, cols=200, block_rows=128, scale_col=3)

    def g(A=None, B=None, **kw):
        a = {**dict(ta=0, tb=1, alpha=1.0, A=ctypes.byref(matrix() if A is None else A), B=ctypes.byref(W if B is None else B), beta=0.0, dtype=0,
                    C=DUMMY, ldc=300, work=0, size=0), **kw}
        return lib.regtile_gemm_f8(*a.values(), 0)

    assert g(ta=2) == -1 and g(tb=-1) == -2
    for bad in BAD:
        assert g(matrix(**bad)) == -4, bad
        assert g(B=matrix(**{**dict(rows=300, block_rows=128), **bad})) == -5, bad
    assert g(ta=1, A=matrix(rows=200, cols=4)) == -4                   # scales of 1 x 128 across k
    assert g(tb=0, B=matrix(rows=200, cols=300, block_rows=1)) == -5
    assert g(B=matrix(rows=300, cols=199, block_rows=128)) == -5       # inner sizes
    assert g(B=matrix(rows=300, cols=200, type=5)) == -5
    assert g(dtype=3) == -7 and g(C=0) == -8 and g(C=DUMMY + 2) == -8 and g(dtype=1, C=DUMMY + 1) == -8 and g(ldc=299) == -9
    assert g(work=DUMMY + 8, size=64) == -10 and g(work=DUMMY, size=-1) == -11 and g(size=16) == -11
    assert g(A=matrix(rows=0), C=0) == 0 and rt.last_kernel() == "quick-return"
    # a null matrix
    assert lib.regtile_gemm_f8(0, 1, 1.0, None, ctypes.byref(W), 0.0, 0, DUMMY, 300, None, 0, None) == -4


def rows_struct(tokens=4, k=2, experts=3, align=128, **kw):
    r = dict(slots=DUMMY, position=DUMMY, offsets=DUMMY, counts=DUMMY, tokens=tokens, k=k, experts=experts, align=align,
             rows=f8.rows_size(tokens * k, experts, max(align, 1)))
    return RowsStruct(**{**r, **kw})


BAD_ROWS = [dict(tokens=-1), dict(k=0), dict(experts=0), dict(align=0), dict(rows=7), dict(slots=0), dict(position=0), dict(offsets=0),
            dict(counts=0)]


def test_experts_arguments(lib):
    R = rows_struct()
    n = R.rows
    b = ctypes.byref
    stack = matrix(rows=300, cols=200, block_rows=128, stack=3, codes_stack=60000, scales_stack=6)

    def g(r=R, gather=1, tb=1, A=matrix(rows=4), B=stack, dtype=1, C=DUMMY, ldc=300, work=None, size=0):
        return lib.regtile_gemm_f8_experts(b(r), gather, tb, 1.0, b(A), b(B), 0.0, dtype, C, ldc, work, size, None)

    def dw(r=R, A=matrix(rows=64, cols=n), B=matrix(rows=32, cols=n), dtype=0, C=DUMMY, ldc=32, stack=2048, work=None, size=0):
        return lib.regtile_gemm_f8_experts_dw(b(r), 1.0, b(A), b(B), 0.0, dtype, C, ldc, stack, work, size, None)

    for bad in BAD_ROWS:
        r = rows_struct(**bad)
        assert g(r) == -1 and dw(r) == -1 and lib.regtile_order_experts(DUMMY, b(r), None, 0, None) == -2, bad
        assert lib.regtile_combine_experts(b(r), 1, 8, DUMMY, 8, None, DUMMY, 8, None) == -1
        assert lib.regtile_combine_experts_grad(b(r), 1, 8, DUMMY, 8, DUMMY, 8, None, DUMMY, 8, None, None) == -1
    assert g(gather=2) == -2 and g(tb=3) == -3
    assert g(gather=0) == -5 and g(A=matrix(rows=n)) == -5                 # tokens with gather, rows without
    assert g(B=matrix(rows=300, block_rows=128, stack=2)) == -6 and g(B=matrix(rows=300, block_rows=128, cols=100, stack=3)) == -6
    assert g(tb=0, B=matrix(rows=200, cols=300, stack=3)) == -6
    assert g(dtype=4) == -8 and g(C=0) == -9 and g(ldc=299) == -10
    assert dw(rows_struct(align=64)) == -1 and dw(A=matrix(rows=64, cols=n - 1)) == -3 and dw(B=matrix(rows=32, cols=n + 1)) == -4
    assert dw(A=matrix(rows=64, cols=n, block_rows=128)) == -3 and dw(dtype=7) == -6 and dw(C=0) == -7 and dw(ldc=31) == -8
    assert g(work=DUMMY + 8, size=64) == -11 and g(work=DUMMY, size=-1) == -12 and g(size=16) == -12
    assert dw(work=DUMMY + 8, size=64) == -10 and dw(work=DUMMY, size=-1) == -11 and dw(size=16) == -11
    assert dw(stack=2047) == -9 and dw(stack=-1) == -9
    assert lib.regtile_order_experts(None, b(R), None, 0, None) == -1
    assert lib.regtile_order_experts(DUMMY, b(rows_struct(experts=1025)), None, 0, None) == -2
    big = rows_struct(tokens=5000, align=1)
    need = lib.regtile_order_experts_workspace(5000, 2, 3)
    assert need > 0 and lib.regtile_order_experts_workspace(4, 2, 3) == 0
    assert lib.regtile_order_experts(DUMMY, b(big), DUMMY + 4, need, None) == -3
    assert lib.regtile_order_experts(DUMMY, b(big), DUMMY, need - 1, None) == -4
    for args, want in ((dict(dtype=3), -2), (dict(n=-1), -3), (dict(Y=0), -4), (dict(ldy=7), -5), (dict(out=0), -7), (dict(ldo=7), -8)):
        a = {**dict(dtype=1, n=8, Y=DUMMY, ldy=8, w=0, out=DUMMY, ldo=8), **args}
        assert lib.regtile_combine_experts(b(R), *a.values(), None) == want, args
    for args, want in ((dict(dtype=3), -2), (dict(n=-1), -3), (dict(dout=0), -4), (dict(ldd=7), -5), (dict(Y=0), -6), (dict(ldy=7), -7),
                       (dict(dY=0), -9), (dict(lddy=7), -10)):
        a = {**dict(dtype=1, n=8, dout=DUMMY, ldd=8, Y=DUMMY, ldy=8, w=0, dY=DUMMY, lddy=8, dw=DUMMY), **args}
        assert lib.regtile_combine_experts_grad(b(R), *a.values(), None) == want, args


def test_route_arguments(lib):
    def f(**kw):
        a = {**dict(score=0, dtype=0, tokens=3, experts=16, k=4, groups=4, top=2, best=1, renorm=1, scale=1.0, x=DUMMY, ldl=16, bias=0,
                    chosen=DUMMY, w=DUMMY), **kw}
        return lib.regtile_route_experts(*a.values(), None)

    for args, want in ((dict(score=2), -1), (dict(dtype=3), -2), (dict(tokens=-1), -3), (dict(experts=0), -4), (dict(experts=1025, ldl=2000), -4),
                       (dict(k=0), -5), (dict(k=17), -5), (dict(experts=128, ldl=128, k=65), -5), (dict(groups=0), -6), (dict(groups=3), -6),
                       (dict(experts=130, ldl=130, groups=65), -6), (dict(top=0), -7), (dict(top=5), -7), (dict(best=3), -8), (dict(renorm=2), -9),
                       (dict(x=0), -11), (dict(x=DUMMY + 2), -11), (dict(ldl=15), -12), (dict(chosen=0), -14), (dict(w=0), -15)):
        assert f(**args) == want, args
    assert f(tokens=0, x=0, chosen=0, w=0) == 0

    def g(**kw):
        a = {**dict(score=0, dtype=0, tokens=3, experts=16, k=4, renorm=1, scale=1.0, x=DUMMY, ldl=16, chosen=DUMMY, dw=DUMMY, dx=DUMMY, ldd=16), **kw}
        return lib.regtile_route_experts_grad(*a.values(), None)

    for args, want in ((dict(score=2), -1), (dict(dtype=3), -2), (dict(tokens=-1), -3), (dict(experts=0), -4), (dict(k=17), -5), (dict(renorm=2), -6),
                       (dict(x=0), -8), (dict(ldl=15), -9), (dict(chosen=0), -10), (dict(dw=0), -11), (dict(dx=0), -12), (dict(ldd=15), -13)):
        assert g(**args) == want, args
    assert g(tokens=0, x=0, chosen=0, dw=0, dx=0) == 0


def test_rows_size():
    lib = rt.load()
    for tokens, k, experts, align in ((0, 1, 1, 1), (1, 1, 1, 128), (7, 3, 5, 1), (7, 3, 5, 128), (2, 2, 64, 128), (100000, 8, 256, 128)):
        assert lib.regtile_expert_rows_size(tokens, k, experts, align) == f8.rows_size(tokens * k, experts, align) == rt.expert_rows_size(
            tokens, k, experts, align)
    assert lib.regtile_expert_rows_size(2**30, 4, 8, 1) == -1 and lib.regtile_expert_rows_size(2**31 - 1, 1, 1, 128) == -1
    assert lib.regtile_expert_rows_size(-1, 1, 1, 1) == -1


def test_every_choice_fits_its_rows():
    rng = np.random.default_rng(0)
    for _ in range(200):
        T, k, E, align = int(rng.integers(1, 9)), int(rng.integers(1, 4)), int(rng.integers(1, 12)), int(rng.choice([1, 2, 5, 128]))
        c = rng.integers(-1, E, (T, k))
        slots, position, offsets, counts = f8.expert_rows(c, E, align)
        assert offsets[-1] <= slots.size and np.array_equal(np.sort(slots[slots >= 0]), np.flatnonzero(c.reshape(-1) >= 0))


def host_matrix(rows=4, cols=200, block_rows=1, kind=torch.float8_e4m3fn, **kw):
    n = -(-rows // block_rows)
    return rt.F8Matrix(torch.zeros(rows, cols, dtype=torch.uint8).view(kind), torch.ones(n, f8.blocks(cols)), block_rows, **kw)


def test_matrix_checks():
    m = host_matrix()
    assert m.shape == (4, 200) and m.t().shape == (200, 4) and m.t().t().shape == (4, 200) and "transposed" in repr(m.t())
    z, e = torch.zeros, torch.float8_e4m3fn
    s = rt.F8Matrix(z(3, 4, 200, dtype=torch.uint8).view(e), z(3, 1, 2), 128)
    assert s.shape == (3, 4, 200) and s.t().shape == (3, 200, 4)
    codes = z(4, 200, dtype=torch.uint8).view(e)
    for args, match in (((z(4, 200), z(4, 2)), "float8"), ((codes, z(4, 2), 64), "block_rows"), ((codes, z(4, 2).half()), "float32"),
                        ((codes, z(4, 1)), "scales must be"), ((codes, z(4, 2), 128), "scales must be"), ((codes, z(1, 4, 2)), "2-D"),
                        ((codes[0], z(2)), "2-D"), ((codes.t(), z(200, 1)), "row-major"),
                        ((codes[:1].expand(4, 200), z(4, 2)), "overlap")):
        with pytest.raises(ValueError, match=match):
            rt.F8Matrix(*args)


def test_binding_refusals():
    X = torch.zeros(4, 200)
    with pytest.raises(ValueError, match="device tensor"):
        rt.quantize_f8(X)
    with pytest.raises(ValueError, match="float32, bfloat16"):
        rt.quantize_f8(X.double())
    with pytest.raises(ValueError, match="dtype"):
        rt.quantize_f8(X, torch.float16)
    with pytest.raises(ValueError, match="device tensors"):
        rt.dequantize_f8(host_matrix())
    with pytest.raises(ValueError, match="device tensors"):
        rt.gemm_f8(host_matrix(), host_matrix(rows=300).t())
    with pytest.raises(ValueError, match="F8Matrix"):
        rt.gemm_f8(X, host_matrix())
    for logits, match in ((X, "device tensor"), (X.double(), "float32")):
        with pytest.raises(ValueError, match=match):
            rt.route_experts(logits, 2)
    with pytest.raises(ValueError, match="score"):
        rt.route_experts(X, 2, score=2)
    with pytest.raises(ValueError, match="device tensor"):
        rt.expert_rows(torch.zeros(4, 2, dtype=torch.int32), 8)
    i32 = dict(dtype=torch.int32)
    with pytest.raises(ValueError, match="slots"):
        rt.ExpertRows(torch.zeros(7, **i32), torch.zeros(4, 2, **i32), torch.zeros(9, **i32), torch.zeros(8, **i32))
    r = rt.ExpertRows(torch.zeros(8, **i32), torch.zeros(4, 2, **i32), torch.zeros(9, **i32), torch.zeros(8, **i32))
    assert r.rows == 8 and r.token_of_row().tolist() == [0] * 8
    with pytest.raises(ValueError, match="ExpertRows"):
        rt.combine_experts(X, None)


@pytest.mark.parametrize("kind", [f8.E4M3, f8.E5M2])
def test_reference_codes(kind):
    table = f8.decode_table(kind)
    assert np.array_equal(torch.arange(256, dtype=torch.uint8).view(TYPES[kind]).double().numpy(), table, equal_nan=True)
    finite = f8.finite_codes(kind)
    assert np.array_equal(f8.decode_table(kind)[f8.nearest_code(table[finite], kind)], table[finite])
    rng = np.random.default_rng(1)
    x = rng.standard_normal(20000) * np.exp2(rng.integers(-20, 10, 20000))
    x = np.clip(x, -f8.TOP[kind], f8.TOP[kind]).astype(np.float32)
    assert np.array_equal(torch.from_numpy(x).to(TYPES[kind]).view(torch.uint8).numpy(), f8.nearest_code(x.astype(np.float64), kind))


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("renormalize", [False, True])
def test_reference_gradient_is_the_differences(sigmoid, renormalize):
    """Central differences with h = 1e-5 are off by h^2 / 6 of the third derivative, some 1e-10 here, and by
    rounding over h, some 1e-11."""
    rng = np.random.default_rng(2)
    x, d = rng.standard_normal((3, 10)), rng.standard_normal((3, 4))
    chosen, _ = f8.route(x, 4, sigmoid=sigmoid)
    chosen[1, 3] = -1
    g = f8.route_grad(x, chosen, d, sigmoid, renormalize, 1.5)
    for t in range(3):
        for e in range(10):
            h = np.zeros_like(x)
            h[t, e] = 1e-5
            diff = (f8.route_loss(x + h, chosen, d, sigmoid, renormalize, 1.5) - f8.route_loss(x - h, chosen, d, sigmoid, renormalize, 1.5)) / 2e-5
            assert abs(diff - g[t, e]) < 1e-8
