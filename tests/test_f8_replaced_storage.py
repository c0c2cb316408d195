"""Matrices and experts' rows describe the tensors that they hold at each call: one whose storage is replaced between two calls
(as when weights are moved out and back, or loaded anew) is read where it is then."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import f8_reference as f8
import register_tiled_matrix_amd as rt
from register_tiled_matrix_amd._f8 import MatrixStruct, RowsStruct

E4 = torch.float8_e4m3fn


def codes(rows, cols, device="cpu"):
    return torch.randint(0, 100, (rows, cols), dtype=torch.uint8, device=device).view(E4)


def described(m):
    c = MatrixStruct.from_address(m._at)
    return c.codes, c.ld, c.scales, c.scale_row, c.scale_col, c.rows, c.cols, c.stack


def test_matrix():
    m = rt.F8Matrix(codes(4, 200), torch.ones(4, 2))
    turned, old = m.t(), (m.codes.data, m.scales.data)
    first = described(m)
    assert first[0] == old[0].data_ptr() and first[2] == old[1].data_ptr() and described(m) == first
    m.codes.data = torch.zeros(4, 208, dtype=torch.uint8).view(E4)[:, :200]
    m.scales.data = torch.ones(2, 4).t()
    for v in (m, turned):
        assert described(v) == (m.codes.data_ptr(), 208, m.scales.data_ptr(), 1, 4, 4, 200, 1)
    m.codes, m.scales = old
    assert described(m) == first and turned.t().codes is turned.codes
    m.scales.data = torch.ones(4, 2)
    assert described(m)[2] == m.scales.data_ptr()


@pytest.mark.parametrize("what,match", [(dict(codes=codes(5, 200)), "scales must be|shape"), (dict(codes=codes(4, 201)), "shape"),
                                        (dict(scales=torch.ones(5, 2)), "scales must be"), (dict(scales=torch.ones(4, 2).half()), "float32"),
                                        (dict(codes=torch.ones(4, 200)), "float8"), (dict(scales=torch.ones(4, 2, device="meta")), "devices")])
def test_what_no_longer_fits_is_refused(what, match):
    m = rt.F8Matrix(codes(4, 200), torch.ones(4, 2))
    for name, t in what.items():
        setattr(m, name, t)
    with pytest.raises(ValueError, match=match):
        m._at
    two = rt.F8Matrix(codes(4, 200), torch.ones(4, 2))
    two.codes, two.scales = codes(6, 300), torch.ones(6, 3)  # whole, but another matrix than its views say
    with pytest.raises(ValueError, match="shape"):
        two._at


def test_rows():
    i32 = dict(dtype=torch.int32)
    parts = [torch.zeros(n, **i32) for n in ((8,), (4, 2), (9,), (8,))]
    r = rt.ExpertRows(*parts)

    def at():
        c = RowsStruct.from_address(r._at)
        return [c.slots, c.position, c.offsets, c.counts]

    assert at() == [t.data_ptr() for t in parts]
    keep = [t.data for t in parts]
    for t in parts:
        t.data = torch.zeros_like(t)
        assert at() == [t.data_ptr() for t in parts]
    assert len(keep) == 4
    parts[0].data = torch.zeros(9, **i32)
    with pytest.raises(ValueError, match="slots"):
        r._at


@pytest.mark.gpu
def test_products_read_the_new_storage():
    x, w = rt.F8Matrix(codes(20, 300, "cuda"), torch.rand(20, 3, device="cuda")), rt.F8Matrix(codes(40, 300, "cuda"), torch.rand(1, 3, device="cuda"), 128)
    view = w.t()
    before = rt.gemm_f8(x, view)
    old = w.codes.data, w.scales.data  # (they stay, so that nothing reads freed memory whichever is read)
    w.codes.data, w.scales.data = codes(40, 300, "cuda"), torch.rand(1, 3, device="cuda")
    after = rt.gemm_f8(x, view)
    want = rt.gemm_f8(x, rt.F8Matrix(w.codes.data, w.scales.data, 128).t())
    assert torch.equal(after, want) and not torch.equal(after, before)
    w.codes.data, w.scales.data = old
    assert torch.equal(rt.gemm_f8(x, view), before)
    out = rt.F8Matrix(codes(20, 300, "cuda"), torch.zeros(20, 3, device="cuda"))
    held = out.codes.data
    was = held.view(torch.uint8).clone()
    out.codes.data = torch.empty_like(held)
    X = torch.randn(20, 300, device="cuda")
    rt.quantize_f8(X, out=out)
    assert torch.equal(held.view(torch.uint8), was)
    q = rt.quantize_f8(X)
    assert torch.equal(out.codes.view(torch.uint8), q.codes.view(torch.uint8))
    assert torch.equal(rt.dequantize_f8(out, torch.float32), rt.dequantize_f8(q, torch.float32))


@pytest.mark.gpu
def test_experts_read_the_new_rows():
    chosen = torch.randint(0, 5, (30, 2), dtype=torch.int32, device="cuda")
    other = torch.randint(0, 5, (30, 2), dtype=torch.int32, device="cuda")
    r, s = rt.expert_rows(chosen, 5), rt.expert_rows(other, 5)
    Y = torch.randn(r.rows, 64, device="cuda")
    keep = r.position.data
    a, b = rt.combine_experts(Y, r), rt.combine_experts(Y, s)
    r.position.data = s.position
    assert torch.equal(rt.combine_experts(Y, r), b) and not torch.equal(a, b)
    assert np.array_equal(f8.expert_rows(chosen.cpu().numpy(), 5, 1)[1], keep.cpu().numpy())
