"""What an 8-bit float product makes of a workspace that holds only a part of what it asks for."""
from __future__ import annotations

import ctypes

import pytest
import torch

import f8_reference as f8
import register_tiled_matrix_amd as rt
from register_tiled_matrix_amd._f8 import MatrixStruct

E4 = torch.float8_e4m3fn
DTYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}


def tight(gen, rows, cols, block_rows=1):
    """Rows of codes next to each other, scales of a row next to each other."""
    codes = torch.randint(0, 120, (rows, cols), dtype=torch.uint8, device="cuda", generator=gen)
    scales = torch.rand(-(-rows // block_rows), f8.blocks(cols), device="cuda", generator=gen)
    return rt.F8Matrix(codes.view(E4), scales, block_rows)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("sb", [1, 128])
def test_copies_without_turned_scales(dtype, sb):
    """Rows that need copies, scales whose rows are apart, 2^37 operations: with room for the copies only, the scales stay as
    they are. The same kernel, and the same bits: it reads the same scales from elsewhere."""
    gen = torch.Generator(device="cuda").manual_seed(9)
    M, N, K = 4100, 4090, 4101
    assert 2 * M * N * K >= 2**37
    A, B = tight(gen, M, K), tight(gen, N, K, sb).t()
    lib = rt.load()
    need = lib.regtile_gemm_f8_workspace(0, 1, A._at, B._at, DTYPES[dtype], N)
    copies = (M + N) * ((K + 15) // 16 * 16)
    assert need > copies
    work = torch.empty(need, dtype=torch.uint8, device="cuda")
    out, names = [], []
    for size in (need, need - 16, copies, copies - 16):
        C = torch.empty(M, N, device="cuda", dtype=dtype)
        assert lib.regtile_gemm_f8(0, 1, 1.0, A._at, B._at, 0.0, DTYPES[dtype], C.data_ptr(), N, work.data_ptr(), size,
                                   torch.cuda.current_stream().cuda_stream) == 0
        out.append(C)
        names.append(rt.last_kernel())
    assert names[0].startswith("f8_tile") and names[1:3] == names[:1] * 2 and names[3].startswith("f8_any"), names
    assert torch.equal(out[0], out[1]) and torch.equal(out[0], out[2])


def test_the_size_is_the_sum_of_its_parts():
    """Copies, turned scales: no GPU needed for the question."""
    lib = rt.load()

    def m(rows, cols, ld, block_rows=1, by_rows=True):
        blocks, n = f8.blocks(cols), -(-rows // block_rows)
        return MatrixStruct(codes=0x1000, ld=ld, scales=0x1000, scale_row=blocks if by_rows else 1, scale_col=1 if by_rows else n,
                            codes_stack=0, scales_stack=0, rows=rows, cols=cols, stack=1, type=0, block_rows=block_rows)

    def need(a, b):
        return lib.regtile_gemm_f8_workspace(0, 1, ctypes.byref(a), ctypes.byref(b), 1, a.rows)

    n, copy, turned = 4101, 4101 * 4112, (4101 * 33 * 4 + 15) // 16 * 16
    assert need(m(n, n, 4112, by_rows=False), m(n, n, 4112, 128)) == 0
    assert need(m(n, n, 4112), m(n, n, 4112, 128)) == turned
    assert need(m(n, n, 4112), m(n, n, 4112)) == 2 * turned
    assert need(m(n, n, n, by_rows=False), m(n, n, n, 128)) == 2 * copy
    assert need(m(n, n, n), m(n, n, n)) == 2 * copy + 2 * turned


def test_parts_of_k_are_the_exact_products_and_those_of_few_tiles():
    """Aligned products ask for a workspace for parts of k only: those of up to 512 tiles of 64 x 64, and past that those with
    an fp32 C of up to 256 tiles of 128 x 128 (half of what the chip holds). M from 65 on: few rows take none."""
    lib = rt.load()

    def need(M, N, K, dtype):
        a, b = (MatrixStruct(codes=0x1000, ld=K, scales=0x1000, scale_row=1, scale_col=n, codes_stack=0, scales_stack=0, rows=n, cols=K, stack=1,
                             type=0, block_rows=1) for n in (M, N))
        return lib.regtile_gemm_f8_workspace(0, 1, ctypes.byref(a), ctypes.byref(b), dtype, N)

    for M in (65, 100, 128, 300, 1000, 1408, 1500, 2048, 2100, 5000):
        for N in (64, 129, 700, 1024, 1500, 2000, 2048, 4096):
            tiles64, tiles128 = f8.blocks(2 * M) * f8.blocks(2 * N), f8.blocks(M) * f8.blocks(N)
            for K in (128, 1024, 2048, 4096, 8192):
                part, n = M * N * 4, K // 128
                for dtype in (0, 1):
                    parts = (min(256 // tiles64, n // 8) if tiles64 <= 512 else min(512 // tiles128, n // 8) if dtype == 0 else 1)
                    if tiles64 <= 512 and parts == 2 and dtype == 1 and n < 32:
                        parts = 1
                    assert need(M, N, K, dtype) == (parts * part if parts > 1 else 0), (M, N, K, dtype)
