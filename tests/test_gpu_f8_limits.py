"""8-bit float products of more columns, and of more experts, than one kind of launch counts."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import f8_reference as f8
import register_tiled_matrix_amd as rt
from f8_gpu_util import assert_close

pytestmark = pytest.mark.gpu
E4 = torch.float8_e4m3fn


@pytest.mark.parametrize("M,K", [(1, 16), (3, 16), (1, 5)])
def test_few_rows_times_many_columns(M, K):
    """2^27 + 40 columns: 2^23 workgroups of 512 threads and 16 columns would pass 2^32 threads."""
    N = 2**27 + 40
    if torch.cuda.mem_get_info()[0] < 12 << 30:
        pytest.skip("needs 12 GB of free memory")
    gen = torch.Generator(device="cuda").manual_seed(M + K)
    w = torch.randint(0, 100, (N, K), dtype=torch.uint8, device="cuda", generator=gen)
    W = rt.F8Matrix(w.view(E4), torch.rand(f8.blocks(N), 1, device="cuda", generator=gen), 128)
    x = torch.randint(0, 100, (M, K), dtype=torch.uint8, device="cuda", generator=gen)
    X = rt.F8Matrix(x.view(E4), torch.rand(M, 1, device="cuda", generator=gen))
    C = rt.gemm_f8(X, W.t(), dtype=torch.bfloat16)
    at = torch.cat([torch.arange(0, 300), torch.arange(2**27 - 100, N), torch.randint(0, N, (2000,))]).cuda()
    va = f8.decode(x.cpu().numpy(), X.scales.cpu().numpy(), f8.E4M3)
    vb = f8.decode_table(f8.E4M3)[w[at].cpu().numpy()] * W.scales[at // 128].double().cpu().numpy()
    assert_close(C[:, at], va @ vb.T, np.abs(va) @ np.abs(vb).T, rt.last_kernel())


@pytest.mark.parametrize("K", [200, 208])
def test_more_experts_than_a_grid_has_layers(K):
    """70000 experts that share one matrix (a stack with stride 0), most of them without a row; rows that are aligned or not."""
    E, T, N = 70000, 40, 130
    rng = np.random.default_rng(1)
    experts = np.sort(rng.choice(E, T, replace=False))
    experts[-1] = E - 1
    counts = np.zeros(E, np.int32)
    counts[experts] = 1
    gpu = lambda a: torch.from_numpy(np.ascontiguousarray(a)).int().cuda()
    r = rt.ExpertRows(gpu(np.arange(T)), gpu(np.arange(T)[:, None]), gpu(np.r_[0, np.cumsum(counts)]), gpu(counts))
    w = torch.randint(0, 100, (1, N, K), dtype=torch.uint8, device="cuda").view(E4).expand(E, N, K)
    s = torch.rand(1, f8.blocks(N), f8.blocks(K), device="cuda").expand(E, -1, -1)
    x = rt.F8Matrix(torch.randint(0, 100, (T, K), dtype=torch.uint8, device="cuda").view(E4), torch.rand(T, f8.blocks(K), device="cuda"))
    C = rt.gemm_f8_experts(x, rt.F8Matrix(w, s, 128).t(), r)
    one = rt.F8Matrix(w[0], s[0], 128)
    va = f8.decode(x.codes.view(torch.uint8).cpu().numpy(), x.scales.cpu().numpy(), f8.E4M3)
    vb = f8.decode(one.codes.view(torch.uint8).cpu().numpy(), one.scales.cpu().numpy(), f8.E4M3, 128)
    assert_close(C, va @ vb.T, np.abs(va) @ np.abs(vb).T, rt.last_kernel())
