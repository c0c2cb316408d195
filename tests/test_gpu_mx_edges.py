"""Block-scaled operands on the GPU where sizes, strides and streams are unusual: the widest rows,
the default stream's handle, products whose rows are few or unaligned, K in parts."""
from __future__ import annotations

import numpy as np
import pytest

import mx_reference as mx
import register_tiled_matrix_amd as rt
from gpu_util import announce

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    rt.load()
    yield
    torch.cuda.empty_cache()


@pytest.mark.parametrize("cols", [2**31 - 1, 2**31 - 7])
def test_dequantize_the_widest_rows(cols):
    """One row of as many columns as an int holds, where rounding up to whole units passes it: every value,
    and nothing written beside them."""
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB of free memory")
    guard = 4096
    groups = -(-cols // 32)
    gen = torch.Generator(device="cuda").manual_seed(cols)
    Q = torch.randint(0, 256, (1, cols), dtype=torch.uint8, device="cuda", generator=gen)
    S = torch.randint(100, 150, (1, groups), dtype=torch.uint8, device="cuda", generator=gen)
    full = torch.full((cols + 2 * guard,), 7.0, dtype=torch.bfloat16, device="cuda")
    X = full[guard:guard + cols].view(1, cols)
    announce(f"dequantize int8 to bf16, 1 x {cols}")
    rt.dequantize_mx(rt.MXMatrix(rt.MX_INT8, Q, S, cols), out=X)
    torch.cuda.synchronize()
    assert bool((full[:guard] == 7).all()) and bool((full[guard + cols:] == 7).all())
    step = 1 << 28
    for c in range(0, cols, step):
        n = min(step, cols - c)
        scale = torch.exp2(S[0, c // 32:-(-(c + n) // 32)].float() - 133)
        want = (Q[0, c:c + n].view(torch.int8).float() * scale.repeat_interleave(32)[:n]).to(torch.bfloat16)
        assert torch.equal(X[0, c:c + n], want), c
