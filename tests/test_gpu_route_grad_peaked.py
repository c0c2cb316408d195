"""The router's gradient where one expert is nearly certain: it is then small beside the terms that it is the difference of, and
is held to a limit relative to itself.

The 64-bit values below come without that difference: a softmax's row sums to 1, so p_c (d_c - sum_e p_e d_e) is
p_c sum_e p_e (d_c - d_e), where c's own term, the one with the large p, is 0; a sigmoid's 1 - s is 1 / (1 + exp(x)). What is left
are rounding errors of 64-bit sums, some (experts + 10) 2^-53 of the sum of their terms' magnitudes (2^-40 allows for 1024
experts and each term's own roundings), and the rounding of the output, half a step of its type. Softmax without
renormalising takes the probabilities of experts that were not chosen from fp32 exponentials of x - top in fp32: that
difference is rounded, by 2^-24 of itself, which moves the exponential by as much times |x - top|, and the exponential is right
to a step, 2^-23. A gradient is a product of two of those sums at most (p_e dot / total): each is right to as much of itself."""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

import f8_reference as f8
import register_tiled_matrix_amd as rt

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def gradient(logits, chosen, dweights, sigmoid, renormalize, scale):
    """(gradient, sum of its terms' magnitudes), token by token; a repeated choice counts as often as it is made."""
    g, mag = np.zeros(logits.shape), np.zeros(logits.shape)
    for t, x in enumerate(logits.astype(np.float64)):
        c = chosen[t][chosen[t] >= 0]
        d = dweights[t].astype(np.float64)[chosen[t] >= 0]
        e = np.exp(x - x.max())
        terms = {}
        if not sigmoid and not renormalize:
            p = e / math.fsum(e)
            D = np.zeros(x.size)
            np.add.at(D, c, d)
            for i in range(x.size):
                terms[i] = list(p[i] * p * (D[i] - D)) if i in c else [-p[i] * p[j] * D[j] for j in set(c)]
        else:
            s, rest = 1 / (1 + np.exp(-x)), 1 / (1 + np.exp(x))
            w = (s if sigmoid else e)[c]
            if renormalize:
                w = w / math.fsum(w)
            for j, i in enumerate(c):
                mine = w[j] * (w * (d[j] - d) if renormalize else d[j:j + 1]) * (rest[i] if sigmoid else 1.0)
                terms.setdefault(int(i), []).extend(mine)
        for i, v in terms.items():
            g[t, i], mag[t, i] = scale * math.fsum(v), abs(scale) * math.fsum(np.abs(v))
    return g, mag


def check(x, chosen, dw, dtype, sigmoid, renormalize, scale):
    logits = torch.from_numpy(x).to(DTYPES[dtype])
    ref, mag = gradient(logits.float().numpy(), chosen, dw, sigmoid, renormalize, scale)
    got = rt.route_experts_grad(logits.cuda(), torch.from_numpy(chosen).cuda(), torch.from_numpy(dw).cuda(),
                                score=rt.SCORE_SIGMOID if sigmoid else rt.SCORE_SOFTMAX, renormalize=renormalize, scale=scale)
    info = torch.finfo(DTYPES[dtype])
    # (fp32: rounded to fp32 once; 16 bits: once more. Half a step of the subnormal numbers, where it is smaller than they are)
    near = 2.0**-40 * mag
    fp32 = 0.0
    if not sigmoid and not renormalize:
        xs = logits.double().numpy()
        fp32 = 2 * 1.01 * (2.0**-23 + 2.0**-24 * (xs.max(1) - xs.min(1)))[:, None] * mag
    limit = near + fp32 + (2.0**-24 + (info.eps / 2 if dtype != "f32" else 0.0)) * 1.01 * (np.abs(ref) + near + fp32) + info.smallest_normal * info.eps
    err = np.abs(got.double().cpu().numpy() - ref)
    assert (err <= limit).all(), (err / limit).max()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("renormalize", [False, True])
@pytest.mark.parametrize("experts,k", [(7, 1), (64, 1), (64, 6), (65, 1), (256, 1), (256, 8), (1000, 1), (1024, 64)])
def test_one_expert_ahead(experts, k, renormalize, sigmoid, dtype):
    rng = np.random.default_rng(experts * 100 + k)
    x = rng.standard_normal((40, experts)).astype(np.float32)
    ahead = np.repeat([4.0, 8, 12, 16, 18, 20, 30, 45], 5)
    x[np.arange(40), rng.integers(0, experts, 40)] += ahead.astype(np.float32)
    x = torch.from_numpy(x).to(DTYPES[dtype]).float().numpy()
    chosen, _ = f8.route(x, k, sigmoid=sigmoid)
    dw = rng.standard_normal((40, k)).astype(np.float32)
    check(x, chosen, dw, dtype, sigmoid, renormalize, 2.5)


@pytest.mark.gpu
@pytest.mark.parametrize("renormalize", [False, True])
@pytest.mark.parametrize("sigmoid", [False, True])
def test_repeated_and_missing_choices(sigmoid, renormalize):
    rng = np.random.default_rng(5)
    x = rng.standard_normal((30, 70)).astype(np.float32) * 3
    chosen = rng.integers(0, 70, (30, 5)).astype(np.int32)
    chosen[:, 3] = chosen[:, 1]          # twice
    chosen[:10, 4] = chosen[:10, 1]      # three times
    chosen[10:20, 0] = -1                # nobody
    chosen[3] = chosen[3, 0]             # only one expert, five times
    x[np.arange(30), chosen[:, 1]] += np.linspace(0, 20, 30).astype(np.float32)
    dw = rng.standard_normal((30, 5)).astype(np.float32)
    dw[:, 3] = -dw[:, 1] * np.float32(1 + 2.0**-20)  # whose gradients nearly cancel
    check(x, chosen, dw, "f32", sigmoid, renormalize, 1.0)


@pytest.mark.parametrize("renormalize", [False, True])
@pytest.mark.parametrize("sigmoid", [False, True])
def test_the_formula_is_the_jacobians(sigmoid, renormalize):
    """Against the full Jacobian, where nothing cancels: some experts 2^-53 of the largest gradient."""
    rng = np.random.default_rng(6)
    x, dw = rng.standard_normal((4, 12)), rng.standard_normal((4, 3)).astype(np.float32)
    chosen = rng.integers(0, 12, (4, 3)).astype(np.int32)
    chosen[2, 1] = chosen[2, 0]
    g, mag = gradient(x, chosen, dw, sigmoid, renormalize, 1.5)
    assert np.abs(g - f8.route_grad(x, chosen, dw, sigmoid, renormalize, 1.5)).max() <= 2.0**-45 * mag.max()
