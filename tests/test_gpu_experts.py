"""A mixture of experts on the GPU: the router, the order of rows, the experts' products and their combination
against 64-bit references, their gradients, edges, graphs, and all of them together as a layer."""
from __future__ import annotations

import numpy as np
import pytest

import f8_reference as f8
import register_tiled_matrix_amd as rt
from gpu_util import announce

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
from f8_gpu_util import DTYPES, TYPES, assert_close, device_codes, device_matrix, device_scales, random_matrix  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    rt.load()
    yield


def gpu(x, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(x)).cuda()
    return t if dtype is None else t.to(dtype)


# ---- routing -------------------------------------------------------------------------------
ROUTES = [  # experts, k, groups, top_groups, group_best
    (1, 1, 1, 1, 1), (2, 2, 1, 1, 1), (7, 3, 1, 1, 1), (64, 8, 1, 1, 1), (64, 64, 1, 1, 1), (65, 6, 5, 2, 1), (128, 8, 8, 3, 2), (160, 6, 8, 3, 1),
    (200, 7, 4, 2, 2), (256, 8, 8, 4, 2), (300, 10, 3, 3, 1), (512, 8, 64, 9, 2), (600, 33, 2, 1, 1), (1024, 10, 8, 1, 2), (1024, 4, 64, 64, 1), (8, 4, 8, 2, 2)]


def weights_close(got, want, what):
    """fp32 results of 64-bit arithmetic: half a step, and as much again for a different order of sums (softmax without
    renormalising sums fp32 exponentials, each off by 2 steps at most, over its experts)."""
    got, what = got.cpu().double().numpy(), what
    assert np.array_equal(np.isnan(got), np.isnan(want)), what
    err = np.abs(got - want)[~np.isnan(want)]
    assert (err <= 4 * 2.0**-23 * np.abs(want)[~np.isnan(want)] + 1e-37).all(), f"{what}: {err.max()}"


@pytest.mark.parametrize("E,k,groups,top_groups,best", ROUTES)
@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("with_bias", [False, True])
def test_route(E, k, groups, top_groups, best, sigmoid, with_bias):
    k = min(k, E // groups * top_groups) if E > 1 else k
    rng = np.random.default_rng(E + k)
    for dtype, T, renorm, scale in (("f32", 67, True, 1.0), ("bf16", 33, False, 2.5), ("f16", 5, True, 2.5), ("f32", 1, False, 1.0)):
        x = torch.from_numpy(rng.standard_normal((T, E)) * 2).to(DTYPES[dtype])
        bias = (rng.standard_normal(E) * 0.1).astype(np.float32) if with_bias else None
        want = f8.route(x.double().numpy(), k, bias, sigmoid, groups, top_groups, best, renorm, scale)
        announce(f"route {E} {k} {groups} {top_groups} {best} {dtype} {T} sigmoid {sigmoid} bias {with_bias}")
        e, w = rt.route_experts(x.cuda(), k, bias=None if bias is None else gpu(bias), score=int(sigmoid), groups=groups,
                                top_groups=top_groups, group_best=best, renormalize=renorm, scale=scale)
        assert np.array_equal(e.cpu().numpy(), want[0])
        weights_close(w, want[1], "weights")


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("groups,top_groups,best", [(1, 1, 1), (4, 2, 1), (4, 2, 2)])
def test_route_ties_masks_and_bad_rows(sigmoid, with_bias, groups, top_groups, best):
    """Ties go to the lowest number; -inf is never chosen; rows with nothing left, NaN or +inf are as documented."""
    E, k = 96, 7
    rng = np.random.default_rng(10)
    x = rng.integers(-2, 3, (40, E)).astype(np.float64)  # many equal values, and -0
    x[3] = 0.0
    x[3, ::2] = -0.0
    x[4] = -np.inf
    x[5] = -np.inf
    x[5, [90, 2, 50]] = 1.0, 1.0, -3.0
    x[6, 11] = np.nan
    x[7, 95] = np.inf
    x[8] = np.nan
    x[9] = np.finfo(np.float32).min
    x[10] = -1e4  # sigmoids that are 0 in 64 bits
    x[11, 10:] = -np.inf
    x[12, ::3] = -np.inf
    x[13, 0] = 3e38
    x[14] = np.linspace(-600, 0, E)
    bias = rng.integers(-1, 2, E).astype(np.float32) * 0.25 if with_bias else None
    if with_bias:
        bias[[5, 60]] = -np.inf, np.nan  # closed
    for renorm in (True, False):
        want = f8.route(x.astype(np.float32), k, bias, sigmoid, groups, top_groups, best, renorm)
        e, w = rt.route_experts(gpu(x, torch.float32), k, bias=None if bias is None else gpu(bias), score=int(sigmoid), groups=groups,
                                top_groups=top_groups, group_best=best, renormalize=renorm)
        assert np.array_equal(e.cpu().numpy(), want[0])
        weights_close(w, want[1], "weights")


@pytest.mark.parametrize("sigmoid", [False, True])
def test_route_tells_values_apart_that_32_bits_do_not(sigmoid):
    """Scores plus bias that differ by less than an fp32 step: the larger is chosen first."""
    E = 64
    x = np.zeros((1, E))
    x[0] = np.linspace(0, 1e-6, E)[np.random.default_rng(0).permutation(E)]
    bias = np.ones(E, np.float32)
    want = f8.route(x.astype(np.float32), 8, bias, sigmoid)
    e, _ = rt.route_experts(gpu(x, torch.float32), 8, bias=gpu(bias), score=int(sigmoid))
    assert np.array_equal(e.cpu().numpy(), want[0])


def test_route_strided_and_empty():
    x = torch.randn(50, 100, device="cuda")
    full = torch.full((50, 117), float("nan"), device="cuda")
    full[:, 9:109] = x
    for a, b in zip(rt.route_experts(x, 5), rt.route_experts(full[:, 9:109], 5)):
        assert torch.equal(a, b)
    e, w = rt.route_experts(x[:0], 5)
    assert e.shape == (0, 5) and w.shape == (0, 5)
    assert rt.route_experts_grad(x[:0], e, w).shape == (0, 100)
    rows = rt.expert_rows(e, 100)
    assert rows.rows == 0 and rows.offsets.tolist() == [0] * 101


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("E,k", [(1, 1), (7, 3), (64, 8), (100, 64), (256, 8), (500, 5), (1000, 9)])
def test_route_grad(E, k, sigmoid, renorm):
    """Against the formula in 64 bits (which the host tests hold against differences). fp32 values of 64-bit arithmetic, but
    for fp32 exponentials: 8 steps of the row's largest term cover them; then half a step of the dtype."""
    rng = np.random.default_rng(E)
    for dtype in ("f32", "bf16", "f16"):
        x = torch.from_numpy(rng.standard_normal((23, E)) * 2).to(DTYPES[dtype])
        xs = x.double().numpy()
        chosen, _ = f8.route(xs, k, None, sigmoid)
        chosen[3, 0], chosen[4] = -1, -1
        if k > 1:
            chosen[5, 1] = chosen[5, 0]  # the same expert twice
        d = rng.standard_normal((23, k)).astype(np.float32)
        want = f8.route_grad(xs, chosen, d, sigmoid, renorm, 1.5)
        got = rt.route_experts_grad(x.cuda(), gpu(chosen), gpu(d), score=int(sigmoid), renormalize=renorm, scale=1.5)
        assert got.dtype == x.dtype
        got = got.double().cpu().numpy()
        limit = 8 * 2.0**-23 * np.abs(d).max(1, keepdims=True) * 1.5 + torch.finfo(x.dtype).eps / 2 * np.abs(want) + 2.0**-25
        assert (np.abs(got - want) <= limit).all(), (np.abs(got - want) / limit).max()


def test_route_grad_of_masked_and_bad_rows():
    x = np.random.default_rng(11).standard_normal((6, 40)).astype(np.float32)
    x[1] = -np.inf
    x[2, 5] = np.nan
    x[3, 7] = np.inf
    x[4, 10:] = -np.inf
    for sigmoid in (False, True):
        for renorm in (False, True):
            chosen, _ = f8.route(x, 12, None, sigmoid)
            d = np.ones((6, 12), np.float32) * np.arange(12, dtype=np.float32)
            got = rt.route_experts_grad(gpu(x), gpu(chosen), gpu(d), score=int(sigmoid), renormalize=renorm).cpu().numpy()
            want = f8.route_grad(x, chosen, d, sigmoid, renorm, 1.0)
            assert np.array_equal(np.isnan(got), np.isnan(want)) and (np.isnan(got).all(1) == [False, False, True, True, False, False]).all()
            assert np.allclose(got, want, rtol=1e-5, atol=1e-5, equal_nan=True)
            assert (got[1] == 0).all() and (got[4, 10:] == 0).all()


def test_route_gradient_through_differences():
    """Weights of the library itself, differenced in fp32: h = 2^-6 makes truncation h^2 / 6 of the third derivative (below 1), 5e-5,
    and rounding 2^-23 / h, 1e-5, for each of the k weights."""
    gen = torch.Generator(device="cuda").manual_seed(4)
    x, d = torch.randn(4, 12, device="cuda", generator=gen), torch.rand(4, 3, device="cuda", generator=gen)
    x += 4 * (x > 0.3)  # choices that a step of h does not change
    for score in (rt.SCORE_SOFTMAX, rt.SCORE_SIGMOID):
        for renorm in (True, False):
            e, _ = rt.route_experts(x, 3, score=score, renormalize=renorm)
            g = rt.route_experts_grad(x, e, d, score=score, renormalize=renorm)
            for i in range(12):
                lo, hi = x.clone(), x.clone()
                lo[:, i] -= 2.0**-6
                hi[:, i] += 2.0**-6
                (el, wl), (eh, wh) = rt.route_experts(lo, 3, score=score, renormalize=renorm), rt.route_experts(hi, 3, score=score, renormalize=renorm)
                same = ((el == e) & (eh == e)).all(1)
                diff = ((wh - wl) * d).sum(1) * 2.0**5
                assert bool(((diff - g[:, i]).abs()[same] < 3 * 6e-5).all())


# ---- rows by expert ------------------------------------------------------------------------
@pytest.mark.parametrize("T,k,E", [(1, 1, 1), (1, 8, 256), (3, 2, 5), (64, 6, 64), (100, 7, 1024), (512, 8, 16), (513, 8, 17), (5000, 3, 100),
                                   (4097, 1, 1), (20000, 8, 256), (1000, 64, 40)])
@pytest.mark.parametrize("align", [1, 7, 128])
def test_expert_rows(T, k, E, align):
    rng = np.random.default_rng(T + E)
    for c in (rng.integers(0, E, (T, k)), rng.integers(-2, E + 2, (T, k)), np.full((T, k), E - 1), np.full((T, k), -1),
              np.minimum(rng.integers(0, 3 * E, (T, k)), E - 1)):
        announce(f"rows {T}x{k} of {E} align {align}")
        rows = rt.expert_rows(gpu(c.astype(np.int32)), E, align)
        valid = np.where((c >= 0) & (c < E), c, -1)
        for got, want in zip((rows.slots, rows.position, rows.offsets, rows.counts), f8.expert_rows(valid, E, align)):
            assert np.array_equal(got.cpu().numpy(), want)


# ---- experts' products ---------------------------------------------------------------------
def choose(rng, T, k, E, how):
    if how == "one":  # every token's first slot on one expert
        c = np.tile(np.arange(k, dtype=np.int32) % E, (T, 1))
    elif how == "holes":
        c = rng.integers(-1, E, (T, k)).astype(np.int32)
        c[c == E // 2] = -1  # an expert with no rows
    else:
        c = rng.integers(0, E, (T, k)).astype(np.int32)
    return c


def stack(rng, E, rows, cols, kind=f8.E4M3):
    parts = [random_matrix(rng, rows, cols, kind, 128) for _ in range(E)]
    return np.stack([p[0] for p in parts]), np.stack([p[1] for p in parts])


EXPERTS = [(1, 1, 1, 16, 128), (1, 2, 8, 64, 256), (5, 2, 4, 100, 130), (16, 6, 32, 256, 512), (33, 4, 7, 130, 777), (200, 3, 5, 260, 384),
           (700, 2, 3, 520, 1024), (2000, 1, 2, 300, 200), (64, 8, 16, 512, 640), (300, 8, 100, 128, 256)]


@pytest.mark.parametrize("T,k,E,N,K", EXPERTS)
@pytest.mark.parametrize("order", ["nt", "nn"])
@pytest.mark.parametrize("align", [1, 128])
def test_experts_products(T, k, E, N, K, order, align):
    rng = np.random.default_rng(T + N)
    codes, scales = stack(rng, E, *((N, K) if order == "nt" else (K, N)))
    vb = [f8.decode(codes[e], scales[e], f8.E4M3, 128) for e in range(E)]
    vb = [v.T if order == "nt" else v for v in vb]
    for dtype, layout, how, gather, beta in (("bf16", "aligned", "random", True, 0.0), ("f32", "aligned", "holes", False, 0.5),
                                             ("f16", "odd", "one", True, 0.0), ("bf16", "tight", "holes", True, 1.0)):
        kind = f8.E4M3 if gather else f8.E5M2
        c = choose(rng, T, k, E, how)
        slots, _, offsets, counts = f8.expert_rows(c, E, align)
        R = slots.size
        a = random_matrix(rng, T if gather else R, K, kind)
        va = f8.decode(*a, kind)
        rows = rt.expert_rows(gpu(c), E, align)
        A = device_matrix(*a, kind, 1, layout, "rows" if layout == "tight" else "columns")
        B = rt.F8Matrix(device_codes(codes, f8.E4M3, layout), device_scales(scales), 128)
        C = torch.full((R, N), 3.0, dtype=DTYPES[dtype], device="cuda")
        ref, mag = np.full((R, N), 3.0), np.zeros((R, N))
        for e in range(E):
            first = offsets[e]
            ref[first:offsets[e + 1]] = 0.0  # rows between groups
            r = np.arange(first, first + counts[e])
            m = va[slots[r] // k] if gather else va[r]
            ref[r] = m @ vb[e] + beta * 3.0
            mag[r] = np.abs(m) @ np.abs(vb[e]) + 3.0 * beta
        what = f"experts {order} T {T} k {k} E {E} N {N} K {K} align {align} {dtype} {layout} {how} gather {gather} beta {beta}"
        announce(what)
        got = rt.gemm_f8_experts(A, B.t() if order == "nt" else B, rows, C, gather=gather, beta=beta)
        assert got is C
        assert_close(C, ref, mag, what)


@pytest.mark.parametrize("T,k,E,M,N", [(1, 1, 1, 16, 16), (5, 2, 4, 100, 130), (64, 6, 16, 200, 300), (1000, 2, 3, 260, 129), (500, 4, 20, 64, 512),
                                       (3000, 1, 2, 300, 520)])
def test_experts_weight_gradients(T, k, E, M, N):
    rng = np.random.default_rng(T + M)
    for dtype, layout, how, align, beta in (("f32", "aligned", "random", 128, 0.0), ("f32", "odd", "holes", 256, 1.0), ("bf16", "aligned", "one", 128, 0.0)):
        c = choose(rng, T, k, E, how)
        slots, _, offsets, counts = f8.expert_rows(c, E, align)
        R = slots.size
        a, b = random_matrix(rng, M, R, f8.E5M2), random_matrix(rng, N, R)
        # what lies behind a group's count has no influence
        for q, bad in ((a, 0x7E), (b, 0x7F)):
            for e in range(E):
                q[0][:, offsets[e] + counts[e]:offsets[e + 1]] = bad
            q[0][:, offsets[E]:] = bad
            q[1][:, offsets[E] // 128:] = np.nan
        rows = rt.expert_rows(gpu(c), E, align)
        A, B = device_matrix(*a, f8.E5M2, 1, layout), device_matrix(*b, f8.E4M3, 1, layout)
        C = torch.full((E, M, N), 2.0, dtype=DTYPES[dtype], device="cuda")
        ref, mag = np.empty((E, M, N)), np.empty((E, M, N))
        with np.errstate(invalid="ignore"):
            va, vb = f8.decode(*a, f8.E5M2), f8.decode(*b, f8.E4M3)
        for e in range(E):
            r = np.arange(offsets[e], offsets[e] + counts[e])
            ref[e] = va[:, r] @ vb[:, r].T + 2.0 * beta
            mag[e] = np.abs(va[:, r]) @ np.abs(vb[:, r]).T + 2.0 * beta
        what = f"dw T {T} k {k} E {E} M {M} N {N} {dtype} {layout} {how} align {align}"
        announce(what)
        rt.gemm_f8_experts_dw(A, B.t(), rows, C, beta=beta)
        assert_close(C, ref, mag, what)


def test_products_keep_inside_whatever_the_rows_say():
    """Offsets, counts and slots out of range are kept inside the operands: rows that lie in a group twice or not at all hold
    something, and nothing else is touched."""
    T, k, E, N, K = 20, 2, 4, 64, 128
    rng = np.random.default_rng(12)
    A, B = device_matrix(*random_matrix(rng, T, K), f8.E4M3), rt.F8Matrix(device_codes(stack(rng, E, N, K)[0], f8.E4M3),
                                                                         torch.ones(E, 1, 1, device="cuda"), 128)
    i32 = dict(dtype=torch.int32, device="cuda")
    full = torch.full((T * k + 4, N), 5.0, device="cuda")
    for slots, offsets, counts in (([2**31 - 1] * 40, [0, 10, 20, 30, 40], [10] * 4), ([-5] * 40, [-7, 50, 3, 2**31 - 1, -1], [2**31 - 1, -1, 4, 7])):
        rows = rt.ExpertRows(torch.tensor(slots, **i32), torch.zeros(T, k, **i32), torch.tensor(offsets, **i32), torch.tensor(counts, **i32))
        rt.gemm_f8_experts(A, B.t(), rows, full[2:-2], gather=True)
        torch.cuda.synchronize()
        assert bool((full[:2] == 5.0).all()) and bool((full[-2:] == 5.0).all())


# ---- combine -------------------------------------------------------------------------------
@pytest.mark.parametrize("T,k,E,N", [(1, 1, 1, 1), (1, 8, 16, 2048), (5, 3, 4, 100), (64, 6, 64, 1024), (300, 5, 7, 777), (40, 2, 3, 8200), (1000, 8, 32, 16)])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("align", [1, 128])
def test_combine(T, k, E, N, dtype, align):
    rng = np.random.default_rng(T + N)
    for how, pad, weighted in (("random", 0, True), ("holes", 3, True), ("holes", 8, False)):
        c = choose(rng, T, k, E, how)
        slots, position, _, _ = f8.expert_rows(c, E, align)
        R = slots.size

        def dev(x):
            full = torch.full((x.shape[0], x.shape[1] + pad), float("nan"), dtype=DTYPES[dtype], device="cuda")
            full[:, :x.shape[1]] = torch.from_numpy(x)
            return full[:, :x.shape[1]]

        y, dy = rng.standard_normal((R, N)), rng.standard_normal((T, N))
        w = rng.random((T, k)).astype(np.float32)
        Y, dY = dev(y), dev(dy)
        y, dy = Y.double().cpu().numpy(), dY.double().cpu().numpy()
        rows = rt.expert_rows(gpu(c), E, align)
        weights = gpu(w) if weighted else None
        wv = w.astype(np.float64) if weighted else np.ones((T, k))
        picked = np.where((position >= 0)[..., None], y[position], 0.0)
        out = torch.full((T, N + pad), 7.0, dtype=DTYPES[dtype], device="cuda")
        got = rt.combine_experts(Y, rows, weights, out=out[:, :N])
        assert_close(got, (picked * wv[..., None]).sum(1), np.abs(picked * wv[..., None]).sum(1), "combine", eight_bit=False)
        assert bool((out[:, N:] == 7.0).all())
        assert torch.equal(rt.combine_experts(Y, rows, weights), got)
        gY, gw = rt.combine_experts_grad(dY, Y, rows, weights)
        there = slots >= 0
        t = np.where(there, slots // k, 0)
        ref = np.where(there[:, None], dy[t] * wv.reshape(-1)[np.where(there, slots, 0)][:, None], 0.0)
        assert_close(gY, ref, np.abs(ref), "dY", eight_bit=False)
        if weighted:
            prod = np.where((position >= 0)[..., None], picked * dy[:, None, :], 0.0)
            assert_close(gw, prod.sum(-1), np.abs(prod).sum(-1), "dw")
        else:
            assert gw is None


# ---- all of them together --------------------------------------------------------------------
def moe(x, logits, W, rows_align, dout, experts=None):
    """A layer with one matrix to an expert and its gradients, in the library's operators: (out, dlogits, dx, dW)."""
    E, k = W.shape[0], 2
    e, w = rt.route_experts(logits, k, score=rt.SCORE_SIGMOID)
    rows = rt.expert_rows(e, E, align=rows_align)
    parts = [rt.quantize_f8(W[i], block_rows=128) for i in range(E)]
    Wq = rt.F8Matrix(torch.stack([p.codes.view(torch.uint8) for p in parts]).view(torch.float8_e4m3fn), torch.stack([p.scales for p in parts]), 128)
    Y = rt.gemm_f8_experts(rt.quantize_f8(x), Wq.t(), rows, gather=True, dtype=x.dtype)
    out = rt.combine_experts(Y, rows, w)
    dY, dw = rt.combine_experts_grad(dout, Y, rows, w)
    dlogits = rt.route_experts_grad(logits, e, dw, score=rt.SCORE_SIGMOID)
    dX = rt.gemm_f8_experts(rt.quantize_f8(dY, torch.float8_e5m2), Wq, rows, dtype=x.dtype)
    dx = rt.combine_experts(dX, rows)
    dW = rt.gemm_f8_experts_dw(rt.quantize_f8(dY, torch.float8_e5m2, transpose=True),
                               rt.quantize_f8(x, transpose=True, rows=rows.token_of_row()).t(), rows)
    return out, dlogits, dx, dW


def moe_inputs(gen, T=150, E=5, N=192, K=272, dtype=torch.float32):
    def n(*s):
        return torch.randn(*s, device="cuda", generator=gen)
    return n(T, K).to(dtype), n(T, E).to(dtype), (n(E, N, K) * K**-0.5).to(dtype), (n(T, N) * 1e-2).to(dtype)


def test_moe_layer():
    """Against the same layer in 64 bits without any 8-bit codes. A product's relative error is 2^-4 + 2^-4 + 2^-8 (e4m3 twice) or
    2^-3 + 2^-4 + 2^-7 at most, at random signs far less: in the 2-norm, half steps are uniform, 1 / sqrt(3) of their bound, at
    mantissas spread over an octave, and two of them add in squares: below 0.075 for all four results (0.3 for rows whose
    weights cancel, as dlogits' do: differences of numbers that are each off by as much)."""
    gen = torch.Generator(device="cuda").manual_seed(5)
    x, logits, W, dout = moe_inputs(gen)
    got = moe(x, logits, W, 128, dout)
    leaves = [t.double().requires_grad_() for t in (logits, x, W)]
    s = torch.sigmoid(leaves[0])
    e = s.topk(2, -1).indices
    w = s.gather(1, e)
    w = w / w.sum(-1, keepdim=True)
    out = sum(w[:, j, None] * torch.matmul(leaves[2][e[:, j]], leaves[1][:, :, None])[..., 0] for j in range(2))
    out.backward(dout.double())
    want = [out.detach()] + [t.grad for t in leaves]
    for g, r, limit, what in zip(got, want, (0.075, 0.3, 0.075, 0.075), ("out", "dlogits", "dx", "dW")):
        rel = float((g.double() - r).norm() / r.norm())
        announce(f"moe {what} off by {rel:.3g} in the 2-norm")
        assert rel < limit, what


def test_moe_layer_captured_and_on_another_stream():
    gen = torch.Generator(device="cuda").manual_seed(6)
    held = moe_inputs(gen, dtype=torch.bfloat16)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        aside = moe(*held[:3], 128, held[3])
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    for a, b in zip(aside, moe(*held[:3], 128, held[3])):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = moe(*held[:3], 128, held[3])
    for _ in range(3):
        for t, new in zip(held, moe_inputs(gen, dtype=torch.bfloat16)):
            t.copy_(new)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, moe(*held[:3], 128, held[3])):
            assert torch.equal(a, b)


def test_refusals():
    x = torch.randn(6, 128, device="cuda")
    e, w = rt.route_experts(x, 2)
    rows = rt.expert_rows(e, 128)
    xq = rt.quantize_f8(x)
    W = rt.F8Matrix(torch.zeros(128, 64, 128, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn), torch.ones(128, 1, 1, device="cuda"), 128)
    for call, match in ((lambda: rt.route_experts(x, 0), "k must be"), (lambda: rt.route_experts(x, 65), "k must be"),
                        (lambda: rt.route_experts(x, 2, groups=3), "groups"), (lambda: rt.route_experts(x, 2, groups=4, top_groups=5), "top_groups"),
                        (lambda: rt.route_experts(x, 2, bias=torch.zeros(5, device="cuda")), "bias"),
                        (lambda: rt.route_experts(torch.zeros(2, 1025, device="cuda"), 2), "experts"),
                        (lambda: rt.route_experts_grad(x, e, w.double()), "dweights"), (lambda: rt.route_experts_grad(x, e[:3], w), "experts"),
                        (lambda: rt.expert_rows(e.long(), 128), "int32"), (lambda: rt.expert_rows(e, 0), "experts"), (lambda: rt.expert_rows(e, 128, 0), "align"),
                        (lambda: rt.gemm_f8_experts(xq, W.t(), rows), "A must have 12 rows"), (lambda: rt.gemm_f8_experts(xq, W, rows, gather=True), "inner"),
                        (lambda: rt.gemm_f8_experts(xq, W.t(), e, gather=True), "ExpertRows"),
                        (lambda: rt.gemm_f8_experts(xq, rt.quantize_f8(x, block_rows=128).t(), rows, gather=True), "stack"),
                        (lambda: rt.gemm_f8_experts_dw(xq, xq.t(), rows), "aligned to 128"),
                        (lambda: rt.combine_experts(x, rows), "Y must have"), (lambda: rt.combine_experts(torch.zeros(12, 4, device="cuda"), rows, w.double()), "weights"),
                        (lambda: rt.combine_experts_grad(x, None, rows, w), "Y must be")):
        with pytest.raises(ValueError, match=match):
            call()
