"""Block-scaled operands on the GPU: conversions against the 64-bit reference code by code, products in
every storage order against 64-bit products, edges, strides, streams, graphs and the three products
of a linear layer together."""
from __future__ import annotations

import numpy as np
import pytest

import mx_reference as mx
import register_tiled_matrix_amd as rt
from gpu_util import announce

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

FORMATS = [mx.FP4, mx.INT8]
HALF = {"bf16": torch.bfloat16, "f16": torch.float16}
GEMM = {"bf16": rt.gemm_bf16_mx, "f16": rt.gemm_f16_mx}
ORDERS = ["nt", "nn", "tn", "tt"]


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    rt.load()
    yield


def dev(x, pad=0, fill=0):
    """`x` on the GPU as a view with `pad` more elements of `fill` before and behind each row."""
    x = torch.as_tensor(x)
    full = torch.full((x.shape[0], x.shape[1] + 2 * pad), fill, dtype=x.dtype, device="cuda")
    v = full[:, pad:pad + x.shape[1]]
    v.copy_(x)
    return v


def dev_aligned(x, fill=0):
    """`x` on the GPU with rows that start at multiples of 16 elements, `fill` behind them."""
    x = torch.as_tensor(x)
    full = torch.full((x.shape[0], (x.shape[1] + 15) // 16 * 16), fill, dtype=x.dtype, device="cuda")
    v = full[:, :x.shape[1]]
    v.copy_(x)
    return v


def random_codes(rng, fmt, rows, cols, e_lo=120, e_hi=130):
    w, g = mx.widths(fmt, cols)
    codes = rng.integers(0, 256, (rows, w), dtype=np.uint8)
    if fmt == mx.FP4 and cols % 2:
        codes[:, -1] |= 0xA0  # the unused half of a row's last byte may hold anything
    return codes, rng.integers(e_lo, e_hi + 1, (rows, g)).astype(np.uint8)


def half_matrix(rng, rows, cols, dtype):
    return torch.from_numpy(rng.standard_normal((rows, cols))).to(HALF[dtype])


def assert_close(got, ref, mag, what):
    """The library's bound: 1e-5 of the sum of the magnitudes an output is made of (fp32 sums of
    exact products)."""
    got = got.cpu().double().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(ref)), f"{what}: NaN where there is none, or none where there is"
    fine = np.isfinite(ref)
    err = np.abs(got - ref)[fine] / (1e-5 * np.maximum(mag[fine], 1e-30))
    assert err.size == 0 or err.max() <= 1.0, f"{what}: |err| / bound {err.max():.3g} at {np.argwhere(fine)[err.argmax()]}"


# ---- conversions ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("fmt", FORMATS)
def test_dequantize_every_code_and_scale(fmt, dtype):
    E = np.arange(256, dtype=np.uint8)
    codes = np.tile(np.arange(256, dtype=np.uint8), (256, 1))
    cols = 512 if fmt == mx.FP4 else 256
    scales = np.repeat(E[:, None], cols // 32, axis=1)
    announce(f"dequantize {fmt} {dtype}")
    got = rt.dequantize_mx(rt.MXMatrix(fmt, dev(codes), dev(scales), cols), dtype=dtype)
    want = torch.from_numpy(mx.decode(codes, scales, fmt, cols)).to(dtype)
    got = got.cpu()
    assert torch.equal(got.isnan(), want.isnan())
    assert torch.equal(got.nan_to_num(7.0), want.nan_to_num(7.0))


def _special_rows(dtype):
    """Rows of 32 whose first value sets the exponent and whose others sit on and beside every border."""
    tiny, top = torch.finfo(dtype).smallest_normal, torch.finfo(dtype).max
    rows = []
    for scale in (1.0, 2.0**-9, 2.0**9):
        for lead in (4.0, 7.75, 6.0):
            ties = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.5, 0.0, -0.0])
            for off in (2.0**-7, 2.0**-20, -(2.0**-20)):
                v = np.concatenate([[lead], ties, -ties, ties * (1 + off)])[:32]
                rows.append(np.pad(v, (0, 32 - len(v))) * scale)
        i8 = np.concatenate([[1.0], (np.arange(-8, 8) + 0.5) / 64, [127.5 / 64, -127.5 / 64, 126.5 / 64, -1.0]])
        rows.append(np.pad(i8, (0, 32 - len(i8))) * scale)
    rows += [np.zeros(32), np.full(32, tiny), np.full(32, tiny / 4), np.linspace(-top, top, 32), np.full(32, top)]
    return np.stack(rows)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("fmt", FORMATS)
def test_quantize_codes(fmt, dtype):
    rng = np.random.default_rng(3)
    blocks = [_special_rows(dtype), rng.standard_normal((64, 32)) * np.exp2(rng.integers(-12, 12, (64, 1)))]
    if dtype != torch.float32:  # every finite value, in the order of its bits
        every = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(dtype).double()
        every = every[every.isfinite()].numpy()
        blocks.append(every[: len(every) // 32 * 32].reshape(-1, 32))
    X = torch.from_numpy(np.concatenate(blocks)).to(dtype)
    announce(f"quantize {fmt} {dtype}")
    Q = rt.quantize_mx(X.cuda(), fmt)
    codes, scales = mx.encode(X.double().numpy(), fmt)
    assert np.array_equal(Q.scales.cpu().numpy(), scales)
    assert np.array_equal(Q.codes.cpu().numpy(), codes)


@pytest.mark.parametrize("fmt", FORMATS)
def test_quantize_groups_with_nan_and_infinity(fmt):
    x = torch.randn(6, 96, dtype=torch.float32)
    x[1, 40] = float("nan")
    x[2, 95] = float("inf")
    x[3, 0] = -float("inf")
    x[4, 32:64] = float("nan")
    Q = rt.quantize_mx(x.cuda(), fmt)
    codes, scales = mx.encode(x.double().numpy(), fmt)
    assert np.array_equal(Q.scales.cpu().numpy(), scales) and np.array_equal(Q.codes.cpu().numpy(), codes)
    back = rt.dequantize_mx(Q, dtype=torch.float32).cpu()
    assert int(back.isnan().sum()) == 4 * 32


@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 2), (3, 7), (5, 31), (2, 33), (7, 64), (4, 95), (33, 777), (257, 129), (1, 8192)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("fmt", FORMATS)
def test_conversions_touch_their_rows_only(fmt, dtype, rows, cols):
    rng = np.random.default_rng(rows * 1000 + cols)
    X = torch.from_numpy(rng.standard_normal((rows, cols))).to(dtype)
    w, g = mx.widths(fmt, cols)
    pad = 3
    cf = torch.full((rows, w + 2 * pad), 0xA5, dtype=torch.uint8, device="cuda")
    sf = torch.full((rows, g + 2 * pad), 0xA5, dtype=torch.uint8, device="cuda")
    out = rt.MXMatrix(fmt, cf[:, pad:pad + w], sf[:, pad:pad + g], cols)
    assert rt.quantize_mx(dev(X, pad, float("nan")), fmt, out=out) is out
    codes, scales = mx.encode(X.double().numpy(), fmt)
    assert np.array_equal(out.codes.cpu().numpy(), codes) and np.array_equal(out.scales.cpu().numpy(), scales)
    for full, n in ((cf, w), (sf, g)):
        assert bool((full[:, :pad] == 0xA5).all()) and bool((full[:, pad + n:] == 0xA5).all())
    xf = torch.full((rows, cols + 2 * pad), 7.0, dtype=dtype, device="cuda")
    rt.dequantize_mx(out, out=xf[:, pad:pad + cols])
    want = torch.from_numpy(mx.decode(codes, scales, fmt, cols)).to(dtype)
    assert torch.equal(xf[:, pad:pad + cols].cpu(), want)
    assert bool((xf[:, :pad] == 7).all()) and bool((xf[:, pad + cols:] == 7).all())


# ---- products ------------------------------------------------------------------------------
def product(rng, fmt, dtype, order, M, N, K, alpha=1.0, beta=0.0, pad=0, e_lo=120, e_hi=130, c_pad=0, label="", aligned=False):
    """One product against 64 bits; the padding of every operand is NaN (codes 0xFF, scales 255), C's
    must stay."""
    A = half_matrix(rng, K, M, dtype) if order[0] == "t" else half_matrix(rng, M, K, dtype)
    rows, cols = (N, K) if order[1] == "t" else (K, N)
    codes, scales = random_codes(rng, fmt, rows, cols, e_lo, e_hi)
    if aligned:
        Ad, Qd, Sd = dev_aligned(A, float("nan")), dev_aligned(codes, 255), dev_aligned(scales, 255)
    else:
        Ad, Qd, Sd = dev(A, pad, float("nan")), dev(codes, pad, 255), dev(scales, pad, 255)
    B = rt.MXMatrix(fmt, Qd, Sd, cols)
    C0 = torch.from_numpy(rng.standard_normal((M, N))).float()
    Cf = torch.full((M, N + 2 * c_pad), 3.0, device="cuda")
    C = Cf[:, c_pad:c_pad + N]
    C.copy_(C0) if beta != 0.0 else C.fill_(float("nan"))
    announce(f"gemm_mx {fmt} {dtype} {order} {M}x{N}x{K} {label}")
    got = GEMM[dtype](Ad.t() if order[0] == "t" else Ad, B.t() if order[1] == "t" else B, C, alpha=alpha, beta=beta)
    torch.cuda.synchronize()
    assert got is C
    a = A.double().numpy()
    b = mx.decode(codes, scales, fmt, cols)
    a, b = (a.T if order[0] == "t" else a), (b.T if order[1] == "t" else b)
    ref = alpha * (a @ b) + (beta * C0.double().numpy() if beta != 0.0 else 0.0)
    mag = abs(alpha) * (np.abs(a) @ np.abs(b)) + np.abs(beta * C0.double().numpy())
    assert_close(C, ref, mag, f"{order} {M}x{N}x{K} {rt.last_kernel()}")
    if c_pad:
        assert bool((Cf[:, :c_pad] == 3).all()) and bool((Cf[:, c_pad + N:] == 3).all())
    return C


SIZES = [(1, 1, 1), (1, 2, 31), (2, 33, 32), (1, 17, 33), (3, 64, 64), (16, 48, 512), (17, 100, 77), (33, 65, 129),
         (64, 64, 64), (65, 127, 191), (1, 256, 1024), (4, 1000, 2049), (5, 130, 4161), (8, 36, 8192), (12, 50, 1100), (32, 40, 4128), (1, 6, 8224), (40, 33, 640), (64, 100, 1152), (49, 18, 8448), (100, 150, 777), (130, 257, 95), (256, 320, 256)]


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("order", ORDERS)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("fmt", FORMATS)
def test_product(fmt, dtype, order, M, N, K):
    product(np.random.default_rng(M * 7 + N * 3 + K), fmt, dtype, order, M, N, K)


@pytest.mark.parametrize("M,N,K", [(1, 100, 100), (5, 96, 515), (40, 70, 130), (129, 200, 333)])
@pytest.mark.parametrize("order", ORDERS)
@pytest.mark.parametrize("fmt", FORMATS)
def test_product_strides_alpha_beta(fmt, order, M, N, K):
    rng = np.random.default_rng(K)
    product(rng, fmt, "bf16", order, M, N, K, alpha=1.5, beta=-0.5, pad=1, c_pad=1, label="odd strides")
    product(rng, fmt, "f16", order, M, N, K, alpha=-0.75, beta=1.0, pad=8, c_pad=4, label="padded")


@pytest.mark.parametrize("M", [1, 3, 5, 8, 9, 16, 17, 32, 33, 48, 49, 64])
@pytest.mark.parametrize("N", [40, 4112, 8200])
@pytest.mark.parametrize("fmt", FORMATS)
def test_product_tokens(fmt, N, M):
    """Every shape of the kernels for a few rows: K of whole chunks and with a short one, fewer
    chunks than waves, unaligned rows."""
    rng = np.random.default_rng(M * N)
    for K, pad in ((1536, 0), (2080, 16), (77, 0), (1100, 1)):
        product(rng, fmt, "bf16" if K != 2080 else "f16", "nt", M, N, K, beta=0.5 if pad else 0.0, pad=pad, c_pad=pad % 2, label="tokens")


# K split over the waves of 64x64 tiles: whole slabs of 128 and a tail, fewer slabs than the ring, one
# part and several
@pytest.mark.parametrize("M,N,K", [(65, 40, 512), (100, 1500, 777), (128, 64, 1024), (130, 200, 4096 + 72), (192, 72, 2049), (300, 520, 640)])
@pytest.mark.parametrize("fmt", FORMATS)
def test_product_split_over_waves(fmt, M, N, K):
    rng = np.random.default_rng(M + N + K)
    product(rng, fmt, "bf16", "nt", M, N, K, label="split-K", aligned=True)
    assert "splitk4" in rt.last_kernel()
    product(rng, fmt, "f16", "nt", M, N, K, alpha=-0.5, beta=2.0, c_pad=1, label="split-K", aligned=True)
    assert "splitk4" in rt.last_kernel()


# the DMA kernels: one slab, slabs that end inside a group of four, tiles that end anywhere, 128 and
# 256 wide tiles
@pytest.mark.parametrize("M,N,K", [(72, 96, 32), (136, 160, 64), (200, 288, 96), (128, 128, 640), (264, 512, 224), (1000, 1504, 800),
                                   (2304, 4096 + 32, 160), (4096, 2304, 64)])
@pytest.mark.parametrize("order", ORDERS)
@pytest.mark.parametrize("fmt", FORMATS)
def test_product_dma(fmt, order, M, N, K):
    rng = np.random.default_rng(M + N + K)
    product(rng, fmt, "bf16", order, M, N, K, label="dma")
    assert "_dma_" in rt.last_kernel() or "_splitk4_" in rt.last_kernel()
    product(rng, fmt, "f16", order, M, N, K, alpha=0.5, beta=-1.0, pad=16, c_pad=1, label="dma, padded")
    assert "_dma_" in rt.last_kernel() or "_splitk4_" in rt.last_kernel()


@pytest.mark.parametrize("M,N,K", [(3000, 3000, 128), (2304, 4096 + 40, 256), (4100, 2304, 640), (33 * 128, 2200, 384), (70, 40, 128), (1300, 2000, 256), (2048, 2048, 4096), (300, 300, 9 * 1024 + 128)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_product_codes_in_lds(dtype, M, N, K):
    """256- and 128-wide tiles with 4-bit codes in LDS: one unit of K, an odd and an even number of them,
    tiles that end anywhere, K split over workgroups."""
    rng = np.random.default_rng(M + N + K)
    product(rng, mx.FP4, dtype, "nt", M, N, K, label="codes", aligned=True)
    assert "_codes_" in rt.last_kernel() or M * N < 2**17
    product(rng, mx.FP4, dtype, "nt", M, N, K, alpha=0.5, beta=-1.0, c_pad=1, label="codes", aligned=True)
    assert "_codes_" in rt.last_kernel() or M * N < 2**17


@pytest.mark.parametrize("order", ["nt", "nn", "tn"])
@pytest.mark.parametrize("fmt", FORMATS)
def test_product_wide_tiles_in_parts(fmt, order):
    """256x256 tiles in parts of a long K, with the workspace and, on narrower tiles, without."""
    rng = np.random.default_rng(10)
    M, N, K = 1040, 1824, 8192 + 96
    assert rt.regtile_gemm_mx_workspace(int(order[0] == "t"), int(order[1] == "t"), M, N, K, M if order[0] == "t" else K, N) > 0
    A = half_matrix(rng, *((K, M) if order[0] == "t" else (M, K)), "bf16").cuda()
    rows, cols = (N, K) if order[1] == "t" else (K, N)
    codes, scales = random_codes(rng, fmt, rows, cols)
    B = rt.MXMatrix(fmt, dev_aligned(codes), dev_aligned(scales), cols)
    ta, tb = int(order[0] == "t"), int(order[1] == "t")
    C = rt.gemm_bf16_mx(A.t() if ta else A, B.t() if tb else B)
    assert "256x256" in rt.last_kernel()
    D = torch.empty_like(C)
    assert rt.regtile_gemm_bf16_mx(fmt, ta, tb, M, N, K, 1.0, A.data_ptr(), A.stride(0), B.codes.data_ptr(), B.codes.stride(0),
                                   B.scales.data_ptr(), B.scales.stride(0), 0.0, D.data_ptr(), N, 0, 0,
                                   torch.cuda.current_stream().cuda_stream) == 0
    assert "128x128" in rt.last_kernel()
    a, b = A.double(), torch.from_numpy(mx.decode(codes, scales, fmt, cols)).cuda()
    a, b = (a.t() if ta else a), (b.t() if tb else b)
    ref, mag = (a @ b).cpu().numpy(), (a.abs() @ b.abs()).cpu().numpy()
    assert_close(C, ref, mag, "wide parts")
    assert_close(D, ref, mag, "128-wide")


@pytest.mark.parametrize("M,N,K", [(72, 96, 2048), (128, 288, 4096 + 32), (264, 136 + 24, 8192)])
@pytest.mark.parametrize("order", ORDERS)
@pytest.mark.parametrize("fmt", FORMATS)
def test_product_split_over_workgroups(fmt, order, M, N, K):
    """Few tiles, long K: partial sums through the workspace, joined in order; with any smaller
    workspace (none among them) the call makes fewer splits."""
    rng = np.random.default_rng(M + N + K)
    ta, tb = order[0] == "t", order[1] == "t"
    size = rt.regtile_gemm_mx_workspace(int(ta), int(tb), M, N, K, M if ta else K, N)
    assert size >= 2 * M * N * 4
    product(rng, fmt, "bf16", order, M, N, K, label="split")
    product(rng, fmt, "f16", order, M, N, K, alpha=-1.5, beta=1.0, c_pad=1, label="split")
    A = half_matrix(rng, *((K, M) if ta else (M, K)), "bf16")
    rows, cols = (N, K) if tb else (K, N)
    codes, scales = random_codes(rng, fmt, rows, cols)
    Ad, Qd, Sd = A.cuda(), dev(codes), dev(scales)
    a, b = A.double().numpy(), mx.decode(codes, scales, fmt, cols)
    a, b = (a.T if ta else a), (b.T if tb else b)
    for parts in (0, 1, 2, 3, 1000):
        work = torch.full((parts * M * N + 4,), float("nan"), device="cuda")
        C = torch.empty(M, N, device="cuda")
        assert rt.regtile_gemm_bf16_mx(fmt, int(ta), int(tb), M, N, K, 1.0, Ad.data_ptr(), Ad.stride(0), Qd.data_ptr(),
                                       Qd.stride(0), Sd.data_ptr(), Sd.stride(0), 0.0, C.data_ptr(), N,
                                       work.data_ptr() if parts else 0, parts * M * N * 4,
                                       torch.cuda.current_stream().cuda_stream) == 0
        torch.cuda.synchronize()
        assert_close(C, a @ b, np.abs(a) @ np.abs(b), f"{parts} parts")
        assert bool(work[parts * M * N:].isnan().all())


@pytest.mark.parametrize("order", ORDERS)
@pytest.mark.parametrize("fmt", FORMATS)
def test_infinite_groups_do_not_reach_past_the_edge(fmt, order):
    """The group at the end of K overflows to infinity: outputs are infinite, not NaN, though the
    kernels multiply what lies past K by zero."""
    M, N, K = 72, 96, 96
    rows, cols = (N, K) if order[1] == "t" else (K, N)
    w, g = mx.widths(fmt, cols)
    codes = np.full((rows, w), 0x11 if fmt == mx.FP4 else 1, dtype=np.uint8)  # all positive
    scales = np.full((rows, g), 120, dtype=np.uint8)
    if order[1] == "t":
        scales[:, -1] = 160
    else:
        scales[-1, :] = 160
    A = torch.full((M, K), 1.0, dtype=torch.float16, device="cuda")
    A = A.t().contiguous().t() if order[0] == "t" else A
    B = rt.MXMatrix(fmt, dev(codes), dev(scales), cols)
    got = rt.gemm_f16_mx(A, B.t() if order[1] == "t" else B)  # 2^26 and more overflow fp16
    assert bool(torch.isposinf(got).all()), (rt.last_kernel(), got.unique())


@pytest.mark.parametrize("order", ORDERS)
@pytest.mark.parametrize("fmt", FORMATS)
def test_product_integers_bitwise(fmt, order):
    """Integer operands whose sums stay below 2^24: every order of summation is exact."""
    rng = np.random.default_rng(1)
    M, N, K = 96, 224, 640
    rows, cols = (N, K) if order[1] == "t" else (K, N)
    A = torch.from_numpy(rng.integers(-3, 4, (K, M) if order[0] == "t" else (M, K))).to(torch.bfloat16)
    codes, _ = random_codes(rng, fmt, rows, cols)
    w, g = mx.widths(fmt, cols)
    scales = np.full((rows, g), 128 if fmt == mx.FP4 else 133, dtype=np.uint8)  # integer values
    B = rt.MXMatrix(fmt, dev(codes), dev(scales), cols)
    Ad = A.cuda()
    got = rt.gemm_bf16_mx(Ad.t() if order[0] == "t" else Ad, B.t() if order[1] == "t" else B)
    a, b = A.double().numpy(), mx.decode(codes, scales, fmt, cols)
    ref = (a.T if order[0] == "t" else a) @ (b.T if order[1] == "t" else b)
    assert np.array_equal(got.cpu().double().numpy(), ref)


@pytest.mark.parametrize("M", [1, 48])
@pytest.mark.parametrize("order", ["nt", "nn"])
@pytest.mark.parametrize("fmt", FORMATS)
def test_nan_groups_reach_their_outputs_only(fmt, order, M):
    rng = np.random.default_rng(2)
    N, K = 96, 160
    rows, cols = (N, K) if order[1] == "t" else (K, N)
    codes, scales = random_codes(rng, fmt, rows, cols)
    scales[5, 1] = 255
    A = half_matrix(rng, M, K, "bf16")
    B = rt.MXMatrix(fmt, dev(codes), dev(scales), cols)
    got = rt.gemm_bf16_mx(A.cuda(), B.t() if order[1] == "t" else B)
    b = mx.decode(codes, scales, fmt, cols)
    b = b.T if order[1] == "t" else b
    a = A.double().numpy()
    assert_close(got, a @ b, np.abs(a) @ np.abs(b), order)


@pytest.mark.parametrize("fmt", FORMATS)
def test_extreme_scales(fmt):
    """Groups at both ends of the scales: subnormal and near-overflow values are kept in bf16."""
    rng = np.random.default_rng(4)
    M, N, K = 3, 64, 64
    codes, scales = random_codes(rng, fmt, N, K)
    scales[:32], scales[32:] = 0, 180
    a = np.zeros((M, K))
    a[:, ::7] = 2.0**-20
    A = torch.from_numpy(a).to(torch.bfloat16)
    B = rt.MXMatrix(fmt, dev(codes), dev(scales), K)
    A2 = (A.double() * 2.0**80).to(torch.bfloat16)
    got = rt.gemm_bf16_mx(A2.cuda(), B.t())
    b = mx.decode(codes, scales, fmt, K).T
    a2 = A2.double().numpy()
    ref = a2 @ b
    assert_close(got, ref, np.abs(a2) @ np.abs(b), "extreme scales")


def test_empty_and_degenerate_sizes():
    e = torch.empty
    for M, N, K in ((0, 5, 7), (5, 0, 7), (5, 6, 0), (0, 0, 0)):
        A = torch.zeros(M, K, dtype=torch.bfloat16, device="cuda")
        w, g = mx.widths(mx.FP4, K)
        B = rt.MXMatrix(mx.FP4, e(N, w, dtype=torch.uint8, device="cuda"), e(N, g, dtype=torch.uint8, device="cuda"), K)
        C = torch.full((M, N), 2.0, device="cuda")
        rt.gemm_bf16_mx(A, B.t(), C, beta=0.5)
        assert bool((C == 1.0).all())
        Q = rt.quantize_mx(A, mx.INT8)
        assert Q.shape == (M, K) and tuple(rt.dequantize_mx(Q).shape) == (M, K)
    # alpha 0 reads neither operand
    A = torch.full((4, 32), float("nan"), dtype=torch.bfloat16, device="cuda")
    B = rt.quantize_mx(torch.full((8, 32), float("nan"), device="cuda"), mx.FP4)
    assert bool((rt.gemm_bf16_mx(A, B.t(), alpha=0.0) == 0).all())


def test_refusals():
    B = rt.quantize_mx(torch.randn(8, 64, device="cuda"), mx.FP4)
    A = torch.zeros(4, 64, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError, match="inner dimensions"):
        rt.gemm_bf16_mx(A, B)
    with pytest.raises(ValueError, match="beta"):
        rt.gemm_bf16_mx(A, B.t(), beta=1.0)
    with pytest.raises(ValueError, match="float32 of shape"):
        rt.gemm_bf16_mx(A, B.t(), torch.zeros(4, 7, device="cuda"))
    with pytest.raises(ValueError, match="row-major"):
        rt.gemm_bf16_mx(A[:, ::2], rt.quantize_mx(torch.randn(8, 32, device="cuda"), mx.FP4).t())
    with pytest.raises(ValueError, match="unit column stride"):
        rt.quantize_mx(torch.randn(8, 64, device="cuda").t())
    with pytest.raises(ValueError, match="out must be"):
        rt.quantize_mx(torch.randn(8, 65, device="cuda"), mx.FP4, out=B)
    with pytest.raises(ValueError, match="out must be"):
        rt.dequantize_mx(B, out=torch.zeros(64, 8, device="cuda"))
    T = rt.dequantize_mx(B.t(), dtype=torch.float32)
    assert tuple(T.shape) == (64, 8) and torch.equal(T, rt.dequantize_mx(B, dtype=torch.float32).t())


def test_repeated_calls_give_identical_bits():
    rng = np.random.default_rng(5)
    for order, M, N, K in (("nt", 1, 1024, 4096), ("nt", 24, 512, 4096), ("nn", 200, 256, 1000), ("tn", 256, 256, 4096), ("tn", 256, 256, 8192)):
        rows, cols = (N, K) if order[1] == "t" else (K, N)
        codes, scales = random_codes(rng, mx.INT8, rows, cols)
        B = rt.MXMatrix(mx.INT8, dev(codes), dev(scales), cols)
        A = half_matrix(rng, K, M, "bf16").cuda().t() if order[0] == "t" else half_matrix(rng, M, K, "bf16").cuda()
        outs = [rt.gemm_bf16_mx(A, B.t() if order[1] == "t" else B) for _ in range(4)]
        assert all(torch.equal(outs[0], o) for o in outs[1:])


def test_rows_past_four_gigabytes():
    """Offsets of A, codes, scales and C past 2^32 bytes."""
    M, N, K = 3, 3, 96
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GB of free memory")
    rng = np.random.default_rng(6)
    codes, scales = random_codes(rng, mx.INT8, N, K)
    big = 2**31 - 1
    qf = torch.empty(2 * big + K, dtype=torch.uint8, device="cuda")
    sf = torch.empty(2 * big + 3, dtype=torch.uint8, device="cuda")
    af = torch.empty(2 * big + K, dtype=torch.bfloat16, device="cuda")
    cf = torch.empty(2 * big + N, dtype=torch.float32, device="cuda")
    Q, S = qf.as_strided((N, K), (big, 1)), sf.as_strided((N, 3), (big, 1))
    A, C = af.as_strided((M, K), (big, 1)), cf.as_strided((M, N), (big, 1))
    Q.copy_(torch.from_numpy(codes)), S.copy_(torch.from_numpy(scales))
    a = half_matrix(rng, M, K, "bf16")
    A.copy_(a)
    rt.gemm_bf16_mx(A, rt.MXMatrix(mx.INT8, Q, S, K).t(), C)
    b = mx.decode(codes, scales, mx.INT8, K).T
    assert_close(C, a.double().numpy() @ b, np.abs(a.double().numpy()) @ np.abs(b), "far rows")
    out = rt.MXMatrix(mx.INT8, qf.as_strided((M, K), (big, 1)), sf.as_strided((M, 3), (big, 1)), K)
    rt.quantize_mx(A, mx.INT8, out=out)
    want, ws = mx.encode(a.double().numpy(), mx.INT8)
    assert np.array_equal(out.codes.cpu().numpy(), want) and np.array_equal(out.scales.cpu().numpy(), ws)


# ---- streams and graphs --------------------------------------------------------------------
def test_side_stream_and_allocation():
    x = torch.randn(64, 2048, device="cuda", dtype=torch.bfloat16)
    W = rt.quantize_mx(torch.randn(512, 2048, device="cuda"), mx.FP4)
    want = rt.gemm_bf16_mx(x, W.t())
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for s in (side, side.cuda_stream):
        Q = rt.quantize_mx(x, mx.INT8, stream=s)
        y = rt.gemm_bf16_mx(x, W.t(), stream=s)
        d = rt.dequantize_mx(Q, stream=s)
        side.synchronize()
        assert torch.equal(y, want)
        assert torch.equal(d, rt.dequantize_mx(rt.quantize_mx(x, mx.INT8)))
    with torch.cuda.stream(side):
        y = rt.gemm_bf16_mx(x, W.t())
    side.synchronize()
    assert torch.equal(y, want)


def test_two_streams_at_once():
    """Calls that use a workspace, and one token's, running together on two streams: each call has its own
    workspace, and the results are those of one stream."""
    X = rt.quantize_mx(torch.randn(4096, 256, device="cuda"), mx.INT8)
    dy = [torch.randn(4096, 192, device="cuda", dtype=torch.bfloat16) for _ in range(2)]
    assert rt.regtile_gemm_mx_workspace(1, 0, 192, 256, 4096, 192, 256) > 0
    want = [rt.gemm_bf16_mx(d.t(), X) for d in dy]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                outs[i].append(rt.gemm_bf16_mx(dy[i].t(), X))
                rt.gemm_bf16_mx(dy[i][:1], rt.quantize_mx(dy[i], mx.FP4).t())
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(o, want[i]) for o in outs[i])


def test_many_columns_of_few_tokens():
    """More columns of C than the token kernels' launches can count threads for."""
    N, K = (1 << 24) + 40, 32
    rng = np.random.default_rng(9)
    codes, scales = random_codes(rng, mx.FP4, 64, K)
    Q = torch.from_numpy(codes).cuda().repeat(N // 64 + 1, 1)[:N].contiguous()
    S = torch.from_numpy(scales).cuda().repeat(N // 64 + 1, 1)[:N].contiguous()
    A = half_matrix(rng, 2, K, "bf16")
    got = rt.gemm_bf16_mx(A.cuda(), rt.MXMatrix(mx.FP4, Q, S, K).t())
    a, b = A.double().numpy(), mx.decode(codes, scales, mx.FP4, K).T
    assert_close(got[:, :64], a @ b, np.abs(a) @ np.abs(b), "many columns")
    whole = N // 64 * 64
    assert torch.equal(got[:, :whole].reshape(2, -1, 64), got[:, None, :64].expand(2, N // 64, 64))
    assert torch.equal(got[:, whole:], got[:, : N - whole])


def test_graph_of_a_linear_layer():
    """Forward, checkpoint and both gradients captured together; every replay on new inputs equals the
    eager calls."""
    T, I, O = 200, 320, 264
    x, dy = torch.empty(T, I, device="cuda", dtype=torch.bfloat16), torch.empty(T, O, device="cuda", dtype=torch.bfloat16)
    W = rt.quantize_mx(torch.randn(O, I, device="cuda"), mx.FP4)

    def layer():
        y = rt.gemm_bf16_mx(x, W.t())
        kept = rt.quantize_mx(x, mx.INT8)
        dx = rt.gemm_bf16_mx(dy, W)
        dw = rt.gemm_bf16_mx(dy.t(), kept)
        one = rt.gemm_bf16_mx(x[:1], W.t())
        return y, kept.codes, kept.scales, dx, dw, one

    x.normal_(), dy.normal_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = layer()
    for version in range(4):
        x.normal_(), dy.normal_()
        eager = layer()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for o, e in zip(outs, eager):
            assert torch.equal(o, e), version


# ---- a linear layer ------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_linear_layer_gradients(dtype):
    """y = x W^T with W in 4 bits; dx through W and dW from x kept in 8 bits against 64 bits, and dx and dW
    against differences of the loss sum(g * y)."""
    rng = np.random.default_rng(8)
    T, I, O = 70, 200, 130
    gemm = GEMM[dtype]
    W = rt.quantize_mx(torch.from_numpy(rng.standard_normal((O, I))).float().cuda(), mx.FP4)
    w = rt.dequantize_mx(W, dtype=torch.float32).cpu().double().numpy()
    x, g = half_matrix(rng, T, I, dtype), half_matrix(rng, T, O, dtype)
    xd, gd = x.cuda(), g.cuda()
    X8 = rt.quantize_mx(xd, mx.INT8)
    x8 = rt.dequantize_mx(X8, dtype=torch.float32).cpu().double().numpy()
    xn, gn = x.double().numpy(), g.double().numpy()
    y, dx = gemm(xd, W.t()), gemm(gd, W)
    dw = torch.ones(O, I, device="cuda")
    gemm(gd.t(), X8, dw, beta=1.0)
    assert_close(y, xn @ w.T, np.abs(xn) @ np.abs(w.T), "y")
    assert_close(dx, gn @ w, np.abs(gn) @ np.abs(w), "dx")
    assert_close(dw, gn.T @ x8 + 1, np.abs(gn.T) @ np.abs(x8) + 1, "dw")
    # int8 elements are within half a step of 2^-6 of the group's top power of two: 2^-7 of the
    # group's largest magnitude at most (one whole step, 2^-6, where 127 saturates)
    groups = np.abs(np.pad(xn, ((0, 0), (0, -I % 32)))).reshape(T, -1, 32).max(-1)
    assert (np.abs(x8 - xn) <= np.repeat(groups, 32, 1)[:, :I] * 2.0**-7).all()
    # differences: the loss is linear in x, so its central difference along d is <dx, d> up to
    # the roundings of y, 1e-5 of the magnitudes each
    d = torch.from_numpy(rng.integers(-2, 3, (T, I))).to(HALF[dtype]).cuda()
    loss = lambda t: float((gemm(t, W.t()).double() * gd.double()).sum())  # noqa: E731
    base = d * 8
    diff = (loss(base + d) - loss(base - d)) / 2
    bound = 1e-5 * float((9 * d.abs().double().cpu() @ torch.from_numpy(np.abs(w.T)) * g.double().abs()).sum())
    assert abs(diff - float((dx.double() * d.double()).sum())) <= 2 * bound
