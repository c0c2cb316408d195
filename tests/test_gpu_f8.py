"""8-bit float matrices on the GPU: conversions against the 64-bit reference code by code, products in every
storage order, type, size and alignment against 64-bit products, edges, streams, graphs, and the three products of
a linear layer together."""
from __future__ import annotations

import numpy as np
import pytest

import f8_reference as f8
import register_tiled_matrix_amd as rt
from gpu_util import announce

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
from f8_gpu_util import DTYPES, TYPES, assert_close, device_codes, device_matrix, device_scales, random_matrix  # noqa: E402

KINDS = [f8.E4M3, f8.E5M2]


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    rt.load()
    yield


def host(Q):
    """(codes, scales) of an F8Matrix"""
    return Q.codes.view(torch.uint8).cpu().numpy(), Q.scales.cpu().numpy()


# ---- conversions ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("kind", KINDS)
def test_dequantize_every_code(kind, dtype):
    codes = np.tile(np.arange(256, dtype=np.uint8), (6, 1))
    scales = np.array([[1.0, 0.3], [2.0**-126, 2.0**-20], [1e-3, 3e37 / f8.TOP[kind]], [np.nan, 1.0], [7e-6, 1.25], [2.0**10, 0.0]], np.float32)
    announce(f"dequantize {kind} {dtype}")
    got = rt.dequantize_f8(device_matrix(codes, scales, kind), dtype=DTYPES[dtype]).cpu()
    # code * scale in fp32 (one rounding, as documented by its type), then to the dtype
    want = torch.from_numpy(f8.decode_table(kind)[codes].astype(np.float32) * scales.repeat(128, 1)).to(DTYPES[dtype])
    assert torch.equal(got.isnan(), want.isnan()) and torch.equal(got.nan_to_num(7.0), want.nan_to_num(7.0))


def special_rows(kind, dtype):
    """Rows whose first value sets the scale and whose others sit on and beside the borders between codes."""
    table = f8.decode_table(kind)[:128]
    table = table[np.isfinite(table)]
    border = (table[1:] + table[:-1]) / 2
    values = np.concatenate([border, -border, border * (1 + 2.0**-20), border * (1 - 2.0**-20), table])
    rows = []
    for scale in (1.0, 3.0, 2.0**-9, 0.7, 2.0**5):
        for part in np.array_split(values, -(-len(values) // 127)):
            rows.append(np.pad(np.concatenate([[table[-1]], part]), (0, 127 - len(part))) * scale / (table[-1] if dtype == torch.float16 else 1))
    tiny, top = torch.finfo(dtype).smallest_normal, torch.finfo(dtype).max
    rows += [np.zeros(128), np.full(128, tiny), np.full(128, tiny / 4), np.linspace(-top, top, 128), np.full(128, top),
             np.linspace(-tiny, tiny, 128), np.linspace(0, tiny * 1000, 128)]
    return np.stack(rows)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("kind", KINDS)
def test_quantize_codes(kind, dtype):
    rng = np.random.default_rng(3)
    blocks = [special_rows(kind, DTYPES[dtype]), rng.standard_normal((300, 128)) * np.exp2(rng.integers(-12, 12, (300, 1)))]
    if dtype != "f32":  # every finite value, in the order of its bits
        every = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(DTYPES[dtype]).double()
        every = every[every.isfinite()].numpy()
        blocks.append(every[: len(every) // 128 * 128].reshape(-1, 128))
    X = torch.from_numpy(np.concatenate(blocks)).to(DTYPES[dtype])
    announce(f"quantize {kind} {dtype}")
    want = f8.encode(X.double().numpy(), kind)
    for got in (rt.quantize_f8(X.cuda(), TYPES[kind]), rt.quantize_f8(X.t().contiguous().cuda(), TYPES[kind], transpose=True)):
        codes, scales = host(got)
        assert np.array_equal(scales, want[1])
        assert np.array_equal(codes, want[0])


def test_quantize_f32_at_random_is_the_nearest_code():
    """Many quotients: a division that is off in its last place would show at the borders."""
    gen = torch.Generator(device="cuda").manual_seed(1)
    X = torch.randn(4096, 1024, device="cuda", generator=gen)
    Q = rt.quantize_f8(X)
    s = Q.scales.double().repeat_interleave(128, 1)
    y = X.double() / s
    step = torch.exp2((torch.frexp(y).exponent - 1).clamp(min=-6).double() - 3)
    want = (torch.round(y / step) * step).clamp(-448, 448)
    assert torch.equal(Q.codes.float().double(), want)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("block_rows,transpose", [(1, False), (128, False), (1, True)])
def test_quantize_blocks_with_nan_and_infinity(kind, block_rows, transpose):
    rng = np.random.default_rng(4)
    x = rng.standard_normal((300, 270))
    x[1, 40], x[130, 200], x[299, 0], x[200, 269] = np.nan, np.inf, -np.inf, np.nan
    X = torch.from_numpy(x).float()
    Q = rt.quantize_f8(X.cuda(), TYPES[kind], block_rows=block_rows, transpose=transpose)
    want = f8.encode((X.t() if transpose else X).double().numpy(), kind, block_rows)
    codes, scales = host(Q)
    assert np.array_equal(scales, want[1], equal_nan=True) and np.array_equal(codes, want[0])
    assert np.isnan(scales).sum() == 4 and bool(rt.dequantize_f8(Q).isnan().any())


SIZES = [(1, 1), (1, 127), (3, 7), (5, 128), (2, 129), (7, 64), (33, 777), (257, 513), (130, 1000), (1, 8192), (129, 1040)]


@pytest.mark.parametrize("rows,cols", SIZES)
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("block_rows,transpose", [(1, False), (128, False), (1, True)])
def test_conversions_touch_their_rows_only(dtype, block_rows, transpose, rows, cols):
    rng = np.random.default_rng(rows * 1000 + cols)
    kind = KINDS[cols % 2]
    X = torch.from_numpy(rng.standard_normal((rows, cols))).to(DTYPES[dtype])
    want = f8.encode((X.t() if transpose else X).double().numpy(), kind, block_rows)
    q_rows, q_cols = want[0].shape
    for pad in (0, 3, 16):  # tight rows; odd ones; aligned ones
        x = torch.full((rows, cols + 2 * pad), float("nan"), dtype=DTYPES[dtype], device="cuda")
        x[:, pad:pad + cols] = X.cuda()
        full = torch.full((q_rows, q_cols + 2 * pad), 0xA5, dtype=torch.uint8, device="cuda")
        srows, scols = want[1].shape
        sfull = torch.full((srows + 2, scols + 2), -5.0, device="cuda")
        out = rt.F8Matrix(full[:, pad:pad + q_cols].view(TYPES[kind]), sfull[1:1 + srows, 1:1 + scols], block_rows)
        announce(f"quantize {kind} {dtype} {rows}x{cols} pad {pad} blocks of {block_rows} transpose {transpose}")
        got = rt.quantize_f8(x[:, pad:pad + cols], TYPES[kind], block_rows=block_rows, transpose=transpose, out=out)
        assert got is out
        codes, scales = host(out)
        assert np.array_equal(scales, want[1]) and np.array_equal(codes, want[0])
        around = full.clone()
        around[:, pad:pad + q_cols] = 0xA5
        assert bool((around == 0xA5).all())
        saround = sfull.clone()
        saround[1:1 + srows, 1:1 + scols] = -5.0
        assert bool((saround == -5.0).all())
        back = torch.full((q_rows, q_cols + 2 * pad), 9.0, dtype=DTYPES[dtype], device="cuda")
        rt.dequantize_f8(out, out=back[:, pad:pad + q_cols])
        value = torch.from_numpy(f8.decode_table(kind)[codes].astype(np.float32) * scales[np.arange(q_rows) // block_rows].repeat(128, 1)[:, :q_cols])
        assert torch.equal(back[:, pad:pad + q_cols].cpu(), value.to(DTYPES[dtype]))
        back[:, pad:pad + q_cols] = 9.0
        assert bool((back == 9.0).all())
    assert torch.equal(rt.dequantize_f8(out.t(), dtype=DTYPES[dtype]), rt.dequantize_f8(out, dtype=DTYPES[dtype]).t())


@pytest.mark.parametrize("block_rows,transpose", [(1, False), (128, False), (1, True)])
def test_quantize_takes_rows_by_number(block_rows, transpose):
    rng = np.random.default_rng(5)
    X = torch.from_numpy(rng.standard_normal((50, 200))).float()
    index = rng.integers(0, 50, 333).astype(np.int32)
    index[[3, 100, 101, 332]] = [-1, 50, 2**31 - 1, -7]  # no rows of X: zeros
    there = (index >= 0) & (index < 50)
    x = np.where(there[:, None], X.double().numpy()[np.where(there, index, 0)], 0.0)
    want = f8.encode(x.T if transpose else x, f8.E4M3, block_rows)
    codes, scales = host(rt.quantize_f8(X.cuda(), block_rows=block_rows, transpose=transpose, rows=torch.from_numpy(index).cuda()))
    assert np.array_equal(scales, want[1]) and np.array_equal(codes, want[0])
    none = rt.quantize_f8(X.cuda(), rows=torch.empty(0, dtype=torch.int32, device="cuda"))
    assert none.shape == (0, 200)


def test_quantize_more_rows_than_a_grid_holds():
    """Row groups and column tiles past the launch's caps are reached by the kernels' strides."""
    X = torch.randn(2**20 + 5, 8, device="cuda", dtype=torch.bfloat16)
    Q = rt.quantize_f8(X)
    top = X.float().abs().amax(1) * (torch.ones((), device="cuda") / 448)
    assert torch.equal(Q.scales[:, 0], top.clamp(min=2.0**-126))
    assert torch.equal(rt.dequantize_f8(Q, dtype=torch.float32), Q.codes.float() * Q.scales)


# ---- products ------------------------------------------------------------------------------
def products(rng, M, N, K, ka, kb, order, b_block=128):
    """(A, B as op, ref, mag) with A M x K in `order[0]` storage and B in `order[1]`."""
    def side(rows_are_k, n, kind, block):
        rows, cols = (K, n) if rows_are_k else (n, K)
        codes, scales = random_matrix(rng, rows, cols, kind, block)
        v = f8.decode(codes, scales, kind, block)
        return codes, scales, v.T if rows_are_k else v

    a = side(order[0] == "t", M, ka, 128 if order[0] == "t" else 1)
    b = side(order[1] == "n", N, kb, b_block)
    ref = a[2] @ b[2].T
    mag = np.abs(a[2]) @ np.abs(b[2]).T
    return a[:2], b[:2], ref, mag


def on_device(codes, scales, kind, block, transposed, layout="aligned", order="columns"):
    m = device_matrix(codes, scales, kind, block, layout, order)
    return m.t() if transposed else m


def check(M, N, K, ka=f8.E4M3, kb=f8.E4M3, order="nt", b_block=128, dtype="f32", layout="aligned", s_order="columns", alpha=1.0, beta=0.0, seed=0):
    rng = np.random.default_rng(seed + M * 7 + N * 3 + K)
    a, b, ref, mag = products(rng, M, N, K, ka, kb, order, b_block)
    A = on_device(*a, ka, 128 if order[0] == "t" else 1, order[0] == "t", layout, s_order)
    B = on_device(*b, kb, b_block, order[1] == "t", layout, s_order)
    what = f"{order} {M}x{N}x{K} {ka} {kb} b_block {b_block} {dtype} {layout} {s_order} alpha {alpha} beta {beta}"
    announce(what)
    full = torch.full((M + 2, N + 3), float("nan"), dtype=DTYPES[dtype], device="cuda")
    C = full[1:1 + M, 1:1 + N] if layout == "odd" else torch.full((M, N), float("nan"), dtype=DTYPES[dtype], device="cuda")
    ref, mag = alpha * ref, abs(alpha) * mag
    if beta:
        C.copy_(torch.from_numpy(rng.standard_normal((M, N))))
        c = C.double().cpu().numpy()
        ref, mag = ref + beta * c, mag + np.abs(beta * c)
    got = rt.gemm_f8(A, B, C, alpha=alpha, beta=beta)
    assert got is C
    assert_close(C, ref, mag, what)
    if layout == "odd":
        C.fill_(float("nan"))
        assert bool(full.isnan().all())
    return rt.last_kernel()


SHAPES = [(1, 1, 1), (1, 16, 128), (1, 4096, 1024), (3, 100, 130), (16, 256, 512), (17, 300, 1000), (64, 64, 127), (64, 1024, 129), (100, 1500, 777),
          (128, 128, 128), (129, 257, 384), (256, 256, 640), (257, 500, 1300), (300, 129, 2048)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("order,b_block", [("nt", 128), ("nt", 1), ("nn", 128), ("tt", 128), ("tn", 128)])
def test_products(M, N, K, order, b_block):
    for i, (dtype, layout) in enumerate((("f32", "aligned"), ("bf16", "aligned"), ("f16", "odd"), ("f32", "tight"))):
        check(M, N, K, KINDS[(M + i) % 2], KINDS[0], order, b_block, dtype, layout, "columns" if i % 2 == 0 else "rows",
              alpha=(1.0, 0.5, -1.5, 1.0)[i], beta=(0.0, 1.0, 0.5, 0.0)[i])


@pytest.mark.parametrize("ka", KINDS)
@pytest.mark.parametrize("kb", KINDS)
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_types(ka, kb, dtype):
    for M, N, K in ((5, 130, 300), (200, 300, 520), (300, 520, 1024)):
        check(M, N, K, ka, kb, "nt", 128, dtype)
        check(M, N, K, ka, kb, "nt", 1, dtype)
        check(M, N, K, ka, kb, "nn", 128, dtype)


LARGE = [(1024, 1024, 512), (2048, 1000, 1111), (1000, 4096, 256), (513, 2049, 1537), (64, 8192, 2048), (200, 2048, 8192), (2, 777, 9000)]


@pytest.mark.parametrize("M,N,K", LARGE)
@pytest.mark.parametrize("order,b_block", [("nt", 128), ("nt", 1), ("nn", 128)])
def test_large_products(M, N, K, order, b_block):
    check(M, N, K, f8.E5M2 if order == "nn" else f8.E4M3, f8.E4M3, order, b_block, "bf16")
    check(M, N, K, f8.E4M3, f8.E4M3, order, b_block, "f32", beta=1.0)


@pytest.mark.parametrize("order,b_block", [("nt", 128), ("nt", 1), ("nn", 128)])
@pytest.mark.parametrize("M", [1, 40, 300])
def test_nan_scales_and_codes_stay_in_their_rows_and_columns(order, b_block, M):
    """A NaN (infinite) code or a NaN scale makes exactly the outputs of its row, column or block NaN."""
    N, K = 300, 530
    rng = np.random.default_rng(6)
    a, b, _, _ = products(rng, M, N, K, f8.E5M2, f8.E4M3, order, b_block)
    a[0][M - 1, 529] = 0x7C  # infinity, in the last, short block
    a[0][0, 3] = 0x7E        # NaN
    b[0][(529, 7) if order == "nn" else (7, 529)] = 0x7F
    b[1][-1, 0] = np.nan
    A, B = on_device(*a, f8.E5M2, 1, False), on_device(*b, f8.E4M3, b_block, order == "nt")
    va, vb = f8.decode(*a, f8.E5M2), f8.decode(*b, f8.E4M3, b_block)
    with np.errstate(invalid="ignore"):
        ref = va @ (vb if order == "nn" else vb.T)
    for dtype in (torch.float32, torch.bfloat16):
        got = rt.gemm_f8(A, B, dtype=dtype).cpu().double().numpy()
        assert np.array_equal(np.isnan(got), np.isnan(ref)) and np.array_equal(np.isinf(got), np.isinf(ref))


def test_beta_zero_never_reads_C_and_alpha_zero_never_reads_the_operands():
    rng = np.random.default_rng(7)
    a, b, ref, mag = products(rng, 40, 200, 256, f8.E4M3, f8.E4M3, "nt")
    A, B = on_device(*a, f8.E4M3, 1, False), on_device(*b, f8.E4M3, 128, True)
    C = torch.full((40, 200), float("nan"), device="cuda")
    assert_close(rt.gemm_f8(A, B, C), ref, mag, "C of NaN")
    bad = rt.F8Matrix(device_codes(np.full((40, 256), 0x7F, np.uint8), f8.E4M3), device_scales(np.full((40, 2), np.nan, np.float32)))
    C = torch.ones(40, 200, device="cuda")
    assert bool((rt.gemm_f8(bad, B, C, alpha=0.0, beta=2.0) == 2.0).all())
    assert bool((rt.gemm_f8(bad, B, alpha=0.0) == 0.0).all())
    a, b, _, _ = products(rng, 700, 300, 257, f8.E4M3, f8.E4M3, "nt")  # more rows than go straight to registers, unaligned
    C = torch.ones(700, 300, device="cuda", dtype=torch.bfloat16)
    rt.gemm_f8(on_device(*a, f8.E4M3, 1, False, "tight"), on_device(*b, f8.E4M3, 128, True, "tight"), C, alpha=0.0, beta=-3.0)
    assert bool((C == -3.0).all())


@pytest.mark.parametrize("M,N,K", [(0, 5, 128), (5, 0, 128), (5, 7, 0), (0, 0, 0), (300, 513, 0), (0, 300, 1024)])
def test_empty(M, N, K):
    e = torch.float8_e4m3fn

    def empty(r, c, block=1):
        return rt.F8Matrix(torch.empty(r, c, dtype=torch.uint8, device="cuda").view(e), torch.empty(-(-r // block), f8.blocks(c), device="cuda"), block)

    C = rt.gemm_f8(empty(M, K), empty(N, K, 128).t(), torch.ones(M, N, device="cuda"), beta=3.0)
    assert C.shape == (M, N) and bool((C == 3.0).all())
    assert bool((rt.gemm_f8(empty(M, K), empty(N, K, 128).t(), dtype=torch.bfloat16) == 0).all())
    for r, c in ((0, 5), (5, 0)):
        X = torch.empty(r, c, device="cuda")
        for t in (False, True):
            Q = rt.quantize_f8(X, transpose=t)
            assert rt.dequantize_f8(Q).shape == ((c, r) if t else (r, c))


def test_refusals_on_the_device():
    X = torch.randn(40, 256, device="cuda")
    x, W = rt.quantize_f8(X), rt.quantize_f8(torch.randn(200, 256, device="cuda"), block_rows=128)
    for args, match in (((x.t(), x), "must run along k"), ((x, rt.quantize_f8(torch.randn(256, 50, device="cuda"))), "must run along k"),
                        ((x, W), "inner dimensions"), ((x, W.t(), torch.empty(40, 201, device="cuda")), "C must be"),
                        ((x, W.t(), torch.empty(40, 200, device="cuda").t().contiguous().t()), "row-major")):
        with pytest.raises(ValueError, match=match):
            rt.gemm_f8(*args)
    with pytest.raises(ValueError, match="beta"):
        rt.gemm_f8(x, W.t(), beta=1.0)
    with pytest.raises(ValueError, match="dtype must be"):
        rt.gemm_f8(x, W.t(), dtype=torch.float64)
    with pytest.raises(ValueError, match="block_rows"):
        rt.quantize_f8(X, block_rows=128, transpose=True)
    with pytest.raises(ValueError, match="out must be"):
        rt.quantize_f8(X, out=W)
    with pytest.raises(ValueError, match="int32"):
        rt.quantize_f8(X, rows=torch.zeros(3, dtype=torch.int64, device="cuda"))


def test_same_bits_every_time():
    for M, N, K in ((1, 4096, 4096), (48, 1024, 4096), (300, 700, 5000), (1024, 1024, 1024)):
        rng = np.random.default_rng(8)
        A = device_matrix(*random_matrix(rng, M, K), f8.E4M3)
        W = device_matrix(*random_matrix(rng, N, K, block_rows=128), f8.E4M3, 128)
        for dtype in (torch.float32, torch.bfloat16):
            first = rt.gemm_f8(A, W.t(), dtype=dtype)
            for _ in range(3):
                assert torch.equal(first, rt.gemm_f8(A, W.t(), dtype=dtype))


def test_another_stream_and_two_at_once():
    rng = np.random.default_rng(9)
    M, N, K = 200, 512, 4096
    a, b, ref, mag = products(rng, M, N, K, f8.E4M3, f8.E4M3, "nt")
    A, B = on_device(*a, f8.E4M3, 1, False), on_device(*b, f8.E4M3, 128, True)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    out = [rt.gemm_f8(A, B, stream=streams[i % 2]) for i in range(8)]
    out.append(rt.gemm_f8(A, B, stream=streams[0].cuda_stream))
    torch.cuda.synchronize()
    for C in out:
        assert_close(C, ref, mag, "streams")


def test_captured_layer():
    """The three products of a layer and the conversions that they need, captured and replayed on new inputs."""
    gen = torch.Generator(device="cuda").manual_seed(2)
    M, N, K = 70, 260, 640
    x, W, dy = (torch.empty(*s, device="cuda", dtype=torch.bfloat16) for s in ((M, K), (N, K), (M, N)))

    def layer():
        w = rt.quantize_f8(W, block_rows=128)
        y = rt.gemm_f8(rt.quantize_f8(x), w.t(), dtype=torch.bfloat16)
        dx = rt.gemm_f8(rt.quantize_f8(dy, torch.float8_e5m2), w, dtype=torch.bfloat16)
        dW = rt.gemm_f8(rt.quantize_f8(dy, torch.float8_e5m2, transpose=True), rt.quantize_f8(x, transpose=True).t())
        return y, dx, dW

    def fill():
        x.copy_(torch.randn(M, K, device="cuda", generator=gen))
        W.copy_(torch.randn(N, K, device="cuda", generator=gen) * K**-0.5)
        dy.copy_(torch.randn(M, N, device="cuda", generator=gen) * 1e-3)

    fill()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = layer()
    for _ in range(4):
        fill()
        graph.replay()
        torch.cuda.synchronize()
        for got, want in zip(held, layer()):
            assert torch.equal(got, want)


def test_linear_layer():
    """y, dx and dW of a layer against 64-bit products of the values that the operands are held as, and those against the
    unrounded ones: a code is off by half a step, 2^-4 (e4m3) or 2^-3 (e5m2) of its value, so a product by at most
    2^-4 + 2^-4 + 2^-8 or 2^-3 + 2^-4 + 2^-7 of the sum of magnitudes (subnormal codes: less than 2^-8 of a block's
    largest, bounded by the same sums of a matrix with those added)."""
    gen = torch.Generator(device="cuda").manual_seed(3)
    M, N, K = 384, 260, 650
    x, W = torch.randn(M, K, device="cuda", generator=gen), torch.randn(N, K, device="cuda", generator=gen) * K**-0.5
    dy = torch.randn(M, N, device="cuda", generator=gen) * 1e-3
    w = rt.quantize_f8(W, block_rows=128)
    ops = {"y": (rt.quantize_f8(x), w.t(), x, W.t(), 2.0**-3 + 2.0**-8),
           "dx": (rt.quantize_f8(dy, torch.float8_e5m2), w, dy, W, 2.0**-3 + 2.0**-4 + 2.0**-7),
           "dW": (rt.quantize_f8(dy, torch.float8_e5m2, transpose=True), rt.quantize_f8(x, transpose=True).t(), dy.t(), x, 2.0**-3 + 2.0**-4 + 2.0**-7)}
    for name, (A, B, a, b, rel) in ops.items():
        C = rt.gemm_f8(A, B)
        va, vb = (rt.dequantize_f8(m, dtype=torch.float32).double().cpu().numpy() for m in (A, B))
        assert_close(C, va @ vb, np.abs(va) @ np.abs(vb), name)
        a, b = a.double().cpu().numpy(), b.double().cpu().numpy()
        floor_a, floor_b = 2.0**-8 * np.abs(a).max(), 2.0**-8 * np.abs(b).max()
        mag = (np.abs(a) + floor_a) @ (np.abs(b) + floor_b)
        assert (np.abs(C.double().cpu().numpy() - a @ b) <= rel * mag).all()
