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


def dev_rows(x, row, fill):
    """`x` on the GPU with rows that start `row` elements apart, `fill` behind them."""
    x = torch.as_tensor(x)
    full = torch.full((x.shape[0], row), fill, dtype=x.dtype, device="cuda")
    full[:, :x.shape[1]] = x.cuda()
    return full[:, :x.shape[1]]


def random_matrix(rng, fmt, rows, cols, aligned=True):
    """(MXMatrix, its values in 64 bits on the GPU); rows aligned for DMA, or close together."""
    w, g = mx.widths(fmt, cols)
    codes = rng.integers(0, 256, (rows, w), dtype=np.uint8)
    scales = rng.integers(120, 131, (rows, g)).astype(np.uint8)
    B = rt.MXMatrix(fmt, dev_rows(codes, -(-w // 16) * 16 if aligned else w, 255),
                    dev_rows(scales, -(-g // 4) * 4 if aligned else g, 255), cols)
    return B, torch.from_numpy(mx.decode(codes, scales, fmt, cols)).cuda()


def assert_close(C, a, b, what, alpha=1.0, beta=0.0, C0=None):
    """Within 1e-5 of the sum of the magnitudes that an output is made of: the library's bound for fp32 sums
    of exact products. a and b are in 64 bits."""
    a, b = a.contiguous(), b.contiguous()
    ref, mag = alpha * (a @ b), abs(alpha) * (a.abs() @ b.abs())
    if beta:
        ref, mag = ref + beta * C0.double(), mag + (beta * C0.double()).abs()
    assert bool(C.isfinite().all()), what
    worst = ((C.double() - ref).abs() / (1e-5 * mag).clamp(min=1e-30)).max()
    assert float(worst) <= 1.0, f"{what}: |err| / bound {float(worst):.3g}"


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


@pytest.mark.parametrize("fmt,order", [(mx.FP4, "nt"), (mx.INT8, "nt"), (mx.INT8, "nn")])
def test_long_k_on_rows_too_far_apart_for_wide_tiles(fmt, order):
    """256 rows of A pass 2^31 bytes, and what lies behind each of them is NaN."""
    M, N, K, lda = 300, 8448, 8288, 5 * 2**20
    if torch.cuda.mem_get_info()[0] < 20 << 30:
        pytest.skip("needs 20 GB of free memory")
    rng = np.random.default_rng(11)
    A = dev_rows(torch.from_numpy(rng.standard_normal((M, K))).bfloat16(), lda, float("nan"))
    B, b = random_matrix(rng, fmt, *((N, K) if order[1] == "t" else (K, N)))
    announce(f"gemm_mx {fmt} {order} {M}x{N}x{K} lda {lda}")
    C = rt.gemm_bf16_mx(A, B.t() if order[1] == "t" else B)
    assert "_dma_128x128" in rt.last_kernel(), rt.last_kernel()
    assert_close(C, A.double(), b.t() if order[1] == "t" else b, "far rows")


def test_handle_of_the_default_stream():
    """Handle 0 is the default stream, as in the other entry points: work queued there before a call has run
    before it, work queued after it waits for it."""
    default = torch.cuda.default_stream()
    assert default.cuda_stream == 0
    with rt._Launch(torch.device("cuda", 0), 0) as handle:
        assert handle == 0 and torch.cuda.current_stream() == default
    spin = torch.randn(4096, 4096, device="cuda")
    x = torch.zeros(64, 2048, device="cuda", dtype=torch.bfloat16)
    W = rt.quantize_mx(torch.randn(512, 2048, device="cuda"), rt.MX_FP4)
    new = torch.randn(64, 2048, device="cuda", dtype=torch.bfloat16)
    want, kept = rt.gemm_bf16_mx(new, W.t()), rt.quantize_mx(new, rt.MX_INT8)
    back = rt.dequantize_mx(kept)
    torch.cuda.synchronize()
    for _ in range(4):
        x.zero_()
        for _ in range(8):
            spin = spin @ spin * 1e-3  # keeps the default stream busy while the calls below are queued
        x.copy_(new)
        y = rt.gemm_bf16_mx(x, W.t(), stream=0).clone()
        q = rt.quantize_mx(x, rt.MX_INT8, stream=0)
        d = rt.dequantize_mx(q, stream=0).clone()
        torch.cuda.synchronize()
        assert torch.equal(y, want) and torch.equal(d, back)
        assert torch.equal(q.codes, kept.codes) and torch.equal(q.scales, kept.scales)


def run_with_workspace(dtype, A, B, C, alpha, beta, work, parts):
    """The C call with a workspace of `parts` M x N parts at the start of `work` (0: none)."""
    ta = A.stride(0) == 1 and A.shape[0] > 1
    (M, K), N = A.shape, B.shape[1]
    fn = rt.regtile_gemm_bf16_mx if dtype == torch.bfloat16 else rt.regtile_gemm_f16_mx
    assert fn(B.format, int(ta), int(B.transposed), M, N, K, alpha, A.data_ptr(), A.stride(1 if ta else 0), B.codes.data_ptr(),
              B.codes.stride(0), B.scales.data_ptr(), B.scales.stride(0), beta, C.data_ptr(), C.stride(0),
              work.data_ptr() if parts else 0, parts * M * N * 4, torch.cuda.current_stream().cuda_stream) == 0


# (M, N, K, tile, parts): the last part shorter than the others in both
@pytest.mark.parametrize("M,N,K,tile,parts", [(1000, 1000, 129 * 128, 128, 8), (1040, 1824, 65 * 128, 256, 6)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_codes_in_lds_in_parts_of_k(dtype, M, N, K, tile, parts):
    """K split over workgroups where B stays in codes in LDS: the parts that the binding asks for, fewer (which
    256-wide tiles do not make), and none."""
    rng = np.random.default_rng(M + N)
    A = torch.from_numpy(rng.standard_normal((M, K))).to(dtype).cuda()
    B, b = random_matrix(rng, mx.FP4, N, K)
    C0 = torch.randn(M, N + 4, device="cuda")
    announce(f"gemm_mx fp4 nt {M}x{N}x{K} {dtype} in parts")
    assert rt.regtile_gemm_mx_workspace(0, 1, M, N, K, K, N + 4) == parts * M * N * 4
    gemm = rt.gemm_bf16_mx if dtype == torch.bfloat16 else rt.gemm_f16_mx
    full = C0.clone()
    C = gemm(A, B.t(), full[:, :N], alpha=-0.5, beta=2.0)
    assert f"_codes_{tile}x{tile}" in rt.last_kernel(), rt.last_kernel()
    assert torch.equal(full[:, N:], C0[:, N:])
    a = A.double()
    assert_close(C, a, b.t(), "binding", -0.5, 2.0, C0[:, :N])
    work = torch.empty(parts * M * N + 64, device="cuda")
    for n in (0, 1, 3, parts):
        work.fill_(float("nan"))
        D = C0[:, :N].contiguous()
        run_with_workspace(dtype, A, B.t(), D, -0.5, 2.0, work, n)
        narrow = tile == 128 or n < parts
        assert ("_codes_128x128" if narrow else "_codes_256x256") in rt.last_kernel(), (n, rt.last_kernel())
        assert_close(D, a, b.t(), f"{n} parts", -0.5, 2.0, C0[:, :N])
        assert bool(work[max(n, 1) * M * N:].isnan().all())
        if n == parts:
            assert torch.equal(D, C)


def workspace_of(A, B, ldc):
    """regtile_gemm_mx_workspace_ex of a product's operands."""
    ta = A.stride(0) == 1 and A.shape[0] > 1
    (M, K), N = A.shape, B.shape[1]
    return rt.regtile_gemm_mx_workspace_ex(B.format, int(ta), int(B.transposed), M, N, K, A.data_ptr(), A.stride(1 if ta else 0),
                                           B.codes.data_ptr(), B.codes.stride(0), B.scales.data_ptr(), B.scales.stride(0), ldc)


# (order, M, N, K, rows of codes and scales aligned): few rows of A, 64-wide tiles' sizes on rows that are not
# aligned for them (90 and 91 scale bytes), and those that split nothing
IN_PARTS = [("nn", 1, 1024, 4096, True, 8), ("nn", 16, 1024, 8320, False, 15), ("tn", 16, 1024, 4160, True, 8), ("tt", 48, 520, 2880, False, 5),
            ("nt", 48, 600, 2880, False, 5), ("nt", 256, 1024, 2880, False, 5), ("nt", 130, 264, 2912, False, 5),
            ("nt", 48, 600, 2944, True, 0), ("nt", 16, 600, 2880, False, 0), ("nt", 256, 4096, 1024, True, 0)]


@pytest.mark.parametrize("order,M,N,K,aligned,parts", IN_PARTS)
@pytest.mark.parametrize("fmt", [mx.FP4, mx.INT8])
def test_workspace_query_is_what_a_call_uses(fmt, order, M, N, K, aligned, parts):
    rng = np.random.default_rng(M + N + K)
    ta, tb = order[0] == "t", order[1] == "t"
    A = torch.from_numpy(rng.standard_normal((K, M) if ta else (M, K))).bfloat16().cuda()
    A = A.t() if ta else A
    B, b = random_matrix(rng, fmt, *((N, K) if tb else (K, N)), aligned)
    B, b = (B.t(), b.t()) if tb else (B, b)
    size = workspace_of(A, B, N)
    assert size % (4 * M * N) == 0
    n = size // (4 * M * N)
    assert n == parts
    for given in {n, n + 3}:
        work = torch.full(((n + 3) * M * N,), float("nan"), device="cuda")
        C = torch.empty(M, N, device="cuda")
        announce(f"gemm_mx {fmt} {order} {M}x{N}x{K}, workspace of {given} parts")
        run_with_workspace(torch.bfloat16, A, B, C, 1.0, 0.0, work, given)
        assert_close(C, A.double(), b, rt.last_kernel())
        assert bool(work[:n * M * N].isfinite().all()) and bool(work[n * M * N:].isnan().all())


class Spy:
    """The library, with the last workspace that a product was given on record."""

    def __init__(self, lib):
        self.lib, self.given = lib, None

    def __getattr__(self, name):
        f = getattr(self.lib, name)
        if name not in ("regtile_gemm_bf16_mx", "regtile_gemm_f16_mx"):
            return f

        def call(*args):
            self.given = args[17]
            return f(*args)

        return call


@pytest.mark.parametrize("order,M,N,K,aligned,parts", IN_PARTS + [
    ("nn", 16, 8192, 8192, True, 8), ("nn", 64, 4096, 4096, True, 8), ("tn", 16, 4096, 8192, True, 16), ("nt", 33, 2880, 2880, False, 5),
    ("nt", 64, 600, 2944, True, 0), ("nt", 32, 600, 2880, False, 0), ("nn", 64, 1024, 1000, True, 0), ("tn", 300, 512, 2048, True, 0), ("tn", 304, 512, 2048, True, 4)])
@pytest.mark.parametrize("fmt", [mx.FP4, mx.INT8])
def test_binding_gives_each_call_its_workspace(monkeypatch, fmt, order, M, N, K, aligned, parts):
    """dx and dW of a few rows among them: K in parts, as the library's query says, and the same bits as the C
    call with that workspace."""
    rng = np.random.default_rng(M + N + K)
    ta, tb = order[0] == "t", order[1] == "t"
    A = torch.from_numpy(rng.standard_normal((K, M) if ta else (M, K))).bfloat16().cuda()
    A = A.t() if ta else A
    B, b = random_matrix(rng, fmt, *((N, K) if tb else (K, N)), aligned)
    B, b = (B.t(), b.t()) if tb else (B, b)
    spy = Spy(rt.load())
    monkeypatch.setattr(rt, "_lib", spy)
    announce(f"gemm_mx {fmt} {order} {M}x{N}x{K}, the binding's workspace")
    C = rt.gemm_bf16_mx(A, B)
    assert spy.given == workspace_of(A, B, N) == parts * M * N * 4, spy.given
    assert_close(C, A.double(), b, rt.last_kernel())
    D = torch.empty_like(C)
    run_with_workspace(torch.bfloat16, A, B, D, 1.0, 0.0, torch.empty(parts * M * N + 4, device="cuda"), parts)
    assert torch.equal(C, D)


def test_binding_and_misaligned_rows(monkeypatch):
    """33 to 64 rows whose codes or scales start off the alignment of the token kernel."""
    rng = np.random.default_rng(12)
    M, N, K = 48, 600, 2944
    A = torch.from_numpy(rng.standard_normal((M, K))).bfloat16().cuda()
    w, g = mx.widths(mx.INT8, K)
    codes = rng.integers(0, 256, (N, w), dtype=np.uint8)
    scales = rng.integers(120, 131, (N, g)).astype(np.uint8)
    b = torch.from_numpy(mx.decode(codes, scales, mx.INT8, K)).cuda().t()
    spy = Spy(rt.load())
    monkeypatch.setattr(rt, "_lib", spy)
    for q_off, s_off, parts in ((0, 0, 0), (16, 4, 0), (8, 0, 5), (0, 1, 5)):
        Q = dev_rows(np.pad(codes, ((0, 0), (q_off, 0))), w + 16, 255)[:, q_off:]
        S = dev_rows(np.pad(scales, ((0, 0), (s_off, 0))), g + 4, 255)[:, s_off:]
        B = rt.MXMatrix(mx.INT8, Q, S, K).t()
        C = rt.gemm_bf16_mx(A, B)
        assert spy.given == workspace_of(A, B, N) == parts * M * N * 4, (q_off, s_off, spy.given)
        assert_close(C, A.double(), b, rt.last_kernel())


def test_graph_of_few_rows_with_workspaces():
    """dx and dW of a few rows, each with a workspace, captured one after the other: every replay on new inputs
    gives the eager calls' bits, with eager calls of other sizes between the replays."""
    M, I, O = 16, 1024, 2048
    W = rt.quantize_mx(torch.randn(O, I, device="cuda"), rt.MX_FP4)
    kept = rt.quantize_mx(torch.randn(O, I, device="cuda", dtype=torch.bfloat16), rt.MX_INT8)
    dy = torch.empty(M, O, device="cuda", dtype=torch.bfloat16)
    dz = torch.empty(O, M, device="cuda", dtype=torch.float16)
    acc = torch.zeros(M, I, device="cuda")
    assert workspace_of(dy, W, I) > 0 and workspace_of(dz.t(), kept, I) > 0

    def step():
        dx = rt.gemm_bf16_mx(dy, W)
        dw = rt.gemm_f16_mx(dz.t(), kept)
        rt.gemm_f16_mx(dz.t(), kept, acc, alpha=0.5, beta=1.0)
        return dx, dw, rt.gemm_bf16_mx(dy[:3], W)

    side = torch.cuda.Stream()
    dy.normal_(), dz.normal_()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for version in range(4):
        dy.normal_(), dz.normal_(), acc.normal_()
        before = acc.clone()
        eager = [t.clone() for t in step()]
        after = acc.clone()
        acc.copy_(before)
        rt.gemm_bf16_mx(dy[:9], W)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(acc, after), version
        for o, e in zip(outs, eager):
            assert torch.equal(o, e), version


def test_few_rows_on_two_streams_at_once():
    """Calls of few rows that use workspaces, running together on two streams: the results are those of one."""
    W = rt.quantize_mx(torch.randn(4096, 1024, device="cuda"), rt.MX_FP4)
    dy = [torch.randn(16, 4096, device="cuda", dtype=torch.bfloat16) for _ in range(2)]
    want = [rt.gemm_bf16_mx(d, W) for d in dy]
    torch.cuda.synchronize()
    streams, outs = [torch.cuda.Stream() for _ in range(2)], [[], []]
    for i in range(40):
        with torch.cuda.stream(streams[i % 2]):
            outs[i % 2].append(rt.gemm_bf16_mx(dy[i % 2], W))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(o, want[i]) for o in outs[i])
