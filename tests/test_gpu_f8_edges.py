"""8-bit float products where sizes, strides, workspaces and streams are unusual: every kernel that a product can
take, operands and outputs past 2^31 bytes, workspaces of every size, graphs that are replayed in turn."""
from __future__ import annotations

import pytest

import f8_reference as f8
import register_tiled_matrix_amd as rt
from gpu_util import announce

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

E4, E5 = torch.float8_e4m3fn, torch.float8_e5m2


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    rt.load()
    yield
    torch.cuda.empty_cache()


def make(gen, rows, cols, block=1, kind=E4, tight=False, by_rows=False):
    Q = rt.quantize_f8(torch.randn(rows, cols, device="cuda", generator=gen), kind, block_rows=block)
    codes, scales = Q.codes, Q.scales
    if tight:
        codes = codes.view(torch.uint8).contiguous().view(kind)
    if by_rows:
        scales = scales.contiguous()
    return rt.F8Matrix(codes, scales, block)


def values(Q):
    """64-bit values on the GPU, by the definition."""
    rows, cols = Q.codes.shape[-2:]
    s = Q.scales.double().repeat_interleave(128, -1)[..., :cols]
    if Q.block_rows != 1:
        s = s.repeat_interleave(128, -2)[..., :rows, :]
    v = Q.codes.float().double() * s
    return v.transpose(-1, -2).contiguous() if Q.transposed else v


def assert_close(C, a, b, what, extra=0.0):
    """f8_gpu_util's bounds, on the GPU. extra: what was in C, times beta."""
    if C.numel() == 0:
        return
    ref, mag = a @ b + extra, a.abs() @ b.abs() + abs(extra)
    eight = C.dtype != torch.float32
    limit = (2.0**-12 + 1e-5 if eight else 1e-5) * mag
    if eight:
        limit = limit + torch.finfo(C.dtype).eps / 2 * (ref.abs() + limit) + 2.0**-25
    worst = ((C.double() - ref).abs() / (limit + 1e-37)).max()
    assert float(worst) <= 1.0, f"{what}: |err| / bound {float(worst):.3g}"


KERNELS = [  # M, N, K, C, order, B by columns' scales, tight rows, the kernel
    (3, 500, 1000, torch.bfloat16, "nt", False, True, "f8_token"), (30, 500, 1000, torch.float32, "nt", True, False, "f8_token"),
    (50, 300, 700, torch.bfloat16, "nt", False, False, "f8_token"), (60, 4000, 2001, torch.bfloat16, "nt", False, True, "f8_token"),
    (64, 2048, 8192, torch.bfloat16, "nt", False, False, "f8_tile_64x64"), (500, 500, 5000, torch.float32, "nt", True, True, "f8_tile_64x64_exact"),
    (500, 500, 1000, torch.bfloat16, "nn", False, True, "f8_tile_64x64"), (5, 700, 900, torch.float32, "nn", False, False, "f8_tile_64x64_exact"),
    (1800, 1700, 4200, torch.bfloat16, "nt", True, False, "f8_tile_128x128_deep"), (1800, 1700, 1111, torch.bfloat16, "nn", False, True, "f8_tile_128x128_deep"),
    (1800, 1700, 4200, torch.float32, "nt", False, True, "f8_tile_128x128_exact"), (2600, 2300, 999, torch.float16, "nt", True, False, "f8_tile_128x128"),
    (2600, 2300, 999, torch.float32, "nn", False, False, "f8_tile_128x128_exact"), (3500, 3600, 1000, torch.bfloat16, "nt", False, False, "f8_tile_256x256"),
    (3500, 3601, 1001, torch.bfloat16, "nn", False, True, "f8_tile_256x256")]


@pytest.mark.parametrize("M,N,K,dtype,order,sb,tight,name", KERNELS, ids=lambda v: str(v).replace("torch.", ""))
@pytest.mark.parametrize("kind", [E4, E5])
def test_every_kernel(M, N, K, dtype, order, sb, tight, name, kind):
    gen = torch.Generator(device="cuda").manual_seed(M + N)
    A = make(gen, M, K, kind=kind, tight=tight)
    B = make(gen, N, K, 1 if sb else 128, tight=tight).t() if order == "nt" else make(gen, K, N, 128, tight=tight)
    announce(f"{name} {M}x{N}x{K} {dtype} {order} {kind}")
    C = torch.full((M, N), 2.0, device="cuda", dtype=dtype)
    rt.gemm_f8(A, B, C, beta=-0.5)
    assert rt.last_kernel() == name
    assert_close(C, values(A), values(B), name, extra=-1.0)


def raw(A, B, C, beta, work, size):
    return rt.load().regtile_gemm_f8(int(A.transposed), int(B.transposed), 1.0, A._at, B._at, beta, {torch.float32: 0, torch.bfloat16: 1}[C.dtype],
                                     C.data_ptr(), C.shape[1], work, size, torch.cuda.current_stream().cuda_stream)


@pytest.mark.parametrize("M,N,K,dtype,tight", [(300, 400, 8200, torch.float32, False), (300, 400, 8200, torch.bfloat16, True), (100, 130, 16400, torch.bfloat16, False),
                                               (1800, 1700, 4200, torch.float32, True), (700, 700, 1000, torch.bfloat16, True)])
def test_workspaces_of_every_size(M, N, K, dtype, tight):
    """The whole workspace, parts of it and none: the same product within its bounds, the same bits from the same size, and
    nothing written beside the workspace."""
    gen = torch.Generator(device="cuda").manual_seed(K)
    A, B = make(gen, M, K, tight=tight), make(gen, N, K, 128, tight=tight).t()
    need = rt.load().regtile_gemm_f8_workspace(0, 1, A._at, B._at, {torch.float32: 0, torch.bfloat16: 1}[dtype], N)
    assert need > 0 and need % 4 == 0
    a, b = values(A), values(B)
    for size in (need, need - 16, need // 2 // 16 * 16, 16, 0):
        buf = torch.full((size + 512,), 0xA5, dtype=torch.uint8, device="cuda")
        outs = []
        for _ in range(2):
            C = torch.empty(M, N, device="cuda", dtype=dtype)
            announce(f"workspace {size} of {need}")
            assert raw(A, B, C, 0.0, buf.data_ptr() + 256 if size else None, size) == 0
            outs.append(C)
        assert bool((buf[:256] == 0xA5).all()) and bool((buf[256 + size:] == 0xA5).all())
        assert torch.equal(*outs)
        assert_close(C, a, b, f"workspace {size} of {need}")


@pytest.mark.parametrize("sb", [False, True])
def test_scales_by_rows_or_by_columns_give_the_same_bits(sb):
    """Large enough that scales whose rows are apart are turned first."""
    gen = torch.Generator(device="cuda").manual_seed(3)
    M, N, K = 4000, 4500, 4200
    x, w = torch.randn(M, K, device="cuda", generator=gen), torch.randn(N, K, device="cuda", generator=gen)
    out = []
    for by_rows in (False, True):
        A, B = rt.quantize_f8(x), rt.quantize_f8(w, block_rows=1 if sb else 128)
        if by_rows:
            A, B = (rt.F8Matrix(q.codes, q.scales.contiguous(), q.block_rows) for q in (A, B))
        out.append(rt.gemm_f8(A, B.t(), dtype=torch.bfloat16))
    assert torch.equal(*out)
    at = torch.randint(0, M, (50,), device="cuda", generator=gen)
    assert_close(out[1][at], values(A)[at], values(B.t()), "scales by rows")


def test_broadcast_scales():
    """Strides of 0: one scale for a whole matrix, or for a whole row."""
    gen = torch.Generator(device="cuda").manual_seed(4)
    for M, N, K in ((5, 300, 700), (300, 500, 1000)):
        A, B = make(gen, M, K), make(gen, N, K, 128)
        A = rt.F8Matrix(A.codes, torch.full((1, 1), 0.25, device="cuda").expand(M, f8.blocks(K)))
        B = rt.F8Matrix(B.codes, torch.rand(f8.blocks(N), 1, device="cuda").expand(f8.blocks(N), f8.blocks(K)), 128)
        for dtype in (torch.float32, torch.bfloat16):
            assert_close(rt.gemm_f8(A, B.t(), dtype=dtype), values(A), values(B.t()), "broadcast scales")


def test_rows_too_far_apart_for_32_bits():
    """Rows 8 MB apart (a tile of 256 spans 2 GB): still right, on the kernel that has 64-bit offsets only."""
    gen = torch.Generator(device="cuda").manual_seed(5)
    if torch.cuda.mem_get_info()[0] < 8 << 30:
        pytest.skip("needs 8 GB of free memory")
    M, N, K = 300, 200, 500
    A, B = make(gen, M, K), make(gen, N, K, 128)
    full = torch.zeros(M, 2**23 + 128, dtype=torch.uint8, device="cuda")
    full[:, :K] = A.codes.view(torch.uint8)
    far = rt.F8Matrix(full[:, :K].view(E4), A.scales)
    C = rt.gemm_f8(far, B.t(), dtype=torch.bfloat16)
    assert rt.last_kernel().startswith("f8_any")
    assert_close(C, values(A), values(B.t()), "far rows")


def test_C_past_2_31_elements():
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 24 GB of free memory")
    gen = torch.Generator(device="cuda").manual_seed(6)
    M, N, K = 66000, 33000, 130
    A, B = make(gen, M, K), make(gen, N, K, 128)
    C = rt.gemm_f8(A, B.t(), dtype=torch.bfloat16)
    at = torch.tensor([0, 1, 65072, 65073, M - 2, M - 1], device="cuda")
    assert_close(C[at], values(A)[at], values(B.t()), "large C")


def test_experts_stack_past_2_31_bytes():
    if torch.cuda.mem_get_info()[0] < 16 << 30:
        pytest.skip("needs 16 GB of free memory")
    gen = torch.Generator(device="cuda").manual_seed(7)
    E, N, K = 40, 8192, 8192
    codes = torch.randint(0, 100, (E, N, K), dtype=torch.uint8, device="cuda", generator=gen).view(E4)
    W = rt.F8Matrix(codes, torch.rand(E, 64, 64, device="cuda", generator=gen), 128)
    for T in (3, 300):
        x = make(gen, T, K)
        chosen = torch.randint(0, E, (T, 2), device="cuda", generator=gen).int()
        chosen[0, 0], chosen[T - 1, 1] = E - 1, E - 1
        rows = rt.expert_rows(chosen, E)
        C = rt.gemm_f8_experts(x, W.t(), rows, gather=True, dtype=torch.bfloat16)
        first, n = int(rows.offsets[E - 1]), int(rows.counts[E - 1])
        m = values(x)[rows.slots[first:first + n].long() // 2]
        last = rt.F8Matrix(codes[E - 1], W.scales[E - 1], 128).t()
        assert_close(C[first:first + n], m, values(last), f"the last of a large stack, {T} tokens")


def test_graphs_replayed_in_turn():
    """Two captured products with workspaces, replayed in turn and on two streams at once, with eager work between."""
    gen = torch.Generator(device="cuda").manual_seed(8)
    held, graphs = [], []
    for M, N, K in ((300, 400, 8200), (500, 500, 5001)):
        A, B = make(gen, M, K, tight=True), make(gen, N, K, 128, tight=True).t()
        rt.gemm_f8(A, B)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            C = rt.gemm_f8(A, B)
        held.append((A, B, C))
        graphs.append(g)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for i in range(4):
        for A, B, C in held:
            C.fill_(float("nan"))
            A.codes.view(torch.uint8).copy_(torch.randint(0, 120, A.codes.shape, device="cuda", generator=gen, dtype=torch.uint8))
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            if i % 2:
                with torch.cuda.stream(s):
                    g.replay()
            else:
                g.replay()
        torch.cuda.synchronize()
        for A, B, C in held:
            assert torch.equal(C, rt.gemm_f8(A, B))


def test_millions_of_slots():
    """More slots than 1024 chunks hold: workgroups then take several, and the order is still the stable sort's."""
    gen = torch.Generator(device="cuda").manual_seed(9)
    tokens, k, E = 1_400_001, 3, 37
    chosen = torch.randint(-1, E + 1, (tokens, k), device="cuda", generator=gen).int()
    for align in (1, 128):
        rows = rt.expert_rows(chosen, E, align=align)
        flat = chosen.flatten().long()
        valid = (flat >= 0) & (flat < E)
        key, order = torch.sort(torch.where(valid, flat, E), stable=True)
        counts = torch.bincount(key, minlength=E + 1)[:E]
        room = (counts + align - 1) // align * align
        offsets = torch.cat([torch.zeros(1, device="cuda", dtype=torch.int64), room.cumsum(0)])
        assert torch.equal(rows.counts.long(), counts) and torch.equal(rows.offsets.long(), offsets)
        n = int(counts.sum())
        begin = counts.cumsum(0) - counts
        at = torch.arange(n, device="cuda") - begin[key[:n]] + offsets[key[:n]]
        slots = torch.full((rows.rows,), -1, device="cuda", dtype=torch.int64)
        slots[at] = order[:n]
        position = torch.full((tokens * k,), -1, device="cuda", dtype=torch.int64)
        position[order[:n]] = at
        assert torch.equal(rows.slots.long(), slots) and torch.equal(rows.position.flatten().long(), position)


def test_gathered_rows_of_a_large_unaligned_matrix():
    """Rows whose aligned copy would reach 2^31 bytes, where the matrix itself does not."""
    if torch.cuda.mem_get_info()[0] < 8 << 30:
        pytest.skip("needs 8 GB of free memory")
    gen = torch.Generator(device="cuda").manual_seed(10)
    tokens, K, N, E = 2**20, 2047, 64, 4
    codes = torch.randint(0, 100, (tokens, K), dtype=torch.uint8, device="cuda", generator=gen).view(E4)
    A = rt.F8Matrix(codes, torch.rand(f8.blocks(K), tokens, device="cuda", generator=gen).t())
    W = rt.F8Matrix(torch.randint(0, 100, (E, N, K), dtype=torch.uint8, device="cuda", generator=gen).view(E4),
                    torch.rand(E, 1, f8.blocks(K), device="cuda", generator=gen), 128)
    chosen = torch.full((tokens, 1), -1, device="cuda", dtype=torch.int32)
    taken = torch.cat([torch.arange(300, device="cuda"), torch.arange(tokens - 300, tokens, device="cuda")])
    chosen[taken, 0] = torch.randint(0, E, (600,), device="cuda", generator=gen).int()
    rows = rt.expert_rows(chosen, E)
    C = torch.zeros(rows.rows, N, device="cuda", dtype=torch.bfloat16)
    rt.gemm_f8_experts(A, W.t(), rows, C, gather=True)
    for e in range(E):
        first, n = int(rows.offsets[e]), int(rows.counts[e])
        at = rows.slots[first:first + n].long()
        m = rt.F8Matrix(codes[at], A.scales[at])
        assert_close(C[first:first + n], values(m), values(rt.F8Matrix(W.codes[e], W.scales[e], 128).t()), f"expert {e}")


@pytest.mark.parametrize("M,N,K,name", [(3501, 3603, 400, "f8_tile_256x256"), (2601, 2307, 400, "f8_tile_128x128"), (1800, 1701, 1100, "f8_tile_128x128_deep")])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_ragged_columns_of_an_aligned_C(M, N, K, name, dtype):
    """C's rows are aligned for whole stores and N is not: what lies beside C stays."""
    gen = torch.Generator(device="cuda").manual_seed(N)
    wide_b = name == "f8_tile_128x128"  # (a scale for each column keeps it off the larger tiles)
    A, B = make(gen, M, K), make(gen, N, K, 1 if wide_b else 128).t()
    whole = torch.full((M + 2, (N + 15) // 8 * 8), 7.0, device="cuda", dtype=dtype)
    C = whole[1:-1, :N]
    rt.gemm_f8(A, B, C, alpha=0.5)
    assert rt.last_kernel() == name
    assert_close(C, values(A) * 0.5, values(B), name)
    assert bool((whole[0] == 7).all()) and bool((whole[-1] == 7).all()) and bool((whole[:, N:] == 7).all())


@pytest.mark.parametrize("tokens,k,E,align", [(1500, 2, 8, 1), (3000, 2, 16, 64), (1000, 2, 16, 128)])
def test_ragged_groups_of_an_aligned_C(tokens, k, E, align):
    """Tiles that groups fill in part: rows between groups become 0, rows behind the last and columns beside C stay."""
    gen = torch.Generator(device="cuda").manual_seed(tokens)
    N, K = 2051, 300
    x = make(gen, tokens, K)
    W = [make(gen, N, K, 128) for _ in range(E)]
    stack = rt.F8Matrix(torch.stack([w.codes.view(torch.uint8) for w in W]).view(E4), torch.stack([w.scales for w in W]), 128)
    chosen = (torch.randn(tokens, E, device="cuda", generator=gen) + torch.arange(E, device="cuda") * 0.2).topk(k).indices.int()
    chosen[:7] = -1
    rows = rt.expert_rows(chosen, E, align=align)
    whole = torch.full((rows.rows, 2064), 7.0, device="cuda", dtype=torch.bfloat16)
    C = whole[:, :N]
    rt.gemm_f8_experts(x, stack.t(), rows, C, gather=True)
    offsets, counts, X = rows.offsets.tolist(), rows.counts.tolist(), values(x)
    for e in range(E):
        first, n = offsets[e], counts[e]
        assert_close(C[first:first + n], X[rows.slots[first:first + n].long() // k], values(W[e].t()), f"expert {e}")
        assert bool((C[first + n:offsets[e + 1]] == 0).all())
    assert bool((whole[offsets[E]:] == 7).all()) and bool((whole[:, N:] == 7).all())
