"""What the 8-bit floating point GEMM operators and a mixture of experts' operators are measured on.

A block-scaled 8-bit float matrix holds e4m3 (or e5m2) codes and one fp32 scale for each block of
128 columns of a row (activations, gradients), or of 128 x 128 values (weights). Operators:

* ``quantize``: to such a matrix and back;
* ``gemm``: the three products of a linear layer whose operands are both held so;
* ``route``: a router's choice of experts for each token, its weights (and their gradient), and the
  order of the tokens' rows by expert;
* ``experts``: those products for rows that fall into groups, one weight matrix to a group;
* ``combine``: each token's weighted sum of its experts' rows, and its gradient.

``own`` false computes every operator in plain torch; ``own`` true calls the framework.
"""
import math

import torch

own = False

BLOCK = 128
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
F8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
# largest value, explicit mantissa bits, exponent of the smallest normal value
F8_SHAPE = {"e4m3": (448.0, 3, -6), "e5m2": (57344.0, 2, -14)}


def listed():
    return [
        # activations of a long prompt, each token's features in blocks of 128
        {"name": "keep_8192x8192", "op": "quantize", "type": "e4m3", "dtype": "bf16", "rows": 8192, "cols": 8192, "block": 1, "transpose": False},
        # the same kind of matrix, transposed for a weight gradient: odd sizes, tokens end inside a block
        {"name": "keep_t_1500x777", "op": "quantize", "type": "e5m2", "dtype": "f32", "rows": 1500, "cols": 777, "block": 1, "transpose": True},
        # one token through a projection: latency counts
        {"name": "token_4096x4096", "op": "gemm", "pass": "forward", "a": "e4m3", "b": "e4m3", "out": "bf16", "M": 1, "N": 4096, "K": 4096, "beta": 0.0},
        # a long prompt (or a training batch): the largest product
        {"name": "prompt8192_8192x8192", "op": "gemm", "pass": "forward", "a": "e4m3", "b": "e4m3", "out": "bf16", "M": 8192, "N": 8192, "K": 8192, "beta": 0.0},
        # the gradient with respect to the layer's input: gradients in e5m2, the weights as the forward pass stores them
        {"name": "dx4096_4096x8192", "op": "gemm", "pass": "dx", "a": "e5m2", "b": "e4m3", "out": "bf16", "M": 4096, "N": 4096, "K": 8192, "beta": 0.0},
        # a weight gradient over a ragged number of tokens, accumulated over micro-batches
        {"name": "dw_2048x1500_8100", "op": "gemm", "pass": "dw", "a": "e5m2", "b": "e4m3", "out": "f32", "M": 2048, "N": 1500, "K": 8100, "beta": 1.0},
        # a decoding batch's router: sigmoid scores, a bias for balance, 4 of 8 groups, 8 of 256 experts
        {"name": "route64_256", "op": "route", "score": "sigmoid", "dtype": "f32", "tokens": 64, "experts": 256, "k": 8, "groups": 8, "top_groups": 4,
         "bias": True, "renormalize": True, "align": 1, "padded": 0, "grad": False},
        # a training step's router with its gradient: softmax, 8 of 64 experts, the batch's end padded
        {"name": "route8192_64_train", "op": "route", "score": "softmax", "dtype": "bf16", "tokens": 8192, "experts": 64, "k": 8, "groups": 1, "top_groups": 1,
         "bias": False, "renormalize": True, "align": 128, "padded": 100, "grad": True},
        # a decoding batch through 64 experts' up-projection: a few rows each, the weights' bytes count
        {"name": "experts64_4096x2048", "op": "experts", "pass": "forward", "a": "e4m3", "b": "e4m3", "out": "bf16", "tokens": 32, "k": 6, "experts": 64,
         "N": 4096, "K": 2048, "align": 1},
        # a prompt through the same experts: groups of unlike size
        {"name": "experts4096_4096x2048", "op": "experts", "pass": "forward", "a": "e4m3", "b": "e4m3", "out": "bf16", "tokens": 4096, "k": 6, "experts": 64,
         "N": 4096, "K": 2048, "align": 1},
        # a decoding batch's experts joined
        {"name": "combine32_2048", "op": "combine", "tokens": 32, "k": 6, "experts": 64, "N": 2048, "dtype": "bf16", "align": 1, "grad": False},
        # a training batch's experts joined, with the gradients of the rows and of the weights
        {"name": "combine8192_2048_train", "op": "combine", "tokens": 8192, "k": 8, "experts": 64, "N": 2048, "dtype": "bf16", "align": 128, "grad": True},
    ]


def _size(rng, lo, hi):
    """A size spread over the logarithm of the range, one in two of them odd or ragged."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if rng.random() < 0.5:
        step = 64 if v >= 512 else 8
        v = max(lo, v // step * step)
    return min(v, hi)


def draw(rng):
    op = rng.choice(["quantize", "gemm", "gemm", "gemm", "route", "experts", "experts", "combine"])
    if op == "quantize":
        block = rng.choice([1, 1, 128])
        return {"op": op, "type": rng.choice(["e4m3", "e5m2"]), "dtype": rng.choice(["bf16", "f16", "f32"]), "rows": _size(rng, 1, 8192),
                "cols": _size(rng, 64, 8192), "block": block, "transpose": block == 1 and rng.random() < 0.5}
    if op == "gemm":
        step = rng.choice(["forward", "forward", "dx", "dw"])
        if step == "forward" and rng.random() < 0.6:  # tokens
            M, N, K = rng.randint(1, 64), _size(rng, 256, 16384), _size(rng, 256, 8192)
        else:
            M, N, K = _size(rng, 128, 8192), _size(rng, 128, 8192), _size(rng, 128, 8192)
        return {"op": op, "pass": step, "a": "e4m3" if step == "forward" else rng.choice(["e4m3", "e5m2"]), "b": "e4m3",
                "out": "f32" if step == "dw" else rng.choice(["f32", "bf16", "f16"]), "M": M, "N": N, "K": K, "beta": rng.choice([0.0, 0.0, 1.0])}
    if op == "route":
        groups = rng.choice([1, 1, 4, 8])
        experts = groups * _size(rng, 8, 512 // groups)
        top_groups = rng.randint(1, groups)
        tokens = _size(rng, 1, 16384)
        return {"op": op, "score": rng.choice(["softmax", "sigmoid"]), "dtype": rng.choice(["f32", "bf16", "f16"]), "tokens": tokens, "experts": experts,
                "k": rng.randint(1, min(10, experts // groups * top_groups)), "groups": groups, "top_groups": top_groups, "bias": rng.random() < 0.5,
                "renormalize": rng.random() < 0.7, "align": rng.choice([1, 128]), "padded": rng.choice([0, tokens // 10]), "grad": rng.random() < 0.5}
    experts, k = _size(rng, 4, 128), rng.randint(1, 4)
    if op == "experts":
        step = rng.choice(["forward", "forward", "dx", "dw"])
        N, K = _size(rng, 128, 4096), _size(rng, 128, 4096)
        experts = max(k, min(experts, 2**29 // (N * K)))
        return {"op": op, "pass": step, "a": "e4m3" if step == "forward" else rng.choice(["e4m3", "e5m2"]), "b": "e4m3",
                "out": "f32" if step == "dw" else rng.choice(["f32", "bf16", "f16"]), "tokens": _size(rng, 1, 4096), "k": k, "experts": experts,
                "N": N, "K": K, "align": 128 if step == "dw" else rng.choice([1, 1, 128])}
    return {"op": op, "tokens": _size(rng, 1, 8192), "k": k, "experts": experts, "N": _size(rng, 64, 8192), "dtype": rng.choice(["f32", "bf16", "f16"]),
            "align": rng.choice([1, 128]), "grad": rng.random() < 0.5}


# ---- 8-bit float matrices in plain torch ----------------------------------------------------
def _blocks(x, block):
    """x (rows x cols) as row blocks x block x column blocks x 128, filled up with zeros."""
    rows, cols = x.shape
    nr, nc = -(-rows // block), -(-cols // BLOCK)
    if (nr * block, nc * BLOCK) != (rows, cols):
        full = x.new_zeros(nr * block, nc * BLOCK)
        full[:rows, :cols] = x
        x = full
    return x.view(nr, block, nc, BLOCK)


def _scales(g, kind):
    return (g.abs().amax((1, 3)) / F8_SHAPE[kind][0]).clamp(min=2.0**-126)


def _encode(x, kind, block):
    """(codes, scales) of finite values; operands are made with it."""
    rows, cols = x.shape
    g = _blocks(x.float(), block)
    s = _scales(g, kind)
    top = F8_SHAPE[kind][0]
    codes = (g / s[:, None, :, None]).clamp(-top, top).to(F8[kind])
    return codes.view(-1, g.shape[2] * BLOCK).view(torch.uint8)[:rows, :cols].contiguous().view(F8[kind]), s


def _values(codes, scales, block):
    """The fp32 values of a matrix, or of a stack of them."""
    rows, cols = codes.shape[-2:]
    s = scales.repeat_interleave(BLOCK, -1)[..., :cols]
    if block != 1:
        s = s.repeat_interleave(block, -2)[..., :rows, :]
    return codes.float() * s


def _kept(x, kind, block):
    """The values that x is held as. The quotient is taken in 64 bits: in 32 it can round onto a
    border between two codes."""
    top, bits, low = F8_SHAPE[kind]
    rows, cols = x.shape
    g = _blocks(x.float(), block)
    s = _scales(g, kind).double()[:, None, :, None]
    y = g.double() / s
    step = torch.exp2((torch.frexp(y).exponent - 1).clamp(min=low).double() - bits)
    v = (torch.round(y / step) * step).clamp(-top, top) * s
    return v.float().view(-1, g.shape[2] * BLOCK)[:rows, :cols]


# ---- routing in plain torch -------------------------------------------------------------------
def _scores(logits, kind):
    """fp64: scores next to each other decide which expert is chosen."""
    x = logits.double()
    if kind == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-x))
    top = x.amax(-1, keepdim=True)
    e = torch.exp(x - torch.where(top.isinf(), torch.zeros_like(top), top))
    total = e.sum(-1, keepdim=True)
    return e / torch.where(total == 0, torch.ones_like(total), total)


def _choose(s, v, case):
    """(experts, weights): the k largest of v, the lowest index among equals."""
    T, E, k = case["tokens"], case["experts"], case["k"]
    if case["groups"] > 1:
        inside = v.view(T, case["groups"], -1)
        if case["score"] == "sigmoid":  # a group counts as much as its two best experts
            best = inside.sort(-1, descending=True).values[..., :2]
            rank = torch.where(best.isinf(), torch.zeros_like(best), best).sum(-1)
            rank = torch.where(best[..., 0].isinf(), best[..., 0], rank)
        else:  # as its best
            rank = inside.amax(-1)
        kept = rank.sort(dim=-1, descending=True, stable=True).indices[:, :case["top_groups"]]
        open_ = torch.zeros_like(rank, dtype=torch.bool).scatter_(1, kept, True)
        v = torch.where(open_[..., None], inside, torch.full_like(inside, -math.inf)).view(T, E)
    best, order = v.sort(dim=-1, descending=True, stable=True)
    best, order = best[:, :k], order[:, :k]
    w = s.gather(1, order).masked_fill(best == -math.inf, 0.0)
    if case["renormalize"]:
        total = w.sum(-1, keepdim=True)
        w = w / torch.where(total == 0, torch.ones_like(total), total)
    return order.masked_fill(best == -math.inf, -1).int(), w


def _capacity(slots, experts, align):
    n = slots + min(slots, experts) * (align - 1)
    return -(-n // align) * align


def _rows_by_expert(experts, E, align):
    """(slots, position, offsets, counts): the slots t * k + j in the order of their experts, each
    expert's from a multiple of `align` on, and where each went."""
    flat = experts.reshape(-1).long()
    n = flat.numel()
    key = torch.where(flat < 0, torch.full_like(flat, E), flat)
    order = key.sort(stable=True).indices
    counts = torch.zeros(E + 1, dtype=torch.long, device=flat.device).scatter_add_(0, key, torch.ones_like(key))
    room = (counts + align - 1) // align * align
    room[E] = 0
    starts = room.cumsum(0) - room
    key = key[order]
    rank = torch.arange(n, device=flat.device) - (counts.cumsum(0) - counts)[key]
    to = torch.where(key < E, starts[key] + rank, torch.full_like(key, -1))
    position = torch.empty_like(flat).scatter_(0, order, to)
    size = _capacity(n, E, align)
    slots = torch.full((size + 1,), -1, dtype=torch.long, device=flat.device)
    slots.scatter_(0, torch.where(to < 0, torch.full_like(to, size), to), torch.where(to < 0, torch.full_like(order, -1), order))
    return slots[:size].int(), position.view(experts.shape).int(), starts.int(), counts[:E].int()


# ---- cases ------------------------------------------------------------------------------------
def _spread(experts, T, k, gen):
    """k different experts a token, some asked for more often than others."""
    liking = torch.randn(experts, device="cuda", generator=gen)
    x = torch.randn(T, experts, device="cuda", generator=gen) + liking
    return x.sort(-1, descending=True).indices[:, :k].int().contiguous()


def _make(case, seed):
    """Inputs of a case, made from the seed alone."""
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, device="cuda", generator=gen)

    def features(rows, cols):  # of unlike size, as activations have them
        return normal(rows, cols) * torch.exp(0.5 * normal(1, cols))

    op = case["op"]
    if op == "quantize":
        x = features(case["rows"], case["cols"]) if case["block"] == 1 else normal(case["rows"], case["cols"]) * case["cols"] ** -0.5
        return {"X": x.to(DTYPES[case["dtype"]])}
    if op == "gemm":
        M, N, K, step = case["M"], case["N"], case["K"], case["pass"]
        A = features(M, K) if step == "forward" else normal(M, K) * 1e-3
        qa, sa = _encode(A, case["a"], 1)
        if step == "dw":  # the input of the layer, transposed: features x tokens
            qb, sb = _encode(features(K, N).t(), case["b"], 1)
        else:
            rows, cols = (N, K) if step == "forward" else (K, N)
            qb, sb = _encode(normal(rows, cols) * cols ** -0.5, case["b"], BLOCK)
        return {"qa": qa, "sa": sa, "qb": qb, "sb": sb, "C": normal(M, N).to(DTYPES[case["out"]]) if case["beta"] else None}
    if op == "route":
        T, E = case["tokens"], case["experts"]
        x = normal(T, E) + 0.5 * normal(1, E)
        if case["padded"]:
            x[T - case["padded"]:] = -math.inf
        s = {"logits": x.to(DTYPES[case["dtype"]]), "bias": 0.1 * normal(E) if case["bias"] else None}
        s["dw"] = normal(T, case["k"]) if case["grad"] else None
        return s
    T, k, E = case["tokens"], case["k"], case["experts"]
    chosen = _spread(E, T, k, gen)
    if op == "combine":
        R, N = _capacity(T * k, E, case["align"]), case["N"]
        s = {"experts": chosen, "Y": normal(R, N).to(DTYPES[case["dtype"]]), "w": torch.rand(T, k, device="cuda", generator=gen) / k}
        s["dy"] = (normal(T, N) * 1e-3).to(DTYPES[case["dtype"]]) if case["grad"] else None
        return s
    N, K, step = case["N"], case["K"], case["pass"]
    s = {"experts": chosen}
    R = _capacity(T * k, E, case["align"])
    if step == "dw":  # both sides transposed, rows in the experts' order with zeros between the groups
        slots = _rows_by_expert(chosen, E, case["align"])[0]
        used = (slots >= 0).float()[None, :]
        s["qa"], s["sa"] = _encode(normal(N, R) * 1e-3 * used, case["a"], 1)
        s["qb"], s["sb"] = _encode(features(R, K).t() * used, case["b"], 1)
        return s
    rows, cols = (N, K) if step == "forward" else (K, N)
    parts = [_encode(normal(rows, cols) * cols ** -0.5, case["b"], BLOCK) for _ in range(E)]
    s["qb"] = torch.stack([p[0].view(torch.uint8) for p in parts]).view(F8[case["b"]])
    s["sb"] = torch.stack([p[1] for p in parts])
    # forward: the tokens; dx: gradients of the rows, in the experts' order
    s["qa"], s["sa"] = _encode(features(T, K) if step == "forward" else normal(R, K) * 1e-3, case["a"], 1)
    return s


def prepare(case, seed):
    s = _make(case, seed)
    s["case"] = case
    return s


def _run_own(s):
    import register_tiled_matrix_amd as rt

    case = s["case"]
    op = case["op"]
    if op == "quantize":
        Q = rt.quantize_f8(s["X"], F8[case["type"]], block_rows=case["block"], transpose=case["transpose"])
        return rt.dequantize_f8(Q, dtype=s["X"].dtype)
    if op == "gemm":
        A = rt.F8Matrix(s["qa"], s["sa"])
        B = rt.F8Matrix(s["qb"], s["sb"], block_rows=1 if case["pass"] == "dw" else BLOCK)
        return rt.gemm_f8(A, B if case["pass"] == "dx" else B.t(), s["C"], beta=case["beta"], dtype=DTYPES[case["out"]])
    if op == "route":
        score = rt.SCORE_SIGMOID if case["score"] == "sigmoid" else rt.SCORE_SOFTMAX
        experts, weights = rt.route_experts(s["logits"], case["k"], bias=s["bias"], score=score, groups=case["groups"],
                                            top_groups=case["top_groups"], group_best=2 if case["score"] == "sigmoid" else 1,
                                            renormalize=case["renormalize"])
        rows = rt.expert_rows(experts, case["experts"], align=case["align"])
        out = [experts, weights, rows.slots, rows.position, rows.offsets, rows.counts]
        if case["grad"]:
            out.append(rt.route_experts_grad(s["logits"], experts, s["dw"], score=score, renormalize=case["renormalize"]))
        return out
    rows = rt.expert_rows(s["experts"], case["experts"], align=case["align"])
    if op == "combine":
        y = rt.combine_experts(s["Y"], rows, s["w"])
        return y if s["dy"] is None else [y, *rt.combine_experts_grad(s["dy"], s["Y"], rows, s["w"])]
    A = rt.F8Matrix(s["qa"], s["sa"])
    if case["pass"] == "dw":
        return rt.gemm_f8_experts_dw(A, rt.F8Matrix(s["qb"], s["sb"]).t(), rows)
    B = rt.F8Matrix(s["qb"], s["sb"], block_rows=BLOCK)
    forward = case["pass"] == "forward"
    out, C = DTYPES[case["out"]], None
    if case["align"] > 1:  # rows behind the last group stay as they were
        C = torch.zeros(rows.slots.numel(), case["N"], dtype=out, device=s["qa"].device)
    return rt.gemm_f8_experts(A, B.t() if forward else B, rows, C, gather=forward, dtype=out)


def _plain_gemm(s, case):
    A, block = _values(s["qa"], s["sa"], 1), 1 if case["pass"] == "dw" else BLOCK
    B = _values(s["qb"], s["sb"], block)
    P = A @ (B if case["pass"] == "dx" else B.t())
    if s["C"] is None:
        return P.to(DTYPES[case["out"]])
    # accumulated in place, as the framework's C is
    return s["C"].copy_(P.add_(s["C"].float(), alpha=case["beta"]))


def _plain_route(s, case):
    p = _scores(s["logits"], case["score"])
    v = p.masked_fill(s["logits"] == -math.inf, -math.inf)
    if s["bias"] is not None:
        v = v + s["bias"].double()
    experts, w = _choose(p, v, case)
    out = [experts, w.float(), *_rows_by_expert(experts, case["experts"], case["align"])]
    if s["dw"] is None:
        return out
    chosen, none = experts.clamp(min=0).long(), experts < 0
    pick = p.gather(1, chosen).masked_fill(none, 0.0)
    ds = s["dw"].double()
    if case["renormalize"]:
        total = pick.sum(-1, keepdim=True)
        total = torch.where(total == 0, torch.full_like(total, math.inf), total)
        ds = (ds - (ds * pick).sum(-1, keepdim=True) / total) / total
    g = torch.zeros_like(p).scatter_add_(1, chosen, ds.masked_fill(none, 0.0))
    d = p * (1 - p) * g if case["score"] == "sigmoid" else p * (g - (g * p).sum(-1, keepdim=True))
    return out + [d.to(s["logits"].dtype)]


def _plain_experts(s, case):
    E, align = case["experts"], case["align"]
    slots, _, offsets, counts = _rows_by_expert(s["experts"], E, align)
    starts, n = offsets.tolist(), counts.tolist()
    if case["pass"] == "dw":
        A, B = _values(s["qa"], s["sa"], 1), _values(s["qb"], s["sb"], 1)
        out = torch.empty(E, case["N"], case["K"], device=A.device)
        for e in range(E):
            part = slice(starts[e], starts[e] + n[e])
            torch.matmul(A[:, part], B[:, part].t(), out=out[e])
        return out
    A = _values(s["qa"], s["sa"], 1)
    if case["pass"] == "forward":
        A = A[slots.clamp(min=0).long() // case["k"]]
    out = torch.zeros(slots.numel(), case["N"], dtype=DTYPES[case["out"]], device=A.device)
    for e in range(E):
        if n[e]:
            part = slice(starts[e], starts[e] + n[e])
            B = _values(s["qb"][e], s["sb"][e], BLOCK)
            out[part] = (A[part] @ (B.t() if case["pass"] == "forward" else B)).to(out.dtype)
    return out


def _plain_combine(s, case):
    slots, position, _, _ = _rows_by_expert(s["experts"], case["experts"], case["align"])
    rows = s["Y"].float()[position.long()]  # every slot is routed here
    y = (rows * s["w"][..., None]).sum(1).to(s["Y"].dtype)
    if s["dy"] is None:
        return y
    dy = s["dy"].float()
    dw = (rows * dy[:, None, :]).sum(-1)
    at = slots.clamp(min=0).long()
    scale = s["w"].reshape(-1)[at].masked_fill(slots < 0, 0.0)
    return [y, (dy[at // case["k"]] * scale[:, None]).to(s["Y"].dtype), dw]


def run(s):
    if own:
        return _run_own(s)
    case = s["case"]
    if case["op"] == "quantize":
        X = s["X"].t() if case["transpose"] else s["X"]
        return _kept(X, case["type"], case["block"]).to(s["X"].dtype)
    return {"gemm": _plain_gemm, "route": _plain_route, "experts": _plain_experts, "combine": _plain_combine}[case["op"]](s, case)


def work(case):
    op = case["op"]
    if op == "quantize":
        n = case["rows"] * case["cols"]
        return {"bytes": 2 * n * (4 if case["dtype"] == "f32" else 2) + 2 * n, "flops": 4 * n}
    if op == "route":
        T, E, k = case["tokens"], case["experts"], case["k"]
        size = 4 if case["dtype"] == "f32" else 2
        rows = _capacity(T * k, E, case["align"])
        moved = T * E * size + T * k * 12 + 4 * rows + 8 * E
        return {"bytes": moved + ((2 * T * E * size + T * k * 8) if case["grad"] else 0), "flops": 20 * T * E * (2 if case["grad"] else 1)}
    if op == "gemm":
        M, N, K = case["M"], case["N"], case["K"]
        size = 4 if case["out"] == "f32" else 2
        scales = 4 * M * -(-K // BLOCK) + (4 * N * -(-K // BLOCK) if case["pass"] == "dw" else 4 * -(-N // BLOCK) * -(-K // BLOCK))
        return {"bytes": M * K + N * K + scales + size * M * N * (2 if case["beta"] else 1), "flops": 2 * M * N * K}
    T, k, E, N = case["tokens"], case["k"], case["experts"], case["N"]
    if op == "combine":
        size = 4 if case["dtype"] == "f32" else 2
        moved = T * k * N * size + T * N * size + 8 * T * k
        return {"bytes": moved + ((T * k * N * size + T * N * size + 4 * T * k) if case["grad"] else 0), "flops": 2 * T * k * N * (3 if case["grad"] else 1)}
    K = case["K"]
    size = 4 if case["out"] == "f32" else 2
    if case["pass"] == "dw":
        moved = T * k * (N + K) + E * N * K * 4
    else:
        moved = (T if case["pass"] == "forward" else T * k) * K + min(E, T * k) * N * K + T * k * N * size
    return {"bytes": moved, "flops": 2 * T * k * N * K}


# ---- the definitions in 64 bits ---------------------------------------------------------------
def _exact_kept(x, kind, block):
    top, bits, low = F8_SHAPE[kind]
    rows, cols = x.shape
    x = x.double()
    nr, nc = -(-rows // block), -(-cols // BLOCK)
    g = torch.nn.functional.pad(x, (0, nc * BLOCK - cols, 0, nr * block - rows)).view(nr, block, nc, BLOCK)
    unit = (g.abs().amax(dim=(1, 3), keepdim=True) / top).float().clamp_min(2.0**-126).double()  # scales are fp32
    y = g / unit
    octave = torch.floor(torch.log2(y.abs().clamp_min(2.0**(low - 1))))
    octave = torch.where(torch.exp2(octave) > y.abs(), octave - 1, octave)
    octave = torch.where(torch.exp2(octave + 1) <= y.abs(), octave + 1, octave).clamp_min(low)
    step = torch.exp2(octave - bits)
    v = torch.minimum(torch.round(y / step) * step, torch.full_like(y, top))
    v = torch.maximum(v, torch.full_like(y, -top)) * unit
    return v.reshape(nr * block, nc * BLOCK)[:rows, :cols]


def _exact_matrix(codes, scales, block):
    rows, cols = codes.shape
    r = torch.arange(rows, device=codes.device) // block
    c = torch.arange(cols, device=codes.device) // BLOCK
    return codes.to(torch.float32).double() * scales.double()[r][:, c]


def _exact_route(s, case):
    x = s["logits"].double()
    if case["score"] == "sigmoid":
        p = torch.sigmoid(x)
    else:
        p = torch.softmax(x, -1).nan_to_num(0.0)
    v = p if s["bias"] is None else p + s["bias"].double()
    v = torch.where(x == -math.inf, x, v)
    T, G = case["tokens"], case["groups"]
    for_group = v.reshape(T, G, -1)
    if G > 1:
        if case["score"] == "sigmoid" and for_group.shape[-1] > 1:
            rank = for_group.topk(2, -1).values.sum(-1)
        else:
            rank = for_group.max(-1).values
        closed = rank.argsort(dim=-1, descending=True, stable=True)[:, case["top_groups"]:]
        v = for_group.scatter(1, closed[..., None].expand(-1, -1, for_group.shape[-1]), -math.inf).reshape(T, -1)
    chosen = v.argsort(dim=-1, descending=True, stable=True)[:, :case["k"]]
    there = v.gather(1, chosen) > -math.inf

    def weights(scores):
        w = scores.gather(1, chosen) * there
        return w / w.sum(-1, keepdim=True).clamp_min(1e-300) if case["renormalize"] else w

    out = [None, weights(p), None, None, None, None]
    if s["dw"] is not None:
        with torch.enable_grad():
            z = x.clone().masked_fill_(x == -math.inf, -1e4).requires_grad_()
            q = torch.sigmoid(z) if case["score"] == "sigmoid" else torch.softmax(z, -1)
            (weights(q) * s["dw"].double() * there).sum().backward()
        out.append(z.grad.masked_fill(x == -math.inf, 0.0))
    return out


def exact(case, seed):
    s = _make(case, seed)
    op = case["op"]
    if op == "quantize":
        return _exact_kept(s["X"].t() if case["transpose"] else s["X"], case["type"], case["block"])
    if op == "route":
        return _exact_route(s, case)
    if op == "gemm":
        A = _exact_matrix(s["qa"], s["sa"], 1)
        B = _exact_matrix(s["qb"], s["sb"], 1 if case["pass"] == "dw" else BLOCK)
        P = torch.mm(A, B if case["pass"] == "dx" else B.T)
        return P if s["C"] is None else P + case["beta"] * s["C"].double()
    # rows by expert, in the order of their slots
    flat, E, align = s["experts"].reshape(-1), case["experts"], case["align"]
    members = [(flat == e).nonzero()[:, 0] for e in range(E)]
    R, at, starts = _capacity(flat.numel(), E, align), 0, []
    for m in members:
        starts.append(at)
        at += -(-m.numel() // align) * align
    if op == "combine":
        T, k, N = case["tokens"], case["k"], case["N"]
        y = torch.zeros(T, N, dtype=torch.float64, device=flat.device)
        dY, dw = torch.zeros(R, N, dtype=torch.float64, device=flat.device), torch.zeros(T * k, dtype=torch.float64, device=flat.device)
        w = s["w"].double().reshape(-1)
        for m, r in zip(members, starts):
            rows = s["Y"][r:r + m.numel()].double()
            y.index_add_(0, m // k, rows * w[m, None])
            if s["dy"] is not None:
                d = s["dy"].double()[m // k]
                dY[r:r + m.numel()] = d * w[m, None]
                dw[m] = (d * rows).sum(-1)
        return y if s["dy"] is None else [y, dY, dw.view(T, k)]
    A = _exact_matrix(s["qa"], s["sa"], 1)
    if case["pass"] == "dw":
        B = _exact_matrix(s["qb"], s["sb"], 1)
        return torch.stack([torch.mm(A[:, r:r + m.numel()], B[:, r:r + m.numel()].T) for m, r in zip(members, starts)])
    out = torch.zeros(R, case["N"], dtype=torch.float64, device=flat.device)
    for e, (m, r) in enumerate(zip(members, starts)):
        if m.numel():
            B = _exact_matrix(s["qb"][e], s["sb"][e], BLOCK)
            rows = A[m // case["k"]] if case["pass"] == "forward" else A[r:r + m.numel()]
            out[r:r + m.numel()] = torch.mm(rows, B.T if case["pass"] == "forward" else B)
    return out
