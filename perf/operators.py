"""What the GEMM operators with a block-scaled (MX) operand are measured on.

A linear layer y = x W^T whose weights W are held in 4 bits, its input gradient dx = dy W through
the same weights, and its weight gradient dW = dy^T x from an activation checkpoint x held in 8
bits; and the conversions to and from those formats. A block-scaled matrix has one scale byte E
(2^(E - 127)) for each group of 32 consecutive columns of a row. Elements:

* ``fp4``:  4-bit floats (sign, 2 exponent, 1 mantissa bit: 0 .5 1 1.5 2 3 4 6), two to a byte,
  the even column in the low half;
* ``int8``: 8-bit integers q that stand for q / 64.

``own`` false computes every operator in plain torch; ``own`` true calls the framework.
"""
import math

import torch

own = False

GROUP = 32
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def listed():
    return [
        # one token through a small projection: latency counts
        {"name": "token_1024x1024", "op": "forward", "format": "fp4", "dtype": "bf16", "M": 1, "N": 1024, "K": 1024, "beta": 0.0},
        # one token through a wide up-projection
        {"name": "token_16384x4096", "op": "forward", "format": "fp4", "dtype": "f16", "M": 1, "N": 16384, "K": 4096, "beta": 0.0},
        # a decoding batch of 16 sequences, one token each
        {"name": "batch16_8192x8192", "op": "forward", "format": "fp4", "dtype": "bf16", "M": 16, "N": 8192, "K": 8192, "beta": 0.0},
        # a short prompt through a layer of odd sizes: rows of x that are not 16-byte aligned, a last
        # group of 9 columns, added to what C holds (a residual)
        {"name": "prompt100_1500x777", "op": "forward", "format": "fp4", "dtype": "bf16", "M": 100, "N": 1500, "K": 777, "beta": 1.0},
        # a few tokens on weights in 8 bits
        {"name": "token4_int8_4096x4096", "op": "forward", "format": "int8", "dtype": "bf16", "M": 4, "N": 4096, "K": 4096, "beta": 0.0},
        # a long prompt (or a training batch): the largest forward product
        {"name": "prompt8192_8192x8192", "op": "forward", "format": "fp4", "dtype": "bf16", "M": 8192, "N": 8192, "K": 8192, "beta": 0.0},
        # the gradient with respect to the layer's input, through frozen 4-bit weights
        {"name": "dx4096_4096x8192", "op": "dx", "format": "fp4", "dtype": "bf16", "M": 4096, "N": 4096, "K": 8192, "beta": 0.0},
        # the same on a layer of odd sizes
        {"name": "dx1000_777x1500", "op": "dx", "format": "fp4", "dtype": "f16", "M": 1000, "N": 777, "K": 1500, "beta": 0.0},
        # the weight gradient over 8192 tokens whose activations were kept in 8 bits
        {"name": "dw_4096x4096_8192", "op": "dw", "format": "int8", "dtype": "bf16", "M": 4096, "N": 4096, "K": 8192, "beta": 0.0},
        # a small layer's weight gradient over many tokens, accumulated over micro-batches
        {"name": "dw_1024x1024_16384", "op": "dw", "format": "int8", "dtype": "f16", "M": 1024, "N": 1024, "K": 16384, "beta": 1.0},
        # an activation checkpoint: kept in 8 bits and restored
        {"name": "keep_8192x8192", "op": "keep", "format": "int8", "dtype": "bf16", "rows": 8192, "cols": 8192},
        # weights of odd sizes taken to 4 bits from fp32 and back
        {"name": "keep_fp4_1500x777", "op": "keep", "format": "fp4", "dtype": "f32", "rows": 1500, "cols": 777},
    ]


def _size(rng, lo, hi):
    """A size spread over the logarithm of the range, one in two of them odd or ragged."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if rng.random() < 0.5:
        step = 64 if v >= 512 else 8
        v = max(lo, v // step * step)
    return min(v, hi)


def draw(rng):
    op = rng.choice(["forward", "forward", "dx", "dw", "keep"])
    fmt, dtype = rng.choice(["fp4", "int8"]), rng.choice(["bf16", "f16"])
    if op == "keep":
        return {"op": op, "format": fmt, "dtype": rng.choice(["bf16", "f16", "f32"]), "rows": _size(rng, 1, 8192), "cols": _size(rng, 64, 8192)}
    if op == "forward" and rng.random() < 0.6:  # tokens
        M, N, K = rng.randint(1, 64), _size(rng, 256, 16384), _size(rng, 256, 8192)
    else:
        M, N, K = _size(rng, 128, 8192), _size(rng, 128, 8192), _size(rng, 128, 8192)
    return {"op": op, "format": fmt, "dtype": dtype, "M": M, "N": N, "K": K, "beta": rng.choice([0.0, 0.0, 1.0])}


# ---- the formats in plain torch ------------------------------------------------------------
def _grouped(x):
    """rows x groups x 32, the last group filled up with zeros."""
    rows, cols = x.shape
    groups = (cols + GROUP - 1) // GROUP
    if cols == groups * GROUP:
        return x.reshape(rows, groups, GROUP)
    full = x.new_zeros(rows, groups * GROUP)
    full[:, :cols] = x
    return full.reshape(rows, groups, GROUP)


def _encode(x, fmt):
    """(codes, scales) of a rows x cols matrix of finite values."""
    rows, cols = x.shape
    g = _grouped(x.float())
    top = g.abs().amax(-1)
    field = top.view(torch.int32) >> 23  # the biased exponent: floor(log2) + 127
    E = (field - (2 if fmt == "fp4" else 0)).clamp(0, 254)
    if fmt == "int8":
        y = torch.round(g.double() * torch.exp2((133 - E).double())[..., None]).clamp(-127, 127)
        codes = y.to(torch.int8).view(torch.uint8).reshape(rows, -1)[:, :cols]
        return codes.contiguous(), E.to(torch.uint8)
    y = (g.double() * torch.exp2((127 - E).double())[..., None]).float()
    a = y.abs()
    # the borders between neighbours of 0 .5 1 1.5 2 3 4 6; a tie goes to the even code
    code = ((a > 0.25).byte() + (a >= 0.75).byte() + (a > 1.25).byte() + (a >= 1.75).byte()
            + (a > 2.5).byte() + (a >= 3.5).byte() + (a > 5.0).byte())
    code = (code | ((y < 0).byte() << 3)).reshape(rows, -1)
    used = (cols + 1) // 2
    return (code[:, 0::2] | (code[:, 1::2] << 4))[:, :used].contiguous(), E.to(torch.uint8)


_FP4 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0]


def _decode(codes, scales, fmt, cols):
    """The values of a block-scaled matrix, fp32."""
    if fmt == "int8":
        v, bias = codes.view(torch.int8).float(), 133
    else:
        table = torch.tensor(_FP4, device=codes.device)
        v, bias = table[torch.stack((codes & 15, codes >> 4), -1).long()].reshape(codes.shape[0], -1)[:, :cols], 127
    step = torch.exp2(scales.float() - bias)
    return v * step.repeat_interleave(GROUP, 1)[:, :cols]


# ---- cases ---------------------------------------------------------------------------------
def _make(case, seed):
    """Inputs of a case, made from the seed alone."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dtype = DTYPES[case["dtype"]]

    def normal(r, c):
        return torch.randn(r, c, device="cuda", generator=gen)

    if case["op"] == "keep":
        x = normal(case["rows"], case["cols"])
        if case["format"] == "int8":  # activations: features of unlike size, and a few far out
            x *= torch.exp(0.5 * torch.randn(1, case["cols"], device="cuda", generator=gen))
        else:  # weights
            x *= case["cols"] ** -0.5
        return {"X": x.to(dtype)}
    M, N, K = case["M"], case["N"], case["K"]
    if case["op"] == "dw":  # a gradient of K tokens x M features, a checkpoint of K tokens x N features
        A = (normal(K, M) * 1e-2).to(dtype)
    else:  # activations, or a gradient, of M tokens x K features
        A = normal(M, K).to(dtype) if case["op"] == "forward" else (normal(M, K) * 1e-2).to(dtype)
    b_rows, b_cols = (N, K) if case["op"] == "forward" else (K, N)
    B = normal(b_rows, b_cols)
    if case["format"] == "fp4" or case["op"] != "dw":
        B *= b_cols ** -0.5
    codes, scales = _encode(B.to(dtype), case["format"])
    return {"A": A, "codes": codes, "scales": scales, "cols": b_cols,
            "C": normal(M, N) if case["beta"] else None}


def prepare(case, seed):
    s = _make(case, seed)
    s.update(op=case["op"], format=case["format"], beta=case.get("beta", 0.0))
    return s


def _run_own(s):
    import register_tiled_matrix_amd as rt

    fmt = rt.MX_FP4 if s["format"] == "fp4" else rt.MX_INT8
    if s["op"] == "keep":
        return rt.dequantize_mx(rt.quantize_mx(s["X"], fmt), dtype=s["X"].dtype)
    B = rt.MXMatrix(fmt, s["codes"], s["scales"], s["cols"])
    A = s["A"]
    gemm = rt.gemm_bf16_mx if A.dtype == torch.bfloat16 else rt.gemm_f16_mx
    if s["op"] == "forward":
        return gemm(A, B.t(), s["C"], beta=s["beta"])
    if s["op"] == "dx":
        return gemm(A, B, s["C"], beta=s["beta"])
    return gemm(A.t(), B, s["C"], beta=s["beta"])


def run(s):
    if own:
        return _run_own(s)
    if s["op"] == "keep":
        X = s["X"]
        codes, scales = _encode(X, s["format"])
        return _decode(codes, scales, s["format"], X.shape[1]).to(X.dtype)
    V = _decode(s["codes"], s["scales"], s["format"], s["cols"])
    A = s["A"].float()
    if s["op"] == "forward":
        V = V.t()
    elif s["op"] == "dw":
        A = A.t()
    P = A @ V
    if s["C"] is None:
        return P
    return s["C"].mul_(s["beta"]).add_(P)  # accumulated in place, as the framework's C is


def work(case):
    if case["op"] == "keep":
        n = case["rows"] * case["cols"]
        size = 4 if case["dtype"] == "f32" else 2
        groups = case["rows"] * ((case["cols"] + GROUP - 1) // GROUP)
        held = (case["rows"] * ((case["cols"] + 1) // 2) if case["format"] == "fp4" else n) + groups
        return {"bytes": 2 * n * size + 2 * held, "flops": 4 * n}
    M, N, K = case["M"], case["N"], case["K"]
    rows, cols = (N, K) if case["op"] == "forward" else (K, N)
    held = rows * ((cols + 1) // 2 if case["format"] == "fp4" else cols) + rows * ((cols + GROUP - 1) // GROUP)
    return {"bytes": 2 * M * K + held + 4 * M * N * (2 if case["beta"] else 1), "flops": 2 * M * N * K}


# ---- the definition in 64 bits -------------------------------------------------------------
def _exact_kept(x, fmt):
    rows, cols = x.shape
    x = x.double()
    groups = -(-cols // GROUP)
    g = torch.nn.functional.pad(x, (0, groups * GROUP - cols)).view(rows, groups, GROUP)
    top = g.abs().max(dim=-1, keepdim=True).values
    exponent = torch.frexp(top).exponent - 1  # floor(log2 top)
    exponent = torch.where(top == 0, torch.full_like(exponent, -127), exponent)
    if fmt == "fp4":
        unit = torch.exp2((exponent - 2).clamp(-127, 127).double())
        y = g / unit
        octave = torch.frexp(y).exponent.clamp(min=1, max=3) - 1  # 0: below 2, 1: below 4, 2: above
        step = torch.exp2(octave.double() - 1)
        v = (torch.round(y / step) * step).clamp(-6, 6) * unit  # torch.round takes ties to even
    else:
        unit = torch.exp2(exponent.clamp(-127, 127).double() - 6)
        v = torch.round(g / unit).clamp(-127, 127) * unit
    return v.view(rows, -1)[:, :cols]


def _exact_values(codes, scales, fmt, cols):
    if fmt == "int8":
        q = codes.double()
        v = torch.where(q > 127, q - 256, q) / 64
    else:
        code = torch.empty(codes.shape[0], 2 * codes.shape[1], dtype=torch.int16, device=codes.device)
        code[:, 0::2], code[:, 1::2] = codes % 16, codes // 16
        e, m = (code // 2 % 4).double(), (code % 2).double()
        size = torch.where(e == 0, m / 2, (1 + m / 2) * torch.exp2(e - 1))
        v = torch.where(code >= 8, -size, size)[:, :cols]
    group = torch.arange(cols, device=codes.device) // GROUP
    return v * torch.exp2(scales.double() - 127)[:, group]


def exact(case, seed):
    s = _make(case, seed)
    if case["op"] == "keep":
        return _exact_kept(s["X"], case["format"])
    V = _exact_values(s["codes"], s["scales"], case["format"], s["cols"])
    A = s["A"].double()
    if case["op"] == "forward":
        P = torch.mm(A, V.T)
    elif case["op"] == "dx":
        P = torch.mm(A, V)
    else:
        P = torch.mm(A.T, V)
    return P if s["C"] is None else P + case["beta"] * s["C"].double()
