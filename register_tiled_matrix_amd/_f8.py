"""Block-scaled 8-bit float matrices, their products, and a mixture of experts: the binding of the second half
of ``include/regtile.h``, which states layouts and formulas. Part of the package's namespace."""
from __future__ import annotations

import ctypes

import register_tiled_matrix_amd as _rt

__all__ = [
    "F8_E4M3", "F8_E5M2", "F8_BLOCK", "F8Matrix", "quantize_f8", "dequantize_f8", "gemm_f8",
    "SCORE_SOFTMAX", "SCORE_SIGMOID", "route_experts", "route_experts_grad", "ExpertRows", "expert_rows", "expert_rows_size",
    "gemm_f8_experts", "gemm_f8_experts_dw", "combine_experts", "combine_experts_grad",
]

F8_E4M3, F8_E5M2 = 0, 1  # regtile_f8_type
F8_BLOCK = 128
SCORE_SOFTMAX, SCORE_SIGMOID = 0, 1  # regtile_score
MAX_EXPERTS = 1024


class MatrixStruct(ctypes.Structure):
    """regtile_f8_matrix of include/regtile.h."""
    _fields_ = [("codes", ctypes.c_void_p), ("ld", ctypes.c_int64), ("scales", ctypes.c_void_p), ("scale_row", ctypes.c_int64),
                ("scale_col", ctypes.c_int64), ("codes_stack", ctypes.c_int64), ("scales_stack", ctypes.c_int64),
                ("rows", ctypes.c_int), ("cols", ctypes.c_int), ("stack", ctypes.c_int), ("type", ctypes.c_int),
                ("block_rows", ctypes.c_int)]


class RowsStruct(ctypes.Structure):
    """regtile_expert_rows of include/regtile.h."""
    _fields_ = [("slots", ctypes.c_void_p), ("position", ctypes.c_void_p), ("offsets", ctypes.c_void_p), ("counts", ctypes.c_void_p),
                ("tokens", ctypes.c_int), ("k", ctypes.c_int), ("experts", ctypes.c_int), ("align", ctypes.c_int), ("rows", ctypes.c_int)]


def declare(lib):
    """The C signatures."""
    I, F, P, L = ctypes.c_int, ctypes.c_float, ctypes.c_void_p, ctypes.c_int64
    for name, args in (("regtile_quantize_f8", [I, I, I, I, P, I, P, P, P]), ("regtile_dequantize_f8", [P, I, P, I, P]),
                       ("regtile_gemm_f8", [I, I, F, P, P, F, I, P, I, P, L, P]),
                       ("regtile_order_experts", [P, P, P, L, P]),
                       ("regtile_gemm_f8_experts", [P, I, I, F, P, P, F, I, P, I, P, L, P]),
                       ("regtile_gemm_f8_experts_dw", [P, F, P, P, F, I, P, I, L, P, L, P]),
                       ("regtile_route_experts", [I] * 9 + [F, P, I, P, P, P, P]),
                       ("regtile_route_experts_grad", [I] * 6 + [F, P, I, P, P, P, I, P]),
                       ("regtile_combine_experts", [P, I, I, P, I, P, P, I, P]),
                       ("regtile_combine_experts_grad", [P, I, I, P, I, P, I, P, P, I, P, P])):
        f = getattr(lib, name)
        f.argtypes = args
        f.restype = I
    for name, args in (("regtile_gemm_f8_workspace", [I, I, P, P, I, I]), ("regtile_expert_rows_size", [I] * 4),
                       ("regtile_gemm_f8_experts_workspace", [P, I, I, P, P, I]), ("regtile_gemm_f8_experts_dw_workspace", [P, P, P, I]),
                       ("regtile_order_experts_workspace", [I] * 3)):
        f = getattr(lib, name)
        f.argtypes = args
        f.restype = L


_torch = None
_types = {}  # regtile_f8_type by torch dtype


def _import_torch():
    global _torch
    torch = _rt._torch or _rt._import_torch()
    _types.update({torch.float8_e4m3fn: F8_E4M3, torch.float8_e5m2: F8_E5M2})
    _torch = torch
    return torch


def _lib():
    return _rt._lib or _rt.load()


def _int32(t, name, device, shape=None):
    if t.dtype is not _torch.int32 or not t.is_contiguous() or t.device != device or (shape is not None and tuple(t.shape) != shape):
        raise ValueError(f"{name} must be a contiguous int32 tensor{'' if shape is None else f' of shape {shape}'} on {device}")


def _blocks(n, block=F8_BLOCK):
    return -(-n // block)


class F8Matrix:
    """A block-scaled 8-bit float matrix (include/regtile.h states the layout), or a stack of them.

    ``codes``: rows x cols (or stack x rows x cols) of ``torch.float8_e4m3fn`` or ``torch.float8_e5m2`` with unit
    column stride. ``scales``: float32, ceil(rows / block_rows) x ceil(cols / 128) (in a stack: of each), any
    strides. ``block_rows``: 1 (activations) or 128 (weights). ``t()`` is the transposed view: the same bytes,
    taken as cols x rows. The tensors are kept, not copied, and described anew where a call finds that their storage has been
    replaced. Products are fastest where rows of codes start at multiples of 16 bytes (``quantize_f8`` lays them out so) and
    scales of one block of columns are contiguous.
    """

    __slots__ = ("codes", "scales", "block_rows", "type", "transposed", "_rows", "_cols", "_stack", "_c", "_address", "_codes_at", "_scales_at")

    def __init__(self, codes, scales, block_rows=1, transposed=False):
        self.codes, self.scales, self.block_rows, self.transposed = codes, scales, block_rows, bool(transposed)
        self._rows = None
        self._describe()

    def _describe(self):
        torch = _torch or _import_torch()
        codes, scales, block_rows = self.codes, self.scales, self.block_rows
        kind = _types.get(codes.dtype)
        if kind is None:
            raise ValueError("codes must be float8_e4m3fn or float8_e5m2")
        if block_rows != 1 and block_rows != F8_BLOCK:
            raise ValueError(f"block_rows must be 1 or {F8_BLOCK}, not {block_rows}")
        if scales.dtype is not torch.float32:
            raise ValueError("scales must be float32")
        dim = codes.dim()
        if dim not in (2, 3) or scales.dim() != dim:
            raise ValueError("codes and scales must both be 2-D, or both 3-D (a stack)")
        shape, strides = codes.shape, codes.stride()
        rows, cols = shape[-2], shape[-1]
        stack = shape[0] if dim == 3 else 1
        want = (_blocks(rows) if block_rows != 1 else rows, _blocks(cols))
        if tuple(scales.shape[-2:]) != want or (dim == 3 and scales.shape[0] != stack):
            raise ValueError(f"scales must be {want}{' for each of the stack' if dim == 3 else ''}, not {tuple(scales.shape)}")
        if (cols > 1 and strides[-1] != 1) or (rows > 1 and strides[-2] < cols):
            raise ValueError("codes must be row-major with rows that do not overlap")
        if codes.device != scales.device:
            raise ValueError("codes and scales are on different devices")
        ld = max(strides[-2], cols, 1)
        _rt._ints(rows, cols, ld, stack)
        now = rows, cols, stack if dim == 3 else 0, kind
        if self._rows is not None and (self._rows, self._cols, self._stack, self.type) != now:
            raise ValueError("the matrix's codes were replaced by some of another shape or type")
        s = scales.stride()
        self._rows, self._cols, self._stack, self.type = now
        self._codes_at, self._scales_at = codes.data_ptr(), scales.data_ptr()
        self._c = MatrixStruct(self._codes_at, ld, self._scales_at, s[-2], s[-1], strides[0] if dim == 3 else 0,
                               s[0] if dim == 3 else 0, rows, cols, stack, kind, block_rows)
        self._address = ctypes.addressof(self._c)

    @property
    def _at(self):
        """The address of its regtile_f8_matrix."""
        if self.codes.data_ptr() != self._codes_at or self.scales.data_ptr() != self._scales_at:
            self._describe()
        return self._address

    @property
    def shape(self):
        """Rows and columns as this view takes them, behind the size of the stack if it is one."""
        own = (self._cols, self._rows) if self.transposed else (self._rows, self._cols)
        return (self._stack, *own) if self.codes.dim() == 3 else own

    @property
    def device(self):
        return self.codes.device

    def t(self):
        v = object.__new__(F8Matrix)
        v.codes, v.scales, v.block_rows, v.type, v.transposed = self.codes, self.scales, self.block_rows, self.type, not self.transposed
        v._rows, v._cols, v._stack, v._c, v._address = self._rows, self._cols, self._stack, self._c, self._address
        v._codes_at, v._scales_at = self._codes_at, self._scales_at
        return v

    def __repr__(self):
        name = "e4m3" if self.type == F8_E4M3 else "e5m2"
        return f"F8Matrix({name}, {' x '.join(map(str, self.shape))}, blocks of {self.block_rows} x {F8_BLOCK}{', transposed' if self.transposed else ''})"


def _new_matrix(like, dtype, rows, cols, block_rows):
    """A matrix to be written: rows of codes from multiples of 16 bytes on, scales of a block of columns together."""
    ld = (cols + 15) // 16 * 16 or 16
    br, bc = (rows if block_rows == 1 else _blocks(rows)), _blocks(cols)
    m = object.__new__(F8Matrix)
    codes = m.codes = like.new_empty_strided((rows, cols), (ld, 1), dtype=dtype)
    scales = m.scales = like.new_empty_strided((br, bc), (1, br or 1), dtype=_torch.float32)
    m.block_rows, m.type, m.transposed = block_rows, _types[dtype], False
    m._rows, m._cols, m._stack = rows, cols, 0
    m._codes_at, m._scales_at = codes.data_ptr(), scales.data_ptr()
    m._c = MatrixStruct(m._codes_at, ld, m._scales_at, 1, br or 1, 0, 0, rows, cols, 1, m.type, block_rows)
    m._address = ctypes.addressof(m._c)
    return m


def quantize_f8(X, dtype=None, block_rows=1, transpose=False, rows=None, out=None, stream=None):
    """The block-scaled 8-bit float form of a row-major device tensor X (float32, bfloat16 or float16), ``dtype``
    float8_e4m3fn (the default) or float8_e5m2, in blocks of ``block_rows`` x 128. ``transpose``: that of X's
    transpose, in blocks of 128 of X's rows (for a product over them, such as a weight gradient). ``rows``: of
    X[rows], an int32 tensor; numbers that are no row of X give zeros. Writes into ``out`` (an F8Matrix) or a new
    F8Matrix, and returns it."""
    torch = _torch or _import_torch()
    if dtype is None:
        dtype = torch.float8_e4m3fn if out is None else out.codes.dtype
    if dtype not in _types:
        raise ValueError(f"dtype must be float8_e4m3fn or float8_e5m2, not {dtype}")
    dt = _rt._mx_dtype(X.dtype, "X")
    if not X.is_cuda:
        raise ValueError("quantize_f8 takes a device tensor")
    if block_rows != 1 and (block_rows != F8_BLOCK or transpose):
        raise ValueError(f"block_rows must be 1, or {F8_BLOCK} without transpose")
    ldx, x_rows, x_cols = _rt._rows(X, "X")
    n = x_rows
    if rows is not None:
        if rows.dim() != 1:
            raise ValueError("rows must be 1-D")
        _int32(rows, "rows", X.device)
        n = rows.shape[0]
    shape = (x_cols, n) if transpose else (n, x_cols)
    if out is not None and (not isinstance(out, F8Matrix) or out.codes.dtype is not dtype or out.block_rows != block_rows or
                            out.transposed or out.shape != shape or out.device != X.device):
        raise ValueError(f"out must be an untransposed F8Matrix of {dtype}, shape {shape}, blocks of {block_rows} x {F8_BLOCK} on {X.device}")
    _rt._ints(ldx, *shape)
    return _rt._launched(_run_quantize, X.device, stream, X, dtype, dt, block_rows, transpose, x_rows, x_cols, ldx, rows, shape, out)


def _run_quantize(X, dtype, dt, block_rows, transpose, x_rows, x_cols, ldx, rows, shape, Q, handle):
    if Q is None:
        Q = _new_matrix(X, dtype, *shape, block_rows)
    if 0 in shape:  # (an empty tensor of row numbers has no address)
        return Q
    status = _lib().regtile_quantize_f8(dt, 1 if transpose else 0, x_rows, x_cols, X.data_ptr(), ldx,
                                        None if rows is None else rows.data_ptr(), Q._at, handle)
    if status:
        _rt._check(status)
    return Q


def dequantize_f8(Q, dtype=None, out=None, stream=None):
    """The values of an F8Matrix (no stack) as a row-major tensor of its shape (of a transposed one: the transposed view of
    a row-major tensor), rounded to ``dtype`` (bfloat16 when neither it nor ``out`` is given). Writes into
    ``out`` or a new tensor, and returns it."""
    torch = _torch or _import_torch()
    if not isinstance(Q, F8Matrix) or not Q.codes.is_cuda or Q.codes.dim() != 2:
        raise ValueError("dequantize_f8 takes a single F8Matrix of device tensors")
    if dtype is None:
        dtype = torch.bfloat16 if out is None else out.dtype
    dt = _rt._mx_dtype(dtype, "dtype")
    if out is not None and (out.dtype != dtype or tuple(out.shape) != Q.shape or out.device != Q.device):
        raise ValueError(f"out must be {dtype} of shape {Q.shape} on {Q.device}")
    X = _rt._launched(_run_dequantize, Q.device, stream, Q, dtype, dt, out)
    if out is not None:
        return out
    return X.t() if Q.transposed else X


def _run_dequantize(Q, dtype, dt, out, handle):
    if out is None:
        X = Q.codes.new_empty((Q._rows, Q._cols), dtype=dtype)
    else:
        X = out.t() if Q.transposed else out
    ldx = _rt._rows(X, "out")[0]
    _rt._ints(ldx)
    _rt._check(_lib().regtile_dequantize_f8(Q._at, dt, X.data_ptr(), ldx, handle))
    return X


def _operands(name, A, B, stack=None):
    """Checks what every product checks; (M, K, N)."""
    if not isinstance(A, F8Matrix) or not isinstance(B, F8Matrix):
        raise ValueError(f"{name} takes F8Matrix operands")
    a, b = A.codes, B.codes
    if a.dim() != 2 or b.dim() != (2 if stack is None else 3):
        raise ValueError(f"{name}: A is a single matrix" + (" and so is B" if stack is None else ", B a stack of them"))
    if stack is not None and B._stack != stack:
        raise ValueError(f"{name}: B must be a stack of {stack} matrices, not {B._stack}")
    index = a.get_device()  # (a number: -1 on the host)
    if index < 0 or b.get_device() != index:
        raise ValueError(f"{name} takes device tensors, all on one device")
    if (A.transposed and A.block_rows == 1) or (not B.transposed and B.block_rows == 1):
        raise ValueError(f"{name}: blocks of 1 x {F8_BLOCK} must run along k (a row-major A, a transposed B); "
                         f"quantize_f8(..., transpose=True) makes them run the other way")
    M, K = (A._cols, A._rows) if A.transposed else (A._rows, A._cols)
    K2, N = (B._cols, B._rows) if B.transposed else (B._rows, B._cols)
    if K != K2:
        raise ValueError(f"inner dimensions differ: {K} vs {K2}")
    return M, K, N


def _c_of(C, dtype, beta, shape, device):
    """(dtype, its number, leading dimension) of C, given or to be made."""
    if dtype is None:
        dtype = _torch.float32 if C is None else C.dtype
    dt = _rt._mx_dtype(dtype, "dtype")
    if C is None:
        if beta != 0.0:
            raise ValueError("beta != 0 needs C")
        return dtype, dt, max(shape[-1], 1)
    if C.dtype is not dtype or tuple(C.shape) != shape or C.device != device:
        raise ValueError(f"C must be {dtype} of shape {shape} on {device}")
    if C.dim() == 3:
        ldc = max(C.stride(1), shape[2], 1)
        if (shape[2] > 1 and C.stride(2) != 1) or (shape[1] > 1 and C.stride(1) < shape[2]):
            raise ValueError("C must be row-major with rows that do not overlap")
        if shape[0] > 1 and shape[1] and shape[2] and C.stride(0) < (shape[1] - 1) * ldc + shape[2]:
            raise ValueError("C's matrices overlap")
    else:
        ldc = _rt._rows(C, "C")[0]
    _rt._ints(ldc)
    return dtype, dt, ldc


def _workspace(A, size):
    """(tensor, address, bytes): the tensor has to stay until the launch is queued."""
    if size <= 0:
        return None, None, 0
    work = A.codes.new_empty(size, dtype=_torch.uint8)
    return work, work.data_ptr(), size


def gemm_f8(A, B, C=None, alpha=1.0, beta=0.0, dtype=None, stream=None):
    """C = alpha*A@B + beta*C; F8Matrix A (M x K) and B (K x N), a row-major C of ``dtype`` (float32, the default, or
    bfloat16 or float16; C's, if it is given); returns C (allocated when None). Scales have to run along k: with
    weights ``W`` in blocks of 128 x 128 and ``x``, ``dy`` in blocks of 1 x 128, ``y = gemm_f8(xq, Wq.t())``,
    ``dx = gemm_f8(dyq, Wq)`` and ``dW = gemm_f8(dyt, xt.t())`` with ``dyt = quantize_f8(dy, transpose=True)`` and
    ``xt`` alike. A float32 C is made of exact products; large products into 16 bits cut off up to 2.4e-4 of the sum of
    magnitudes before they are rounded (include/regtile.h has the figures, and the scales' limits)."""
    M, _, N = _operands("gemm_f8", A, B)
    device = A.codes.device
    dtype, dt, ldc = _c_of(C, dtype, beta, (M, N), device)
    return _rt._launched(_run_gemm, device, stream, A, B, C, float(alpha), float(beta), dtype, dt, M, N, ldc)


def _run_gemm(A, B, C, alpha, beta, dtype, dt, M, N, ldc, handle):
    lib = _lib()
    if C is None:
        C = A.codes.new_empty((M, N), dtype=dtype)
    ta, tb = (1 if A.transposed else 0), (1 if B.transposed else 0)
    a, b = A._at, B._at
    # (a few rows go without)
    work, at, size = _workspace(A, 0 if M <= 16 and tb and N < 1 << 27 else lib.regtile_gemm_f8_workspace(ta, tb, a, b, dt, ldc))
    status = lib.regtile_gemm_f8(ta, tb, alpha, a, b, beta, dt, C.data_ptr(), ldc, at, size, handle)
    if status:
        _rt._check(status)
    return C


# ---- a mixture of experts ----------------------------------------------------------------------
def _logits(logits, score):
    if score != SCORE_SOFTMAX and score != SCORE_SIGMOID:
        raise ValueError(f"unknown score {score!r}")
    dt = _rt._mx_dtype(logits.dtype, "logits")
    if not logits.is_cuda:
        raise ValueError("logits must be a device tensor")
    ld, tokens, experts = _rt._rows(logits, "logits")
    if not 1 <= experts <= MAX_EXPERTS:
        raise ValueError(f"1 to {MAX_EXPERTS} experts, not {experts}")
    _rt._ints(ld, tokens)
    return dt, ld, tokens, experts


def route_experts(logits, k, bias=None, score=SCORE_SOFTMAX, groups=1, top_groups=1, group_best=1, renormalize=True, scale=1.0,
                  stream=None):
    """A router: (experts, weights), tokens x k int32 and float32, from logits (tokens x experts; float32, bfloat16
    or float16). Scores are the softmax or the sigmoid of the logits; the ``k`` largest of score + bias are chosen,
    the lowest number among equals, from the ``top_groups`` best of ``groups`` groups of experts (by a group's
    largest value, or with ``group_best=2`` the sum of its two largest); weights are the chosen scores, divided by their
    sum if ``renormalize``, times ``scale``. Experts with logit -inf are never chosen: slots for which none is
    left hold -1 and weight 0. A row with a NaN or +inf has NaN weights."""
    torch = _torch or _import_torch()
    dt, ld, tokens, experts = _logits(logits, score)
    if not 1 <= k <= min(experts, 64):
        raise ValueError(f"k must be 1 to {min(experts, 64)}, not {k}")
    if not 1 <= groups <= 64 or experts % groups:
        raise ValueError(f"groups must be 1 to 64 and divide {experts}, not {groups}")
    if not 1 <= top_groups <= groups or group_best not in (1, 2):
        raise ValueError("top_groups must be 1 to groups, group_best 1 or 2")
    if bias is not None and (bias.dtype is not torch.float32 or tuple(bias.shape) != (experts,) or not bias.is_contiguous() or
                             bias.device != logits.device):
        raise ValueError(f"bias must be a contiguous float32 tensor of {experts} on {logits.device}")
    return _rt._launched(_run_route, logits.device, stream, score, dt, tokens, experts, k, groups, top_groups, group_best,
                         1 if renormalize else 0, float(scale), logits, ld, bias)


def _run_route(score, dt, tokens, experts, k, groups, top_groups, group_best, renormalize, scale, logits, ld, bias, handle):
    chosen = logits.new_empty((tokens, k), dtype=_torch.int32)
    weights = logits.new_empty((tokens, k), dtype=_torch.float32)
    _rt._check(_lib().regtile_route_experts(score, dt, tokens, experts, k, groups, top_groups, group_best, renormalize, scale,
                                            logits.data_ptr(), ld, None if bias is None else bias.data_ptr(), chosen.data_ptr(),
                                            weights.data_ptr(), handle))
    return chosen, weights


def route_experts_grad(logits, experts, dweights, score=SCORE_SOFTMAX, renormalize=True, scale=1.0, stream=None):
    """The gradient with respect to the logits (their dtype and shape), from the gradient with respect to the weights that
    ``route_experts`` gave with the same arguments (tokens x k, float32). The choice is a constant."""
    torch = _torch or _import_torch()
    dt, ld, tokens, n = _logits(logits, score)
    if experts.dim() != 2 or not 1 <= experts.shape[1] <= min(n, 64):
        raise ValueError("experts must be tokens x k")
    k = experts.shape[1]
    _int32(experts, "experts", logits.device, (tokens, k))
    if dweights.dtype is not torch.float32 or tuple(dweights.shape) != (tokens, k) or dweights.device != logits.device:
        raise ValueError(f"dweights must be float32 of shape {(tokens, k)} on {logits.device}")
    return _rt._launched(_run_route_grad, logits.device, stream, score, dt, tokens, n, k, 1 if renormalize else 0, float(scale), logits, ld,
                         experts, dweights)


def _run_route_grad(score, dt, tokens, n, k, renormalize, scale, logits, ld, experts, dweights, handle):
    dweights = dweights.contiguous()
    dlogits = logits.new_empty((tokens, n))
    _rt._check(_lib().regtile_route_experts_grad(score, dt, tokens, n, k, renormalize, scale, logits.data_ptr(), ld, experts.data_ptr(),
                                                 dweights.data_ptr(), dlogits.data_ptr(), n, handle))
    return dlogits


def expert_rows_size(tokens, k, experts, align=1):
    """Rows that any choice of experts fits into."""
    n = tokens * k
    return (n + min(n, experts) * (align - 1) + align - 1) // align * align


class ExpertRows:
    """The rows that experts work on: the slots t * k + j in the order of their experts, each expert's from a multiple of
    ``align`` on (include/regtile.h). ``slots`` (rows), ``position`` (tokens x k), ``offsets`` (experts + 1) and
    ``counts`` (experts) are contiguous int32 tensors on one device; they are kept, not copied, and described anew where a call
    finds that their storage has been replaced."""

    __slots__ = ("tokens", "k", "experts", "align", "rows", "device", "_parts", "_parts_at", "_c", "_address")

    def __init__(self, slots, position, offsets, counts, align=1):
        _torch or _import_torch()
        if position.dim() != 2 or position.shape[1] < 1 or counts.dim() != 1 or counts.shape[0] < 1 or align < 1:
            raise ValueError("position must be tokens x k, counts one number for each expert, align at least 1")
        tokens, k = position.shape
        experts = counts.shape[0]
        self._parts, self.device = (slots, position, offsets, counts), slots.device
        self.tokens, self.k, self.experts, self.align, self.rows = tokens, k, experts, align, expert_rows_size(tokens, k, experts, align)
        self._describe()

    def _describe(self):
        for t, name, shape in zip(self._parts, ("slots", "position", "offsets", "counts"),
                                  ((self.rows,), (self.tokens, self.k), (self.experts + 1,), (self.experts,))):
            _int32(t, name, self.device, shape)
        self._set([t.data_ptr() for t in self._parts])

    def _set(self, at):
        self._parts_at = at
        self._c = RowsStruct(*at, self.tokens, self.k, self.experts, self.align, self.rows)
        self._address = ctypes.addressof(self._c)

    @property
    def _at(self):
        """The address of its regtile_expert_rows. (Parts that nobody has asked for are as they were made.)"""
        parts = self._parts
        if type(parts) is tuple:
            a, b, c, d = self._parts_at
            if parts[0].data_ptr() != a or parts[1].data_ptr() != b or parts[2].data_ptr() != c or parts[3].data_ptr() != d:
                self._describe()
        return self._address

    def _part(self, i):
        """slots, position, offsets or counts; the four lie in one tensor until one of them is asked for."""
        if type(self._parts) is not tuple:
            n, E = self.tokens * self.k, self.experts
            slots, position, offsets, counts = self._parts[:self.rows + n + 2 * E + 1].split((self.rows, n, E + 1, E))
            self._parts = slots, position.view(self.tokens, self.k), offsets, counts
        return self._parts[i]

    slots = property(lambda self: self._part(0))
    position = property(lambda self: self._part(1))
    offsets = property(lambda self: self._part(2))
    counts = property(lambda self: self._part(3))

    def token_of_row(self):
        """The token of each row (int32), -1 for rows without one: ``quantize_f8``'s ``rows`` for tokens in the
        experts' order."""
        return self.slots.div(self.k, rounding_mode="floor")

    def __repr__(self):
        return f"ExpertRows({self.rows} rows, {self.tokens} tokens x {self.k}, {self.experts} experts, align {self.align})"


def expert_rows(experts, n_experts, align=1, stream=None):
    """The ExpertRows of a choice (tokens x k int32, as ``route_experts`` gives it; numbers that are no expert leave
    their slot without a row) among ``n_experts``. ``align`` 128 is what ``gemm_f8_experts_dw`` needs."""
    _torch or _import_torch()
    if experts.dim() != 2 or experts.shape[1] < 1 or not experts.is_cuda:
        raise ValueError("experts must be a device tensor of tokens x k")
    _int32(experts, "experts", experts.device)
    if not 1 <= n_experts <= MAX_EXPERTS or align < 1:
        raise ValueError(f"1 to {MAX_EXPERTS} experts and an align of at least 1, not {n_experts} and {align}")
    tokens, k = experts.shape
    rows = expert_rows_size(tokens, k, n_experts, align)
    _rt._ints(tokens * k, rows)
    return _rt._launched(_run_rows, experts.device, stream, experts, tokens, k, n_experts, align, rows)


def _run_rows(experts, tokens, k, n_experts, align, rows, handle):
    lib = _lib()
    n = tokens * k
    # one tensor: slots, position, offsets, counts, and behind them (16 bytes aligned) the workspace that many slots need
    used = rows + n + 2 * n_experts + 1
    size = lib.regtile_order_experts_workspace(tokens, k, n_experts) if n > 4096 else 0
    start = (used + 3) // 4 * 4
    parts = experts.new_empty(start + (size + 3) // 4 if size else used)
    at = parts.data_ptr()
    r = object.__new__(ExpertRows)
    r._parts, r.device = parts, experts.device
    r.tokens, r.k, r.experts, r.align, r.rows = tokens, k, n_experts, align, rows
    r._set((at, at + 4 * rows, at + 4 * (rows + n), at + 4 * (rows + n + n_experts + 1)))
    status = lib.regtile_order_experts(experts.data_ptr(), r._address, at + 4 * start if size else None, size, handle)
    if status:
        _rt._check(status)
    return r


def _plan(name, rows, device):
    if not isinstance(rows, ExpertRows) or rows.device != device:
        raise ValueError(f"{name} takes ExpertRows on {device}")


def gemm_f8_experts(A, B, rows, C=None, gather=False, alpha=1.0, beta=0.0, dtype=None, stream=None):
    """The experts' products: row r of C (rows.rows x N) in expert e's group is alpha*A[r]@B[e] + beta*C[r]. ``B`` is a
    stack of F8Matrix (``W.t()`` for weights stored experts x N x K), ``A`` rows.rows x K, or with ``gather`` the
    tokens themselves (rows.tokens x K). Rows between groups become 0, rows behind the last group stay as
    they were (in a new C: are undefined). Returns C."""
    if not isinstance(rows, ExpertRows):
        raise ValueError("gemm_f8_experts takes ExpertRows")
    M, _, N = _operands("gemm_f8_experts", A, B, rows.experts)
    device = A.codes.device
    _plan("gemm_f8_experts", rows, device)
    if A.transposed:
        raise ValueError("gemm_f8_experts takes a row-major A")
    want = rows.tokens if gather else rows.rows
    if M != want:
        raise ValueError(f"A must have {want} rows, not {M}")
    dtype, dt, ldc = _c_of(C, dtype, beta, (rows.rows, N), device)
    return _rt._launched(_run_experts, device, stream, A, B, rows, C, 1 if gather else 0, float(alpha), float(beta), dtype, dt, N, ldc)


def _run_experts(A, B, rows, C, gather, alpha, beta, dtype, dt, N, ldc, handle):
    if C is None:
        C = A.codes.new_empty((rows.rows, N), dtype=dtype)
    lib, tb = _lib(), 1 if B.transposed else 0
    r, a, b = rows._at, A._at, B._at
    work, at, size = _workspace(A, lib.regtile_gemm_f8_experts_workspace(r, gather, tb, a, b, dt))
    status = lib.regtile_gemm_f8_experts(r, gather, tb, alpha, a, b, beta, dt, C.data_ptr(), ldc, at, size, handle)
    if status:
        _rt._check(status)
    return C


def gemm_f8_experts_dw(A, B, rows, C=None, alpha=1.0, beta=0.0, dtype=None, stream=None):
    """The gradient of each expert's matrix: C[e] = alpha*A[:, e's rows]@B[e's rows] + beta*C[e] (experts x M x N, float32
    by default). ``A`` (M x rows.rows) and ``B`` (rows.rows x N, a transposed F8Matrix) are quantised along the
    rows: ``gemm_f8_experts_dw(quantize_f8(dy, transpose=True), quantize_f8(x, transpose=True).t(), rows)`` for
    gradients and inputs in the experts' order (``rows=rows.token_of_row()`` takes the inputs from the tokens'). rows.align
    has to be a multiple of 128."""
    M, K, N = _operands("gemm_f8_experts_dw", A, B)
    device = A.codes.device
    _plan("gemm_f8_experts_dw", rows, device)
    if rows.align % F8_BLOCK:
        raise ValueError(f"gemm_f8_experts_dw needs rows aligned to {F8_BLOCK}, not {rows.align}")
    if A.transposed or not B.transposed or A.block_rows != 1 or B.block_rows != 1:
        raise ValueError(f"gemm_f8_experts_dw takes a row-major A and a transposed B in blocks of 1 x {F8_BLOCK}")
    if K != rows.rows:
        raise ValueError(f"the operands must have {rows.rows} rows inside, not {K}")
    dtype, dt, ldc = _c_of(C, dtype, beta, (rows.experts, M, N), device)
    return _rt._launched(_run_experts_dw, device, stream, A, B, rows, C, float(alpha), float(beta), dtype, dt, M, N, ldc)


def _run_experts_dw(A, B, rows, C, alpha, beta, dtype, dt, M, N, ldc, handle):
    if C is None:
        C = A.codes.new_empty((rows.experts, M, N), dtype=dtype)
    lib = _lib()
    r, a, b = rows._at, A._at, B._at
    work, at, size = _workspace(A, lib.regtile_gemm_f8_experts_dw_workspace(r, a, b, dt))
    status = lib.regtile_gemm_f8_experts_dw(r, alpha, a, b, beta, dt, C.data_ptr(), ldc, C.stride(0), at, size, handle)
    if status:
        _rt._check(status)
    return C


def _weights(weights, rows, device):
    if weights is not None and (weights.dtype is not _torch.float32 or tuple(weights.shape) != (rows.tokens, rows.k) or
                                not weights.is_contiguous() or weights.device != device):
        raise ValueError(f"weights must be a contiguous float32 tensor of {(rows.tokens, rows.k)} on {device}")


def combine_experts(Y, rows, weights=None, out=None, stream=None):
    """Each token's sum of its experts' rows, with ``weights`` (tokens x k, float32; all 1 when None): tokens x N from
    Y (rows.rows x N, row-major), in Y's dtype. Slots without a row add nothing. Writes into ``out`` or a new tensor, and
    returns it."""
    _torch or _import_torch()
    dt = _rt._mx_dtype(Y.dtype, "Y")
    _plan("combine_experts", rows, Y.device)
    ldy, n_rows, n = _rt._rows(Y, "Y")
    if n_rows != rows.rows:
        raise ValueError(f"Y must have {rows.rows} rows, not {n_rows}")
    _weights(weights, rows, Y.device)
    if out is not None and (out.dtype is not Y.dtype or tuple(out.shape) != (rows.tokens, n) or out.device != Y.device):
        raise ValueError(f"out must be {Y.dtype} of shape {(rows.tokens, n)} on {Y.device}")
    ldo = max(n, 1) if out is None else _rt._rows(out, "out")[0]
    _rt._ints(ldy, n, ldo)
    return _rt._launched(_run_combine, Y.device, stream, Y, rows, weights, out, dt, n, ldy, ldo)


def _run_combine(Y, rows, weights, out, dt, n, ldy, ldo, handle):
    if out is None:
        out = Y.new_empty((rows.tokens, n))
    _rt._check(_lib().regtile_combine_experts(rows._at, dt, n, Y.data_ptr(), ldy, None if weights is None else weights.data_ptr(),
                                              out.data_ptr(), ldo, handle))
    return out


def combine_experts_grad(dout, Y, rows, weights=None, stream=None):
    """(dY, dweights) of ``combine_experts``: dY (rows.rows x N, Y's dtype; 0 for rows without a slot) and dweights
    (tokens x k, float32; None when weights is None, and Y is then not read and may be None)."""
    _torch or _import_torch()
    dt = _rt._mx_dtype(dout.dtype, "dout")
    _plan("combine_experts_grad", rows, dout.device)
    ldd, tokens, n = _rt._rows(dout, "dout")
    if tokens != rows.tokens:
        raise ValueError(f"dout must have {rows.tokens} rows, not {tokens}")
    _weights(weights, rows, dout.device)
    ldy = 0
    if weights is not None:
        if Y is None or Y.dtype is not dout.dtype or tuple(Y.shape) != (rows.rows, n) or Y.device != dout.device:
            raise ValueError(f"Y must be {dout.dtype} of shape {(rows.rows, n)} on {dout.device}")
        ldy = _rt._rows(Y, "Y")[0]
    _rt._ints(ldd, n, ldy)
    return _rt._launched(_run_combine_grad, dout.device, stream, dout, Y, rows, weights, dt, n, ldd, ldy)


def _run_combine_grad(dout, Y, rows, weights, dt, n, ldd, ldy, handle):
    dY = dout.new_empty((rows.rows, n))
    dweights = None if weights is None else dout.new_empty((rows.tokens, rows.k), dtype=_torch.float32)
    some = weights is not None
    _rt._check(_lib().regtile_combine_experts_grad(rows._at, dt, n, dout.data_ptr(), ldd, Y.data_ptr() if some else None, ldy,
                                                   weights.data_ptr() if some else None, dY.data_ptr(), max(n, 1),
                                                   dweights.data_ptr() if some else None, handle))
    return dY, dweights
