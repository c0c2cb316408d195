"""register_tiled_matrix_amd -- register-tiled GEMM for MI355X (gfx950), Python binding.

A thin ctypes binding over the C ABI of ``libregtile.so`` (declared in ``include/regtile.h``).
It only marshals arguments: every step of the product runs in the library's HIP kernels.
PyTorch supplies device memory and the current HIP stream.

Entry points (same names as the C ABI):

* ``gemm_f32(A, B, C=None, alpha=1.0, beta=0.0, algo=ALGO_F32_AUTO)``
  fp32 ``C = alpha*A@B + beta*C``; A (M x K) and B (K x N) row-major fp32 CUDA tensors
  (row stride may exceed the width), C (M x N) row-major fp32.
* ``gemm_bf16(A, B, C=None, alpha=1.0, beta=0.0, algo=ALGO_BF16_AUTO)``
  bf16 A (M x K) times bf16 B (K x N), fp32 C; the fast path is row-major A with B given as a
  column-major view (for example ``Bt.t()`` for a contiguous N x K tensor ``Bt``).
* Every tensor entry point accepts A and B either row-major or as transposed (column-major)
  views and passes the layout to the ``regtile_gemm_*_ex`` entry points.
* ``gemm_f16(A, B, C=None, alpha=1.0, beta=0.0, algo=ALGO_BF16_AUTO)`` the same with
  float16 A and B (IEEE binary16); the algorithm values are the bf16 ones.
* ``gemm_bf16_mx(A, B, C=None, alpha=1.0, beta=0.0)`` / ``gemm_f16_mx`` the same products with a
  block-scaled B (``MXMatrix``: 4 or 8 bits an element, one power-of-two scale per group of 32 along
  its rows). For a linear layer with weights ``W`` held as an MXMatrix (out x in):
  ``y = gemm_bf16_mx(x, W.t())`` and ``dx = gemm_bf16_mx(dy, W)``; for an input ``X`` kept as an MXMatrix
  (tokens x in): ``dW = gemm_bf16_mx(dy.t(), X)``.
* ``quantize_mx(X, format)`` -> MXMatrix and ``dequantize_mx(Q, dtype=torch.bfloat16)``; ``MX_FP4`` holds
  weights in 4.25 bits, ``MX_INT8`` activations (a checkpoint for the backward pass) in 8.25.
* ``gemm_f8(A, B, C=None, alpha=1.0, beta=0.0, dtype=torch.float32)`` with both operands block-scaled 8-bit
  floats (``F8Matrix``: e4m3 or e5m2, one fp32 scale per 1 x 128 or 128 x 128 values), from ``quantize_f8``.
* ``route_experts`` (and ``route_experts_grad``), ``expert_rows``, ``gemm_f8_experts`` (and
  ``gemm_f8_experts_dw``) and ``combine_experts`` (and ``combine_experts_grad``): a mixture of experts, whose rows
  fall into groups with a matrix each.
* ``gemm_f32_raw`` / ``gemm_bf16_raw`` / ``gemm_f16_raw`` take the C arguments verbatim
  (integers for pointers).
* ``last_kernel()``, ``last_kernel_info()`` (registers, LDS, scratch and occupancy of that
  kernel, from the HIP runtime), ``strerror(status)``, ``version()``.

The library must be built (``python -m register_tiled_matrix_amd.build``); importing this
package does not build it, and every call raises ``RegtileLibraryMissing`` when it is absent.
"""
from __future__ import annotations

import ctypes
import os
import threading

__all__ = [
    "ALGO_F32_AUTO", "ALGO_F32_NAIVE", "ALGO_F32_LDS", "ALGO_F32_REGTILE", "ALGO_F32_SPLITK",
    "ALGO_F32_REGTILE_SMALL",
    "ALGO_BF16_AUTO", "ALGO_BF16_NAIVE", "ALGO_BF16_MFMA", "ALGO_BF16_MFMA_16X16", "ALGO_BF16_MFMA_SPLITK",
    "RegtileError", "RegtileLibraryMissing", "lib_path", "load",
    "gemm_f32", "gemm_bf16", "gemm_f16", "gemm_f32_raw", "gemm_bf16_raw", "gemm_f16_raw",
    "regtile_gemm_f32_algo", "regtile_gemm_bf16_algo", "regtile_gemm_f16_algo",
    "regtile_gemm_f32_ex", "regtile_gemm_bf16_ex", "regtile_gemm_f16_ex",
    "MX_FP4", "MX_INT8", "MX_GROUP", "MXMatrix", "quantize_mx", "dequantize_mx", "gemm_bf16_mx", "gemm_f16_mx",
    "regtile_quantize_mx", "regtile_dequantize_mx", "regtile_gemm_bf16_mx", "regtile_gemm_f16_mx",
    "regtile_gemm_mx_workspace", "regtile_gemm_mx_workspace_ex", "last_kernel", "last_kernel_info", "strerror", "version", "EXPORTED_SYMBOLS",
]

ALGO_F32_AUTO, ALGO_F32_NAIVE, ALGO_F32_LDS, ALGO_F32_REGTILE, ALGO_F32_SPLITK = 0, 1, 2, 3, 4
ALGO_F32_REGTILE_SMALL = 5
ALGO_BF16_AUTO, ALGO_BF16_NAIVE, ALGO_BF16_MFMA, ALGO_BF16_MFMA_16X16, ALGO_BF16_MFMA_SPLITK = 0, 1, 2, 3, 4
MX_FP4, MX_INT8 = 0, 1  # regtile_mx_format
MX_GROUP = 32  # columns that share a scale

EXPORTED_SYMBOLS = ("gemm_f32", "gemm_bf16", "gemm_f16", "regtile_gemm_f32_algo",
                    "regtile_gemm_bf16_algo", "regtile_gemm_f16_algo", "regtile_gemm_f32_ex",
                    "regtile_gemm_bf16_ex", "regtile_gemm_f16_ex",
                    "regtile_quantize_mx", "regtile_dequantize_mx", "regtile_gemm_bf16_mx",
                    "regtile_gemm_f16_mx", "regtile_gemm_mx_workspace", "regtile_gemm_mx_workspace_ex",
                    "regtile_last_kernel", "regtile_last_kernel_info", "regtile_strerror",
                    "regtile_version", "regtile_quantize_f8", "regtile_dequantize_f8", "regtile_gemm_f8",
                    "regtile_gemm_f8_workspace", "regtile_expert_rows_size", "regtile_order_experts",
                    "regtile_order_experts_workspace", "regtile_gemm_f8_experts", "regtile_gemm_f8_experts_dw",
                    "regtile_gemm_f8_experts_workspace", "regtile_gemm_f8_experts_dw_workspace",
                    "regtile_route_experts", "regtile_route_experts_grad", "regtile_combine_experts",
                    "regtile_combine_experts_grad")

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_HERE, "libregtile.so")
_lib = None
_lock = threading.Lock()


class KernelInfo(ctypes.Structure):
    """regtile_kernel_info of include/regtile.h."""
    _fields_ = [("workgroup_size", ctypes.c_int), ("registers", ctypes.c_int), ("lds_bytes", ctypes.c_int),
                ("scratch_bytes", ctypes.c_int), ("workgroups_per_cu", ctypes.c_int),
                ("waves_per_simd", ctypes.c_int)]


class RegtileError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"regtile status {status}: {message}")
        self.status = status


class RegtileLibraryMissing(RuntimeError):
    pass


def lib_path() -> str:
    return _LIB_PATH


def load():
    """Load libregtile.so (once) and declare the C signatures."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(_LIB_PATH):
            raise RegtileLibraryMissing(
                f"{_LIB_PATH} is not built; run `python -m register_tiled_matrix_amd.build`")
        lib = ctypes.CDLL(_LIB_PATH)
        I, F, P = ctypes.c_int, ctypes.c_float, ctypes.c_void_p
        gemm = [I, I, I, F, P, I, P, I, F, P, I, P]
        gemm_mx = [I, I, I, I, I, I, F, P, I, P, I, P, I, F, P, I, P, ctypes.c_int64, P]
        convert_mx = [I, I, I, I, P, I, P, I, P, I, P]
        for name, args in (("regtile_gemm_bf16_mx", gemm_mx), ("regtile_gemm_f16_mx", gemm_mx),
                           ("regtile_quantize_mx", convert_mx), ("regtile_dequantize_mx", convert_mx),
                           ("gemm_f32", gemm), ("gemm_bf16", gemm), ("gemm_f16", gemm),
                           ("regtile_gemm_f16_algo", [I] + gemm),
                           ("regtile_gemm_f32_ex", [I, I, I] + gemm),
                           ("regtile_gemm_bf16_ex", [I, I, I] + gemm),
                           ("regtile_gemm_f16_ex", [I, I, I] + gemm),
                           ("regtile_gemm_f32_algo", [I] + gemm),
                           ("regtile_gemm_bf16_algo", [I] + gemm)):
            f = getattr(lib, name)
            f.argtypes = args
            f.restype = I
        lib.regtile_gemm_mx_workspace.argtypes = [I] * 7
        lib.regtile_gemm_mx_workspace.restype = ctypes.c_int64
        lib.regtile_gemm_mx_workspace_ex.argtypes = [I, I, I, I, I, I, P, I, P, I, P, I, I]
        lib.regtile_gemm_mx_workspace_ex.restype = ctypes.c_int64
        _f8.declare(lib)
        lib.regtile_last_kernel.argtypes = []
        lib.regtile_last_kernel.restype = ctypes.c_char_p
        lib.regtile_last_kernel_info.argtypes = [ctypes.POINTER(KernelInfo)]
        lib.regtile_last_kernel_info.restype = I
        lib.regtile_strerror.argtypes = [I]
        lib.regtile_strerror.restype = ctypes.c_char_p
        lib.regtile_version.argtypes = []
        lib.regtile_version.restype = I
        _lib = lib
        return lib


def last_kernel() -> str:
    return load().regtile_last_kernel().decode()


def last_kernel_info() -> dict:
    """Resources of the kernel this thread launched last (regtile_last_kernel_info)."""
    info = KernelInfo()
    _check(load().regtile_last_kernel_info(ctypes.byref(info)))
    return {name: getattr(info, name) for name, _ in KernelInfo._fields_}


def strerror(status: int) -> str:
    return load().regtile_strerror(int(status)).decode()


def version() -> int:
    return int(load().regtile_version())


def _check(status: int) -> None:
    if status != 0:
        raise RegtileError(status, strerror(status))


# ---- raw entry points: the C arguments verbatim -------------------------------------------
def gemm_f32_raw(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream=0) -> int:
    return load().gemm_f32(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream)


def gemm_bf16_raw(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream=0) -> int:
    return load().gemm_bf16(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream)


def regtile_gemm_f32_algo(algo, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream=0) -> int:
    return load().regtile_gemm_f32_algo(algo, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc,
                                        stream)


def gemm_f16_raw(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream=0) -> int:
    return load().gemm_f16(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream)


def regtile_gemm_f16_algo(algo, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream=0) -> int:
    return load().regtile_gemm_f16_algo(algo, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc,
                                        stream)


def regtile_gemm_f32_ex(algo, trans_a, trans_b, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc,
                        stream=0) -> int:
    return load().regtile_gemm_f32_ex(algo, trans_a, trans_b, M, N, K, alpha, A, lda, B, ldb,
                                      beta, C, ldc, stream)


def regtile_gemm_bf16_ex(algo, trans_a, trans_b, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc,
                         stream=0) -> int:
    return load().regtile_gemm_bf16_ex(algo, trans_a, trans_b, M, N, K, alpha, A, lda, B, ldb,
                                       beta, C, ldc, stream)


def regtile_gemm_f16_ex(algo, trans_a, trans_b, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc,
                        stream=0) -> int:
    return load().regtile_gemm_f16_ex(algo, trans_a, trans_b, M, N, K, alpha, A, lda, B, ldb,
                                      beta, C, ldc, stream)


def regtile_gemm_bf16_algo(algo, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream=0) -> int:
    return load().regtile_gemm_bf16_algo(algo, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc,
                                         stream)


def regtile_gemm_bf16_mx(format, trans_a, trans_b, M, N, K, alpha, A, lda, Q, ldq, S, lds, beta, C, ldc,
                         work=0, work_bytes=0, stream=0) -> int:
    return load().regtile_gemm_bf16_mx(format, trans_a, trans_b, M, N, K, alpha, A, lda, Q, ldq, S, lds,
                                       beta, C, ldc, work, work_bytes, stream)


def regtile_gemm_f16_mx(format, trans_a, trans_b, M, N, K, alpha, A, lda, Q, ldq, S, lds, beta, C, ldc,
                        work=0, work_bytes=0, stream=0) -> int:
    return load().regtile_gemm_f16_mx(format, trans_a, trans_b, M, N, K, alpha, A, lda, Q, ldq, S, lds,
                                      beta, C, ldc, work, work_bytes, stream)


def regtile_gemm_mx_workspace(trans_a, trans_b, M, N, K, lda, ldc) -> int:
    return load().regtile_gemm_mx_workspace(trans_a, trans_b, M, N, K, lda, ldc)


def regtile_gemm_mx_workspace_ex(format, trans_a, trans_b, M, N, K, A, lda, Q, ldq, S, lds, ldc) -> int:
    return load().regtile_gemm_mx_workspace_ex(format, trans_a, trans_b, M, N, K, A, lda, Q, ldq, S, lds, ldc)


def regtile_quantize_mx(format, dtype, rows, cols, X, ldx, Q, ldq, S, lds, stream=0) -> int:
    return load().regtile_quantize_mx(format, dtype, rows, cols, X, ldx, Q, ldq, S, lds, stream)


def regtile_dequantize_mx(format, dtype, rows, cols, Q, ldq, S, lds, X, ldx, stream=0) -> int:
    return load().regtile_dequantize_mx(format, dtype, rows, cols, Q, ldq, S, lds, X, ldx, stream)


# ---- tensor entry points -------------------------------------------------------------------
def _stream_handle(t, stream):
    import torch

    if stream is None:
        return torch.cuda.current_stream(t.device).cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _row_major_ld(t, name):
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D")
    if t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError(f"{name} must be row-major (unit column stride)")
    if t.shape[0] > 1 and t.stride(0) < t.shape[1]:
        raise ValueError(f"{name} rows overlap (row stride below the width)")
    return max(int(t.stride(0)), int(t.shape[1]), 1)


def _layout(t, name):
    """(trans, ld) of a 2-D operand: row-major storage (unit column stride) -> (0, row stride);
    column-major storage (unit row stride), i.e. the transpose of a row-major matrix ->
    (1, column stride). Anything else (overlapping or non-unit strides) is rejected."""
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D")
    r, c = t.shape
    if (c <= 1 or t.stride(1) == 1) and (r <= 1 or t.stride(0) >= c):
        return 0, max(int(t.stride(0)), int(c), 1)
    if (r <= 1 or t.stride(0) == 1) and (c <= 1 or t.stride(1) >= r):
        return 1, max(int(t.stride(1)), int(r), 1)
    raise ValueError(f"{name} must be row-major or column-major with non-overlapping rows")


def _out(C, M, N, like):
    import torch

    if C is None:
        return torch.empty((M, N), dtype=torch.float32, device=like.device)
    if C.dtype != torch.float32 or tuple(C.shape) != (M, N):
        raise ValueError(f"C must be float32 of shape {(M, N)}")
    return C


def _gemm(fn, want, label, A, B, C, alpha, beta, algo, stream):
    if A.dtype != want or B.dtype != want:
        raise ValueError(f"{label} takes {want} A and B")
    if not (A.is_cuda and B.is_cuda):
        raise ValueError(f"{label} takes device tensors")
    M, K = A.shape
    K2, N = B.shape
    if K != K2:
        raise ValueError(f"inner dimensions differ: {K} vs {K2}")
    if C is None and beta != 0.0:
        raise ValueError("beta != 0 needs C")
    C = _out(C, M, N, A)
    (ta, lda), (tb, ldb) = _layout(A, "A"), _layout(B, "B")
    ldc = _row_major_ld(C, "C")
    st = fn(int(algo), ta, tb, M, N, K, float(alpha), A.data_ptr(), lda, B.data_ptr(), ldb,
            float(beta), C.data_ptr(), ldc, _stream_handle(A, stream))
    _check(st)
    return C


def gemm_f32(A, B, C=None, alpha=1.0, beta=0.0, algo=ALGO_F32_AUTO, stream=None):
    """C = alpha*A@B + beta*C on fp32 CUDA tensors; returns C (allocated when None). A and B
    may each be row-major or a transposed (column-major) view; C is row-major."""
    import torch

    return _gemm(regtile_gemm_f32_ex, torch.float32, "gemm_f32", A, B, C, alpha, beta, algo,
                 stream)


def gemm_bf16(A, B, C=None, alpha=1.0, beta=0.0, algo=ALGO_BF16_AUTO, stream=None):
    """C = alpha*A@B + beta*C; bf16 A (M x K) and B (K x N), each row-major or a transposed
    view (the fast path is row-major A with column-major B, e.g. ``Bt.t()``), fp32 C row-major;
    returns C (allocated when None)."""
    import torch

    return _gemm(regtile_gemm_bf16_ex, torch.bfloat16, "gemm_bf16", A, B, C, alpha, beta, algo,
                 stream)


def gemm_f16(A, B, C=None, alpha=1.0, beta=0.0, algo=ALGO_BF16_AUTO, stream=None):
    """As gemm_bf16 with float16 (IEEE binary16) A and B."""
    import torch

    return _gemm(regtile_gemm_f16_ex, torch.float16, "gemm_f16", A, B, C, alpha, beta, algo,
                 stream)


# ---- block-scaled (MX) operands --------------------------------------------------------------
_INT_MAX = 2**31 - 1


def _row_bytes(format, cols):
    return (cols + 1) // 2 if format == MX_FP4 else cols


def _check_format(format):
    if format != MX_FP4 and format != MX_INT8:
        raise ValueError(f"unknown block-scaled format {format!r}")


_torch = None  # torch, once the first of these calls needs it
_get_device = _get_stream = None  # the current device's index; the current stream's handle on a device
_mx_dtypes = {}  # regtile_mx_dtype by torch dtype


def _import_torch():
    global _torch, _get_device, _get_stream
    import torch

    # the plain numbers, without Device and Stream objects around them
    _get_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
    _get_stream = getattr(torch._C, "_cuda_getCurrentRawStream", lambda i: torch.cuda.current_stream(i).cuda_stream)
    _mx_dtypes.update({torch.float32: 0, torch.bfloat16: 1, torch.float16: 2})
    _torch = torch
    return torch


def _rows(t, name):
    """(leading dimension, rows, columns) of a row-major 2-D tensor; others are rejected."""
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D")
    rows, cols = t.shape
    row, col = t.stride()
    if (col == 1 or cols <= 1) and (row >= cols or rows <= 1):
        return max(row, cols, 1), rows, cols
    return _row_major_ld(t, name), rows, cols  # raises


class MXMatrix:
    """A block-scaled matrix of ``rows`` x ``cols`` values (include/regtile.h states the layout).

    ``codes``: uint8, rows x (cols + 1) // 2 bytes (``MX_FP4``) or rows x cols (``MX_INT8``, int8 is
    taken too); ``scales``: uint8, rows x ceil(cols / 32). Both have unit column stride (their row
    strides may exceed the width) and live on one device. ``t()`` is the transposed view: the same
    bytes, taken as cols x rows. The tensors are kept, not copied.
    """

    __slots__ = ("format", "codes", "scales", "transposed", "_rows", "_cols", "_ldq", "_lds")

    def __init__(self, format, codes, scales, cols, transposed=False):
        torch = _torch or _import_torch()
        _check_format(format)
        cols = int(cols)
        if codes.dtype is not torch.uint8 and not (codes.dtype is torch.int8 and format == MX_INT8):
            raise ValueError("codes must be uint8 (int8 is taken for MX_INT8)")
        if scales.dtype is not torch.uint8:
            raise ValueError("scales must be uint8")
        self._ldq, rows, width = _rows(codes, "codes")
        self._lds, srows, groups = _rows(scales, "scales")
        if cols < 0 or width != _row_bytes(format, cols):
            raise ValueError(f"codes must be {_row_bytes(format, cols)} bytes wide for {cols} columns, not {width}")
        if srows != rows or groups != -(-cols // MX_GROUP):
            raise ValueError(f"scales must be {(rows, -(-cols // MX_GROUP))}, not {(srows, groups)}")
        if codes.device != scales.device:
            raise ValueError("codes and scales are on different devices")
        self.format, self.codes, self.scales = format, codes, scales
        self.transposed = bool(transposed)
        self._rows, self._cols = rows, cols

    @property
    def shape(self):
        return (self._cols, self._rows) if self.transposed else (self._rows, self._cols)

    @property
    def device(self):
        return self.codes.device

    @classmethod
    def _of(cls, format, codes, scales, rows, cols, ldq, lds, transposed):
        """A matrix of parts that are known to fit."""
        v = object.__new__(cls)
        v.format, v.codes, v.scales, v.transposed = format, codes, scales, transposed
        v._rows, v._cols, v._ldq, v._lds = rows, cols, ldq, lds
        return v

    def t(self):
        return self._of(self.format, self.codes, self.scales, self._rows, self._cols, self._ldq, self._lds, not self.transposed)

    def __repr__(self):
        name = "MX_FP4" if self.format == MX_FP4 else "MX_INT8"
        return f"MXMatrix({name}, {self.shape[0]} x {self.shape[1]}{', transposed' if self.transposed else ''})"


class _Launch:
    """Makes `device` the current device and `stream` (None: that device's current one) its current
    stream for what is allocated and launched inside, so that the allocator knows where the memory
    is used; entering gives the stream's handle."""

    __slots__ = ("_device", "_stream")

    def __init__(self, device, stream):
        import torch

        if stream is None:
            stream = torch.cuda.current_stream(device)
        elif isinstance(stream, int):
            # (an ExternalStream of handle 0 would be another stream than the default one)
            stream = torch.cuda.ExternalStream(stream, device=device) if stream else torch.cuda.default_stream(device)
        if stream.device != device:
            raise ValueError(f"the stream is on {stream.device}, the operands on {device}")
        self._device, self._stream = torch.cuda.device(device), torch.cuda.stream(stream)

    def __enter__(self):
        self._device.__enter__()
        self._stream.__enter__()
        return self._stream.stream.cuda_stream

    def __exit__(self, *exc):
        self._stream.__exit__(*exc)
        self._device.__exit__(*exc)


def _launched(run, device, stream, *args):
    """run(*args, handle) on `device` and `stream`, as _Launch arranges it where that is not the
    current device and stream already."""
    index = device.index
    if stream is None and _get_device() == index:
        return run(*args, _get_stream(index))
    with _Launch(device, stream) as handle:
        return run(*args, handle)


def _ints(*values):
    if max(values) > _INT_MAX:
        raise ValueError(f"sizes and leading dimensions go up to 2**31 - 1, not {max(values)}")


def _mx_dtype(dtype, name):
    if _torch is None:
        _import_torch()
    try:
        return _mx_dtypes[dtype]
    except KeyError:
        raise ValueError(f"{name} must be float32, bfloat16 or float16, not {dtype}") from None


def quantize_mx(X, format=MX_INT8, out=None, stream=None):
    """The block-scaled form of a row-major device tensor X (float32, bfloat16 or float16); groups
    run along its rows. Writes into ``out`` (an MXMatrix of X's shape and the format) or a new
    MXMatrix, and returns it."""
    _check_format(format)
    dt = _mx_dtype(X.dtype, "X")
    if not X.is_cuda:
        raise ValueError("quantize_mx takes a device tensor")
    ldx, rows, cols = _rows(X, "X")
    if out is not None and (not isinstance(out, MXMatrix) or out.format != format or out.transposed or
                            out.shape != (rows, cols) or out.device != X.device):
        raise ValueError(f"out must be an untransposed MXMatrix of format {format}, shape {(rows, cols)} on {X.device}")
    return _launched(_run_quantize, X.device, stream, X, format, dt, rows, cols, ldx, out)


def _run_quantize(X, format, dt, rows, cols, ldx, Q, handle):
    if Q is None:
        u8, width, groups = _torch.uint8, _row_bytes(format, cols), -(-cols // MX_GROUP)
        Q = MXMatrix._of(format, X.new_empty((rows, width), dtype=u8), X.new_empty((rows, groups), dtype=u8), rows, cols,
                         max(width, 1), max(groups, 1), False)
    _ints(rows, cols, ldx, Q._ldq, Q._lds)
    _check((_lib or load()).regtile_quantize_mx(format, dt, rows, cols, X.data_ptr(), ldx, Q.codes.data_ptr(), Q._ldq,
                                                Q.scales.data_ptr(), Q._lds, handle))
    return Q


def dequantize_mx(Q, dtype=None, out=None, stream=None):
    """The values of an MXMatrix as a row-major tensor of its shape (of a transposed one: the
    transposed view of a row-major tensor), rounded to ``dtype`` (bfloat16 when neither it nor ``out``
    is given). Writes into ``out`` or a new tensor, and returns it."""
    torch = _torch or _import_torch()
    if not isinstance(Q, MXMatrix) or not Q.codes.is_cuda:
        raise ValueError("dequantize_mx takes an MXMatrix of device tensors")
    if dtype is None:
        dtype = torch.bfloat16 if out is None else out.dtype
    dt = _mx_dtype(dtype, "dtype")
    if out is not None and (out.dtype != dtype or tuple(out.shape) != Q.shape or out.device != Q.device):
        raise ValueError(f"out must be {dtype} of shape {Q.shape} on {Q.device}")
    X = _launched(_run_dequantize, Q.device, stream, Q, dtype, dt, out)
    if out is not None:
        return out
    return X.t() if Q.transposed else X


def _run_dequantize(Q, dtype, dt, out, handle):
    if out is None:
        X = Q.codes.new_empty((Q._rows, Q._cols), dtype=dtype)
    else:
        X = out.t() if Q.transposed else out
    ldx, rows, cols = _rows(X, "out")
    _ints(rows, cols, ldx, Q._ldq, Q._lds)
    _check((_lib or load()).regtile_dequantize_mx(Q.format, dt, rows, cols, Q.codes.data_ptr(), Q._ldq,
                                                  Q.scales.data_ptr(), Q._lds, X.data_ptr(), ldx, handle))
    return X


def _gemm_mx(name, want, A, B, C, alpha, beta, stream):
    if not isinstance(B, MXMatrix):
        raise ValueError(f"{name} takes an MXMatrix B")
    if A.dtype is not want:
        raise ValueError(f"{name} takes {want} A")
    device = A.device
    if not A.is_cuda or B.codes.device != device or (C is not None and C.device != device):
        raise ValueError(f"{name} takes device tensors, all on one device")
    ta, lda = _layout(A, "A")
    M, K = A.shape
    tb = B.transposed
    K2, N = (B._cols, B._rows) if tb else (B._rows, B._cols)
    if K != K2:
        raise ValueError(f"inner dimensions differ: {K} vs {K2}")
    if C is None:
        if beta != 0.0:
            raise ValueError("beta != 0 needs C")
        ldc = N if N > 0 else 1
    else:
        ldc = _rows(_out(C, M, N, A), "C")[0]
    _ints(M, N, K, lda, ldc, B._ldq, B._lds)
    return _launched(_run_gemm_mx, device, stream, name, A, ta, lda, B, 1 if tb else 0, M, N, K, C, ldc, alpha, beta)


def _run_gemm_mx(name, A, ta, lda, B, tb, M, N, K, C, ldc, alpha, beta, handle):
    lib = _lib or load()
    if C is None:
        C = A.new_empty((M, N), dtype=_torch.float32)
    a, q, s = A.data_ptr(), B.codes.data_ptr(), B.scales.data_ptr()
    work, at, size = None, None, 0
    # K is split into parts of 512 at least, and not at all by the kernels for a few rows of A: those take
    # row-major A and B stored N x K, up to 32 rows, and up to 64 where the rows are aligned for DMA
    if K >= 1024 and (M > 64 or ta or not tb or
                      (M > 32 and ((a | q) & 15 or lda & 7 or B._ldq & 15 or s & 3 or B._lds & 3))):
        size = lib.regtile_gemm_mx_workspace_ex(B.format, ta, tb, M, N, K, a, lda, q, B._ldq, s, B._lds, ldc)
        if size > 0:
            work = A.new_empty(size, dtype=_torch.uint8)  # stays until the launch is queued
            at = work.data_ptr()
    status = getattr(lib, name)(B.format, ta, tb, M, N, K, alpha, a, lda, q, B._ldq, s, B._lds, beta, C.data_ptr(), ldc,
                                at, size, handle)
    if status:
        _check(status)
    return C


def gemm_bf16_mx(A, B, C=None, alpha=1.0, beta=0.0, stream=None):
    """C = alpha*A@B + beta*C; bf16 A (M x K), row-major or a transposed view, times a block-scaled B
    (an MXMatrix, K x N; ``W.t()`` for weights stored N x K), fp32 C row-major; returns C (allocated
    when None)."""
    return _gemm_mx("regtile_gemm_bf16_mx", (_torch or _import_torch()).bfloat16, A, B, C, float(alpha), float(beta), stream)


def gemm_f16_mx(A, B, C=None, alpha=1.0, beta=0.0, stream=None):
    """As gemm_bf16_mx with a float16 A; B's values are taken in float16."""
    return _gemm_mx("regtile_gemm_f16_mx", (_torch or _import_torch()).float16, A, B, C, float(alpha), float(beta), stream)


from . import _f8  # noqa: E402
from ._f8 import *  # noqa: E402,F401,F403

__all__ += _f8.__all__
