"""The block-scaled formats in plain numpy, 64 bits: the reference of the tests.

Encoding walks the definition (largest exponent of the group, nearest element, ties to the even
code); decoding is a table. Nothing here is shared with the library."""
from __future__ import annotations

import numpy as np

FP4, INT8 = 0, 1
GROUP = 32
FP4_VALUES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def widths(fmt: int, cols: int) -> tuple[int, int]:
    """(code bytes, scale bytes) of a row."""
    return ((cols + 1) // 2 if fmt == FP4 else cols), -(-cols // GROUP)


def elements(codes: np.ndarray, fmt: int, cols: int) -> np.ndarray:
    """Element values without their scales (int8: q, not q / 64)."""
    codes = np.asarray(codes, dtype=np.uint8)
    if fmt == INT8:
        return codes[:, :cols].astype(np.int8).astype(np.float64)
    nib = np.stack((codes & 15, codes >> 4), axis=-1).reshape(codes.shape[0], -1)[:, :cols]
    v = FP4_VALUES[nib & 7]
    return np.where(nib >= 8, -v, v)


def decode(codes: np.ndarray, scales: np.ndarray, fmt: int, cols: int) -> np.ndarray:
    """float64 values; a scale byte of 255 makes its group NaN."""
    e = scales.astype(np.int64) - (127 if fmt == FP4 else 133)
    step = np.where(scales == 255, np.nan, np.ldexp(1.0, e))
    return elements(codes, fmt, cols) * np.repeat(step, GROUP, axis=1)[:, :cols]


def encode(x: np.ndarray, fmt: int) -> tuple[np.ndarray, np.ndarray]:
    """(codes, scales) of a rows x cols float64 matrix."""
    rows, cols = x.shape
    ng = -(-cols // GROUP)
    g = np.zeros((rows, ng * GROUP))
    g[:, :cols] = x
    g = g.reshape(rows, ng, GROUP)
    bad = ~np.isfinite(g).all(-1)
    a = np.abs(np.where(np.isfinite(g), g, 0.0)).max(-1)
    e = np.where(a > 0, np.frexp(a)[1] - 1, -1000) + 127 - (2 if fmt == FP4 else 0)
    E = np.clip(e, 0, 254)
    with np.errstate(invalid="ignore"):
        y = np.where(bad[..., None], 0.0, np.ldexp(g, ((127 if fmt == FP4 else 133) - E)[..., None]))
    E = np.where(bad, 255, E).astype(np.uint8)
    if fmt == INT8:
        q = np.clip(np.rint(y), -127, 127).astype(np.int8).view(np.uint8)
        return np.ascontiguousarray(q.reshape(rows, -1)[:, :cols]), E
    dist = np.abs(np.abs(y)[..., None] - FP4_VALUES)  # exact
    best = dist.min(-1, keepdims=True)
    near = dist == best
    even = near & (np.arange(8) % 2 == 0)  # of two equally near codes one is even
    code = np.where(even.any(-1), even.argmax(-1), near.argmax(-1)).astype(np.uint8)
    code |= (np.signbit(y).astype(np.uint8) << 3)
    code = np.where(bad[..., None], 0, code).reshape(rows, -1)[:, : (cols + 1) // 2 * 2].astype(np.uint8)
    if cols % 2:
        code[:, -1] = 0
    return np.ascontiguousarray(code[:, 0::2] | (code[:, 1::2] << 4)), E
