"""Block-scaled 8-bit float matrices, routing and experts' rows in plain numpy, 64 bits: what the library's
results are compared with. Shares no code with the library."""
from __future__ import annotations

import numpy as np

E4M3, E5M2 = "e4m3", "e5m2"
TOP = {E4M3: 448.0, E5M2: 57344.0}
_BITS = {E4M3: (4, 3, 7), E5M2: (5, 2, 15)}  # exponent bits, mantissa bits, bias
BLOCK = 128


def decode_table(kind):
    """The value of each of the 256 codes (NaN and infinities included)."""
    eb, mb, bias = _BITS[kind]
    c = np.arange(256)
    e, m = c >> mb & (1 << eb) - 1, c & (1 << mb) - 1
    v = np.where(e == 0, m * 2.0 ** (1 - bias - mb), (1 + m * 2.0**-mb) * 2.0 ** (e - bias))
    if kind == E4M3:
        v = np.where(c & 127 == 127, np.nan, v)
    else:
        v = np.where(e == 31, np.where(m == 0, np.inf, np.nan), v)
    return np.where(c >= 128, -v, v)


def finite_codes(kind):
    v = decode_table(kind)
    return np.arange(256, dtype=np.uint8)[np.isfinite(v)]


def nearest_code(y, kind):
    """The code nearest to each y (finite, within the type's range after saturation), ties to the even code."""
    v = decode_table(kind)[:128]
    v = v[np.isfinite(v)]
    a = np.minimum(np.abs(y), v[-1])
    hi = np.searchsorted(v, a)  # v[hi - 1] < a <= v[hi]
    lo = np.maximum(hi - 1, 0)
    dlo, dhi = a - v[lo], v[hi] - a
    code = np.where((dlo < dhi) | ((dlo == dhi) & (lo % 2 == 0)), lo, hi)
    return (code + np.where(np.signbit(y), 128, 0)).astype(np.uint8)


def blocks(n):
    return -(-n // BLOCK)


def encode(x, kind, block_rows=1):
    """(codes, scales) of x (64 bits): scales are fp32."""
    rows, cols = x.shape
    nr, nc = -(-rows // block_rows), blocks(cols)
    g = np.zeros((nr * block_rows, nc * BLOCK))
    g[:rows, :cols] = x
    g = g.reshape(nr, block_rows, nc, BLOCK)
    a = np.abs(g).max(axis=(1, 3))  # NaN wins
    bad = ~np.isfinite(a)
    inv = np.float32(1.0) / np.float32(TOP[kind])
    s = np.maximum((np.where(bad, 1.0, a).astype(np.float32) * inv).astype(np.float32), np.float32(2.0**-126))
    y = np.where(bad[:, None, :, None], 0.0, g) / s.astype(np.float64)[:, None, :, None]
    codes = nearest_code(y, kind).reshape(nr * block_rows, nc * BLOCK)[:rows, :cols]
    return codes, np.where(bad, np.float32(np.nan), s)


def decode(codes, scales, kind, block_rows=1):
    rows, cols = codes.shape
    s = scales.astype(np.float64)[np.arange(rows) // block_rows][:, np.arange(cols) // BLOCK]
    return decode_table(kind)[codes] * s


# ---- routing -----------------------------------------------------------------------------------
def route(logits, k, bias=None, sigmoid=False, groups=1, top_groups=1, group_best=1, renormalize=True, scale=1.0):
    """(experts, weights) token by token."""
    T, E = logits.shape
    x = logits.astype(np.float64)
    chosen, weights = np.full((T, k), -1, np.int32), np.zeros((T, k))
    for t in range(T):
        l = x[t]
        if np.isnan(l).any() or (l == np.inf).any():
            chosen[t], weights[t] = np.arange(k), np.nan
            continue
        s = scores(l, sigmoid)
        # without a bias the scores' order is the logits' (both functions increase; exp underflows, order does not)
        by_logit = bias is None and (groups == 1 or group_best == 1)
        v = l if by_logit else np.where(l == -np.inf, -np.inf, s if bias is None else s + bias.astype(np.float64))
        v = np.where(np.isnan(v), -np.inf, v)
        if groups > 1:
            g = v.reshape(groups, -1)
            best = np.sort(g, axis=1)[:, ::-1]
            rank = best[:, 0].copy()
            if group_best == 2 and best.shape[1] > 1:
                rank += np.where(best[:, 1] == -np.inf, 0.0, best[:, 1])
            kept = np.argsort(-rank, kind="stable")[:top_groups]
            open_ = np.zeros(groups, bool)
            open_[kept] = True
            v = np.where(open_[:, None], g, -np.inf).reshape(-1)
        order = np.argsort(-v, kind="stable")[:k]
        order = order[v[order] > -np.inf]
        chosen[t, :len(order)] = order
        w = s[order]
        if renormalize:
            total = w.sum()
            w = w / total if total > 0 else w * 0
        weights[t, :len(order)] = w * scale
    return chosen, weights


def scores(l, sigmoid):
    if sigmoid:
        with np.errstate(over="ignore"):
            return 1 / (1 + np.exp(-l))
    top = l.max()
    if top == -np.inf:
        return np.zeros_like(l)
    e = np.exp(l - top)
    return e / e.sum()


def route_loss(logits, chosen, dweights, sigmoid, renormalize, scale):
    """sum of weights * dweights for a fixed choice: its differences are the gradient."""
    total = 0.0
    for l, c, d in zip(logits.astype(np.float64), chosen, dweights.astype(np.float64)):
        s = scores(l, sigmoid)
        there = c >= 0
        w = s[c[there]]
        if renormalize:
            w = w / w.sum() if w.sum() > 0 else w * 0
        total += scale * (w * d[there]).sum()
    return total


def route_grad(logits, chosen, dweights, sigmoid, renormalize, scale):
    """The formula, through the full Jacobian."""
    out = np.zeros(logits.shape)
    for t, (l, c, d) in enumerate(zip(logits.astype(np.float64), chosen, dweights.astype(np.float64))):
        if np.isnan(l).any() or (l == np.inf).any():
            out[t] = np.nan
            continue
        s = scores(l, sigmoid)
        there = c >= 0
        ds = np.zeros_like(s)
        total = s[c[there]].sum()
        for e, g in zip(c[there], d[there] * scale):
            if not renormalize:
                ds[e] += g
            elif total > 0:
                ds[e] += g / total
                np.add.at(ds, c[there], -g * s[e] / total**2)
        out[t] = ds * s * (1 - s) if sigmoid else s * (ds - (ds * s).sum())
    return out


# ---- rows by expert ----------------------------------------------------------------------------
def rows_size(slots, experts, align):
    n = slots + min(slots, experts) * (align - 1)
    return -(-n // align) * align


def expert_rows(chosen, experts, align):
    """(slots, position, offsets, counts)"""
    flat = chosen.reshape(-1)
    slots, position = np.full(rows_size(flat.size, experts, align), -1, np.int32), np.full(flat.size, -1, np.int32)
    offsets, counts, at = np.zeros(experts + 1, np.int32), np.zeros(experts, np.int32), 0
    for e in range(experts):
        mine = np.flatnonzero(flat == e)
        offsets[e], counts[e] = at, mine.size
        slots[at:at + mine.size] = mine
        position[mine] = at + np.arange(mine.size)
        at += -(-mine.size // align) * align
    offsets[experts] = at
    return slots, position.reshape(chosen.shape), offsets, counts
