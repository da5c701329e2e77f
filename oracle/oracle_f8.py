"""CPU oracles of the 8-bit block-scaled family in FP64 (test infrastructure only).

TEST INFRASTRUCTURE ONLY: the library never uses it.

Formats, written out from their definitions:
  e4m3: 1 sign, 4 exponent (bias 7), 3 fraction bits; no infinities, codes with
        all exponent and fraction bits set are NaN; largest 448; subnormals down
        to 2^-9.
  e5m2: 1 sign, 5 exponent (bias 15), 2 fraction bits, IEEE infinities and NaN;
        largest finite 57344; subnormals down to 2^-16.
Quantisation rounds to nearest, ties to even, in the FP32 operations of the
definition (one division each for the factor and the scale, one product per
value), which numpy performs correctly rounded: the result is one bit pattern.
"""
from __future__ import annotations

import numpy as np

BLOCK = 128
FLOOR = np.float32(2.0 ** -90)
LARGEST = {"e4m3": np.float32(448.0), "e5m2": np.float32(57344.0)}
_FRACTION = {"e4m3": 3, "e5m2": 2}
_BIAS = {"e4m3": 7, "e5m2": 15}


def _table(fmt: str) -> np.ndarray:
    f, bias = _FRACTION[fmt], _BIAS[fmt]
    out = np.empty(256)
    for code in range(256):
        e, m = (code & 0x7f) >> f, code & ((1 << f) - 1)
        top = (1 << (7 - f)) - 1
        if fmt == "e4m3" and e == top and m == 7:
            v = np.nan
        elif fmt == "e5m2" and e == top:
            v = np.inf if m == 0 else np.nan
        else:
            v = m * 2.0 ** (1 - bias - f) if e == 0 else (1 + m / (1 << f)) * 2.0 ** (e - bias)
        out[code] = -v if code & 0x80 else v
    return out


VALUES = {fmt: _table(fmt) for fmt in LARGEST}


def decode(codes: np.ndarray, fmt: str) -> np.ndarray:
    return VALUES[fmt][codes]


def encode(x: np.ndarray, fmt: str) -> np.ndarray:
    """float32 values within the format's range (or NaN) -> codes, nearest, ties to even."""
    pos = VALUES[fmt][:0x7f if fmt == "e4m3" else 0x7c]    # finite, ascending: code = index
    a = np.abs(x.astype(np.float64))
    hi = np.searchsorted(pos, a, side="left").clip(0, len(pos) - 1)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - pos[lo], pos[hi] - a
    code = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    code = np.where(a > pos[-1], len(pos) - 1, code).astype(np.uint8)
    code = code | (np.signbit(x).astype(np.uint8) << 7)
    return np.where(np.isnan(x), np.uint8(0x7f), code)


def blocks(n: int) -> int:
    return -(-n // BLOCK)


def _block_max(x: np.ndarray, block: str) -> np.ndarray:
    """Largest |x| of each block (NaN where it holds one), (rows or tile rows, k-blocks)."""
    r, k = x.shape
    rr = r if block == "row" else blocks(r) * BLOCK
    p = np.zeros((rr, blocks(k) * BLOCK), np.float32)
    p[:r, :k] = np.abs(x)
    if block == "row":
        return p.reshape(r, -1, BLOCK).max(axis=2)
    return p.reshape(rr // BLOCK, BLOCK, -1, BLOCK).max(axis=(1, 3))


def spread(per_block: np.ndarray, block: str, rows: int, cols: int) -> np.ndarray:
    """(rows or tile rows, k-blocks) -> one value per element."""
    if block == "tile":
        per_block = np.repeat(per_block, BLOCK, axis=0)[:rows]
    return np.repeat(per_block, BLOCK, axis=1)[:, :cols]


def quantize(x: np.ndarray, block: str, fmt: str):
    """float32 (rows, cols) -> (codes, scales as the library lays them out)."""
    x = np.asarray(x, np.float32)
    with np.errstate(all="ignore"):
        a = np.maximum(_block_max(x, block), FLOOR)          # numpy's maximum keeps a NaN
        inv, s = LARGEST[fmt] / a, a / LARGEST[fmt]
        q = encode(x * spread(inv, block, *x.shape), fmt)
    return q, np.ascontiguousarray(s.T) if block == "row" else s


def values(codes: np.ndarray, scales: np.ndarray, block: str, fmt: str) -> np.ndarray:
    """What codes and scales stand for, in FP64."""
    s = scales.T if block == "row" else scales
    with np.errstate(all="ignore"):
        return decode(codes, fmt) * spread(s.astype(np.float64), block, *codes.shape)


def gemm_f8(a, b, alpha=1.0, beta=0.0, c=None):
    """(D, S) of D = alpha a b^T + beta c on FP64 values; S = sum |a||b|."""
    with np.errstate(all="ignore"):
        d = alpha * (a @ b.T)
        if beta != 0.0:
            d = d + beta * c.astype(np.float64)
        return d, np.abs(a) @ np.abs(b).T


def rmsnorm(x, r, w, eps):
    """(h, rstd, y) in FP64."""
    h = x.astype(np.float64) + (0.0 if r is None else r.astype(np.float64))
    with np.errstate(all="ignore"):
        rstd = 1.0 / np.sqrt((h * h).mean(axis=1) + eps)
        return h, rstd, h * rstd[:, None] * w.astype(np.float64)


def rmsnorm_backward(dy, h, w, rstd, dh=None):
    """(dx, dw) in FP64 by the formula."""
    dy, h, w, rstd = (np.asarray(v, np.float64) for v in (dy, h, w, rstd))
    n, g = h * rstd[:, None], dy * w
    dx = rstd[:, None] * (g - n * (g * n).mean(axis=1, keepdims=True))
    if dh is not None:
        dx = dx + np.asarray(dh, np.float64)
    return dx, (dy * n).sum(axis=0)
