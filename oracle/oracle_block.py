"""CPU oracles in FP64 of the norms around a block, of the quantisation of rows to 8-bit
integers and of their products (test infrastructure only: the library never uses it)."""
from __future__ import annotations

import numpy as np

from .oracle_f8 import FLOOR


def gate_of_rows(gate, gate_rows, rows):
    """The gate's row for each row, or 1."""
    return 1.0 if gate is None else np.asarray(gate, np.float64)[np.arange(rows) // gate_rows]


def block_norm(x, o, w, eps, w_post=None, gate=None, gate_rows=1, alpha=1.0):
    """(h, y, rstd, rstd_post, z) in FP64; z and rstd_post None where there are none."""
    x = np.asarray(x, np.float64)
    h, z, rp = alpha * x, None, None
    with np.errstate(all="ignore"):
        if o is not None:
            z = np.asarray(o, np.float64)
            if w_post is not None:
                rp = 1.0 / np.sqrt((z * z).mean(axis=1) + eps)
                z = z * rp[:, None] * np.asarray(w_post, np.float64)
            h = h + gate_of_rows(gate, gate_rows, len(x)) * z
        rstd = 1.0 / np.sqrt((h * h).mean(axis=1) + eps)
        y = None if w is None else h * rstd[:, None] * np.asarray(w, np.float64)
    return h, y, rstd, rp, z


def block_norm_backward(dy, dh, h, o, w, rstd, w_post=None, rstd_post=None, gate=None, gate_rows=1, alpha=1.0):
    """dx, do, dw, dw_post, dgate by the formulas (None where there is none), and the sizes
    that rounding is measured by: |d|'s terms, do's terms, and sums of |products|."""
    f = lambda v: None if v is None else np.asarray(v, np.float64)  # noqa: E731
    dy, dh, h, o, w, rstd, w_post, rstd_post = map(f, (dy, dh, h, o, w, rstd, w_post, rstd_post))
    rows, cols = (dy if dy is not None else dh).shape
    d, d_size, dw, dw_size = 0.0, 0.0, None, None
    if dy is not None:
        n, g = h * rstd[:, None], dy * w
        d = rstd[:, None] * (g - n * (g * n).mean(axis=1, keepdims=True))
        d_size = rstd[:, None] * (np.abs(g) + np.abs(n) * np.abs(g * n).mean(axis=1, keepdims=True))
        dw, dw_size = (dy * n).sum(axis=0), np.abs(dy * n).sum(axis=0)
    if dh is not None:
        d, d_size = d + dh, d_size + np.abs(dh)
    gr = gate_of_rows(gate, gate_rows, rows)
    back, back_size = gr * d, np.abs(gr) * d_size
    out = dict(dx=alpha * d, dx_size=abs(alpha) * d_size, dw=dw, dw_size=dw_size, do=back, do_size=back_size, dw_post=None,
               dgate=None)
    z = o
    if w_post is not None:
        m = o * rstd_post[:, None]
        z, p, p_size = m * w_post, back * w_post, back_size * np.abs(w_post)
        out["do"] = rstd_post[:, None] * (p - m * (p * m).mean(axis=1, keepdims=True))
        out["do_size"] = rstd_post[:, None] * (p_size + np.abs(m) * (p_size * np.abs(m)).mean(axis=1, keepdims=True))
        out["dw_post"], out["dw_post_size"] = (back * m).sum(axis=0), (back_size * np.abs(m)).sum(axis=0)
    if gate is not None and o is not None:
        gates = -(-rows // gate_rows)
        out["dgate"], out["dgate_size"] = np.zeros((gates, cols)), np.zeros((gates, cols))
        np.add.at(out["dgate"], np.arange(rows) // gate_rows, d * z)
        np.add.at(out["dgate_size"], np.arange(rows) // gate_rows, d_size * np.abs(z))
    return out


def quantize_rows_i8(x):
    """float32 (rows, cols) -> (int8, float32 scales): 127 x / a to the nearest, ties to even.
    The quotient of a 31-bit and a 24-bit number is rounded once to 53 bits, which never moves
    it to or across the middle between two integers below 2^7."""
    x = np.asarray(x, np.float32)
    with np.errstate(all="ignore"):
        a = np.maximum(np.abs(x).max(axis=1), FLOOR)
        q = np.rint(127.0 * x.astype(np.float64) / a.astype(np.float64)[:, None])
        q = np.where(np.isfinite(a)[:, None], q, 0.0)
        return q.astype(np.int8), a / np.float32(127.0)


def gemm_i8(a, sa, b, sb, alpha=1.0, beta=0.0, c=None):
    """(D in FP64, the integer sums)."""
    s = a.astype(np.float64) @ b.astype(np.float64).T        # exact: below 2^53
    with np.errstate(all="ignore"):
        d = alpha * (s * sa.astype(np.float64)[:, None] * sb.astype(np.float64))
        if beta != 0.0:
            d = d + beta * np.asarray(c, np.float64)
    return d, s
