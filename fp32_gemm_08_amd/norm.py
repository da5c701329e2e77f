"""ctypes binding of the norms around a block (argument marshalling only).

The ``sgemm_block_norm*`` functions keep the C names and arguments of
``include/sgemm_norm.h``; ``block_norm`` and ``block_norm_backward`` are the same
calls over torch tensors, in the manner of ``f8``: outputs are the caller's
tensors, written in place, leading dimensions are row strides, the stream is
torch's current one, there is no fallback and no part in torch's gradient
tracking.
"""
from __future__ import annotations

import ctypes

from . import f8
from .f8 import _blocks, _device, _matrix, _run, _scale, _vector, _workspace
from .i8 import _i8_table
from .sgemm import load

Q_E4M3, Q_I8 = 1, 3

# Symbols declared in include/sgemm_norm.h.
NORM_EXPORTS = ("sgemm_block_norm", "sgemm_block_norm_bwd", "sgemm_block_norm_bwd_plan")

_norm = None


def _load_norm():
    global _norm
    if _norm is None:
        lib = load()
        i64, f32, vp, ci = ctypes.c_int64, ctypes.c_float, ctypes.c_void_p, ctypes.c_int
        mat = [vp, i64]
        for name, args in (
                ("sgemm_block_norm", [ci, ci, i64, i64] + 2 * mat + [vp, vp] + mat + [i64, f32, f32] + 2 * mat + [ci] +
                 6 * mat + [vp, vp, vp]),
                ("sgemm_block_norm_bwd", [ci, ci, i64, i64] + 2 * mat + [ci] + 4 * mat + [vp, vp, vp, vp] + mat +
                 [i64, f32] + 2 * mat + [vp, vp] + mat + [vp, i64, vp]),
                ("sgemm_block_norm_bwd_plan", [i64, i64, i64, ctypes.POINTER(i64)])):
            fn = getattr(lib, name)
            fn.restype, fn.argtypes = ci, args
        _norm = lib
    return _norm


def sgemm_block_norm(type, w_type, rows, cols, X, ldx, O, ldo, W, W_post, GATE, ldg, gate_rows, alpha, eps, H, ldh, Y,
                     ldy, q_format, Q, ldq, S, lds, H8, ldh8, SH, ldsh, O8, ldo8, SO, ldso, rstd, rstd_post,
                     stream=0) -> int:
    """Norm, gate and residual after a block, and the norm before the next.  Returns the status code."""
    return _load_norm().sgemm_block_norm(type, w_type, rows, cols, X, ldx, O, ldo, W, W_post, GATE, ldg, gate_rows,
                                         alpha, eps, H, ldh, Y, ldy, q_format, Q, ldq, S, lds, H8, ldh8, SH, ldsh, O8,
                                         ldo8, SO, ldso, rstd, rstd_post, stream)


def sgemm_block_norm_bwd(type, w_type, rows, cols, DY, lddy, DH, lddh, kept, H, ldh, SH, ldsh, O, ldo, SO, ldso, W,
                         W_post, rstd, rstd_post, GATE, ldg, gate_rows, alpha, DX, lddx, DO, lddo, DW, DW_post, DGATE,
                         lddg, workspace, workspace_bytes, stream=0) -> int:
    """Their backward pass.  Returns the status code."""
    return _load_norm().sgemm_block_norm_bwd(type, w_type, rows, cols, DY, lddy, DH, lddh, kept, H, ldh, SH, ldsh, O,
                                             ldo, SO, ldso, W, W_post, rstd, rstd_post, GATE, ldg, gate_rows, alpha, DX,
                                             lddx, DO, lddo, DW, DW_post, DGATE, lddg, workspace, workspace_bytes,
                                             stream)


def sgemm_block_norm_bwd_plan(rows, cols, gate_rows=0):
    """Host-only query: (status, workspace_bytes)."""
    nb = ctypes.c_int64(0)
    st = _load_norm().sgemm_block_norm_bwd_plan(rows, cols, gate_rows, ctypes.byref(nb))
    return st, nb.value


# ---------------------------------------------------------------- over torch tensors

def _rows_like(name, m, kind, rows, cols, dev, of):
    """(address, leading dimension) of a rows x cols matrix of that type; NULL for None."""
    if m is None:
        return 0, 0
    k, r, c, p, ld = _matrix(name, m, f8._TYPE_OF, dev)
    if k != kind or r != rows or c != cols:
        raise ValueError(f"{name} must be of {of}'s type and shape")
    return p, ld


def _kept8(name, m, s_name, s, rows, cols, dev):
    """The same of an e4m3 matrix with row blocks, and of its scales."""
    if m is None:
        return 0, 0, 0, 0
    k, r, c, p, ld = _matrix(name, m, f8._FORMAT_OF, dev)
    if k != 1 or r != rows or c != cols:
        raise ValueError(f"{name} must be float8_e4m3fn of shape {(rows, cols)}")
    if s is None:
        raise ValueError(f"{name} needs {s_name}")
    ps, lds = _scale(s_name, s, (_blocks(cols), rows), dev)
    return p, ld, ps, lds


def _weights(named, cols, dev, of, kind):
    """(their common type, addresses) of vectors of weights, NULL for None."""
    wt, out = kind, []
    first = True
    for name, w in named:
        if w is None:
            out.append(0)
            continue
        k, p = _vector(name, w, cols, dev, f8._TYPE_OF)
        if (k != kind and k != 0) or (not first and k != wt):
            raise TypeError(f"{name} must be of {of}'s type or float32, as the other weights")
        wt, first = k, False
        out.append(p)
    return wt, first, out


def _gate(name, gate, gate_rows, rows, cols, dev, of, kind, wt, free):
    """(type of the weights, address, leading dimension, rows of x for a row of the gate)."""
    if gate is None:
        return wt, 0, 0, 0
    k, g, c, p, ld = _matrix(name, gate if gate.dim() != 1 else gate[None], f8._TYPE_OF, dev)
    if (k != kind and k != 0) or (not free and k != wt):
        raise TypeError(f"{name} must be of {of}'s type or float32, as the other weights")
    if gate_rows is None:
        if g == 0 or rows % g:
            raise ValueError(f"{rows} rows do not divide among {g} rows of {name}: gate_rows is needed")
        gate_rows = max(rows // g, 1)
    if gate_rows < 1 or c != cols or g != (rows + gate_rows - 1) // gate_rows and rows > 0:
        raise ValueError(f"{name} has shape {(g, c)}, not {((rows + gate_rows - 1) // max(gate_rows, 1), cols)}")
    return k, p, ld, gate_rows


def block_norm(X, O, W, eps=1e-6, w_post=None, gate=None, gate_rows=None, alpha=1.0, H=None, Y=None, Q=None, S=None,
               H8=None, SH=None, O8=None, SO=None, rstd=None, rstd_post=None, stream=None):
    """Between two blocks: z = norm(O) * w_post, h = alpha * X + gate * z, y = norm(h) * W.

    X (the residual stream), O (the block's output; None: no block), H and Y are
    (rows, cols) of one type (float32, float16 or bfloat16); W and w_post (cols) and
    gate (cols, or a row of cols for every ``gate_rows`` rows of X; by default the rows
    divide evenly) are of that type or float32.  w_post None: z = O; gate None: 1.
    norm(v) = v / sqrt(mean(v^2) + eps), row by row.  Written where given: H <- h (may
    be X or O itself), Y <- y, Q with S <- y in 8 bits (float8_e4m3fn with S
    (ceil(cols/128), rows), or int8 with S (rows)), H8 with SH and O8 with SO <- h and O
    as float8_e4m3fn with scales (ceil(cols/128), rows), rstd and rstd_post (rows,
    float32): what ``block_norm_backward`` takes.  W may be None if neither Y nor Q
    is given.
    """
    dev = _device(X)
    t, rows, cols, px, ldx = _matrix("X", X, f8._TYPE_OF, dev)
    po, ldo = _rows_like("O", O, t, rows, cols, dev, "X")
    wt, free, (pw, pwp) = _weights((("W", W), ("w_post", w_post)), cols, dev, "X", t)
    wt, pg, ldg, gate_rows = _gate("gate", gate, gate_rows, rows, cols, dev, "X", t, wt, free)
    if O is None and (w_post is not None or gate is not None or O8 is not None or rstd_post is not None):
        raise ValueError("w_post, gate, O8 and rstd_post belong to O")
    if rstd_post is not None and w_post is None:
        raise ValueError("rstd_post belongs to w_post")
    if W is None and (Y is not None or Q is not None):
        raise ValueError("Y and Q need W")
    ph, ldh = _rows_like("H", H, t, rows, cols, dev, "X")
    py, ldy = _rows_like("Y", Y, t, rows, cols, dev, "X")
    pq = ldq = ps = lds = 0
    qf = Q_E4M3
    if Q is not None:
        if S is None:
            raise ValueError("Q needs S")
        if Q.dtype in _i8_table():
            qf = Q_I8
            _, r, c, pq, ldq = _matrix("Q", Q, _i8_table(), dev)
            if r != rows or c != cols:
                raise ValueError("Q must be of X's shape")
            ps = _vector("S", S, rows, dev, f8._F32)[1]
        else:
            pq, ldq, ps, lds = _kept8("Q", Q, "S", S, rows, cols, dev)
    ph8, ldh8, psh, ldsh = _kept8("H8", H8, "SH", SH, rows, cols, dev)
    po8, ldo8, pso, ldso = _kept8("O8", O8, "SO", SO, rows, cols, dev)
    prs = _vector("rstd", rstd, rows, dev, f8._F32)[1] if rstd is not None else 0
    prp = _vector("rstd_post", rstd_post, rows, dev, f8._F32)[1] if rstd_post is not None else 0
    _run(dev, stream, (_norm or _load_norm()).sgemm_block_norm,
         (t, wt, rows, cols, px, ldx, po, ldo, pw, pwp, pg, ldg, gate_rows, alpha, eps, ph, ldh, py, ldy, qf, pq, ldq,
          ps, lds, ph8, ldh8, psh, ldsh, po8, ldo8, pso, ldso, prs, prp))


def block_norm_backward(dY, H, O, W, rstd, dX, dO, SH=None, SO=None, w_post=None, rstd_post=None, gate=None,
                        gate_rows=None, alpha=1.0, dH=None, dW=None, dW_post=None, dGate=None, workspace=None,
                        stream=None):
    """Gradients of ``block_norm``: dX of X, dO of the block's output, and those of W,
    w_post and the gate.

    dY is the gradient of y (None: nothing reaches it, and H, W and rstd are not
    needed), dH what reaches h along the residual path (or None).  H and O are what
    the forward pass kept: both of dY's type, or both float8_e4m3fn with their scales
    SH and SO; O is needed for dGate, or with w_post, and may be None elsewhere.  dX and dO (either may be None) may be dY
    or dH, and H and O themselves where those are of dY's type.  dW and dW_post (cols)
    and dGate (gate's shape) are float32, or None, and need a ``workspace`` of
    sgemm_block_norm_bwd_plan's bytes.
    """
    first = dY if dY is not None else dH
    if first is None:
        raise ValueError("one of dY and dH is needed")
    dev = _device(first)
    t, rows, cols, _, _ = _matrix("dY" if dY is not None else "dH", first, f8._TYPE_OF, dev)
    pdy, lddy = _rows_like("dY", dY, t, rows, cols, dev, "dY")
    pdh, lddh = _rows_like("dH", dH, t, rows, cols, dev, "dY")
    if O is None and (dGate is not None or w_post is not None):
        raise ValueError("w_post and dGate need O")
    if dY is not None and (H is None or W is None or rstd is None):
        raise ValueError("dY needs H, W and rstd")
    if dGate is not None and gate is None:
        raise ValueError("dGate needs gate")
    if w_post is None and dW_post is not None:
        raise ValueError("dW_post needs w_post")
    if w_post is not None and rstd_post is None:
        raise ValueError("w_post needs rstd_post")
    kept = {m.dtype in f8._FORMAT_OF for m in (H if dY is not None else None, O) if m is not None}
    if len(kept) > 1:
        raise TypeError("H and O must both be of dY's type or both float8_e4m3fn")
    kept = kept == {True}
    psh = ldsh = pso = ldso = 0
    if kept:
        ph, ldh, psh, ldsh = _kept8("H", H if dY is not None else None, "SH", SH, rows, cols, dev)
        po, ldo, pso, ldso = _kept8("O", O, "SO", SO, rows, cols, dev)
    else:
        ph, ldh = _rows_like("H", H if dY is not None else None, t, rows, cols, dev, "dY")
        po, ldo = _rows_like("O", O, t, rows, cols, dev, "dY")
    wt, free, (pw, pwp) = _weights((("W", W if dY is not None else None), ("w_post", w_post)), cols, dev, "dY", t)
    wt, pg, ldg, gate_rows = _gate("gate", gate, gate_rows, rows, cols, dev, "dY", t, wt, free)
    pdx, lddx = _rows_like("dX", dX, t, rows, cols, dev, "dY")
    pdo, lddo = _rows_like("dO", dO, t, rows, cols, dev, "dY")
    prs = _vector("rstd", rstd, rows, dev, f8._F32)[1] if dY is not None else 0
    prp = _vector("rstd_post", rstd_post, rows, dev, f8._F32)[1] if w_post is not None else 0
    pdw = _vector("dW", dW, cols, dev, f8._F32)[1] if dW is not None else 0
    pdwp = _vector("dW_post", dW_post, cols, dev, f8._F32)[1] if dW_post is not None else 0
    pdg = lddg = 0
    if dGate is not None:
        if dGate.shape != gate.shape:
            raise ValueError("dGate must have the gate's shape")
        _, _, _, pdg, lddg = _matrix("dGate", dGate if dGate.dim() != 1 else dGate[None], f8._F32, dev)
    pws, nws = _workspace(workspace, dev)
    _run(dev, stream, (_norm or _load_norm()).sgemm_block_norm_bwd,
         (t, wt, rows, cols, pdy, lddy, pdh, lddh, 1 if kept else 0, ph, ldh, psh, ldsh, po, ldo, pso, ldso, pw, pwp,
          prs, prp, pg, ldg, gate_rows, alpha, pdx, lddx, pdo, lddo, pdw, pdwp, pdg, lddg, pws, nws))
