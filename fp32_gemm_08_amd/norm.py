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

from .native import check, tensors
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

def block_norm(X, O, W, eps=1e-6, w_post=None, gate=None, gate_rows=None, alpha=1.0, H=None, Y=None, Q=None, S=None,
               H8=None, SH=None, O8=None, SO=None, rstd=None, rstd_post=None, stream=None):
    """Between two blocks: z = norm(O) * w_post, h = alpha * X + gate * z, y = norm(h) * W.

    X (the residual stream), O (the block's output; None: no block), H and Y are
    (rows, cols) of one type (float32, float16 or bfloat16); W and w_post (cols) and
    gate (cols, or a row of cols for every ``gate_rows`` rows of X; by default the rows
    divide evenly; where X has none, of any number) are all of that type or all float32.
    w_post None: z = O; gate None: 1.
    norm(v) = v / sqrt(mean(v^2) + eps), row by row.  Written where given: H <- h (may
    be X or O itself), Y <- y, Q with S <- y in 8 bits (float8_e4m3fn with S
    (ceil(cols/128), rows), or int8 with S (rows)), H8 with SH and O8 with SO <- h and O
    as float8_e4m3fn with scales (ceil(cols/128), rows), rstd and rstd_post (rows,
    float32): what ``block_norm_backward`` takes.  W may be None if neither Y nor Q
    is given.
    """
    check(tensors().block_norm(X, O, W, eps, w_post, gate, gate_rows, alpha, H, Y, Q, S, H8, SH, O8, SO, rstd, rstd_post,
                               stream))


def block_norm_backward(dY, H, O, W, rstd, dX, dO, SH=None, SO=None, w_post=None, rstd_post=None, gate=None,
                        gate_rows=None, alpha=1.0, dH=None, dW=None, dW_post=None, dGate=None, workspace=None,
                        stream=None):
    """Gradients of ``block_norm``: dX of X, dO of the block's output, and those of W,
    w_post and the gate.

    dY is the gradient of y (None: nothing reaches it, and H, W and rstd are not
    needed), dH what reaches h along the residual path (or None).  H and O are what
    the forward pass kept: both of dY's type, or both float8_e4m3fn with their scales
    SH and SO; O is needed for dGate, or with w_post, and may be None elsewhere.  dX and dO
    (either may be None) may be dY or dH, and H and O themselves where those are of dY's
    type.  dW and dW_post (cols) and dGate (gate's shape) are float32, or None, and need a
    ``workspace`` of sgemm_block_norm_bwd_plan's bytes; without rows they are set to 0.
    """
    check(tensors().block_norm_backward(dY, H, O, W, rstd, dX, dO, SH, SO, w_post, rstd_post, gate, gate_rows, alpha, dH, dW,
                                        dW_post, dGate, workspace, stream))
