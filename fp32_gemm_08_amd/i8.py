"""ctypes binding of the products of 8-bit integers (argument marshalling only).

The ``sgemm_i8_*`` functions keep the C names and arguments of
``include/sgemm_i8.h``; ``i8_gemm`` and ``i8_quantize`` are the same calls over
torch tensors, in the manner of ``f8``: outputs are the caller's tensors, written
in place, leading dimensions are row strides, the stream is torch's current one,
there is no fallback and no part in torch's gradient tracking.
"""
from __future__ import annotations

import ctypes

from .native import check, tensors
from .sgemm import load

I8_MAX_K = 131071

# Symbols declared in include/sgemm_i8.h.
I8_EXPORTS = ("sgemm_i8_gemm", "sgemm_i8_gemm_plan", "sgemm_i8_gemm_workspace", "sgemm_i8_quantize")

_i8 = None


def _load_i8():
    global _i8
    if _i8 is None:
        lib = load()
        i64, f32, vp, ci = ctypes.c_int64, ctypes.c_float, ctypes.c_void_p, ctypes.c_int
        pi, pl = ctypes.POINTER(ci), ctypes.POINTER(i64)
        for name, args in (
                ("sgemm_i8_gemm", [ci, i64, i64, i64, f32, vp, i64, vp, vp, i64, vp, f32, vp, i64, vp, i64, vp]),
                ("sgemm_i8_gemm_plan", [i64, i64, i64, ci, pi, pl, pl, pl, pl]),
                ("sgemm_i8_gemm_workspace", [i64, i64, i64, ci, pl]),
                ("sgemm_i8_quantize", [ci, i64, i64, vp, i64, vp, i64, vp, vp])):
            fn = getattr(lib, name)
            fn.restype, fn.argtypes = ci, args
        _i8 = lib
    return _i8


def sgemm_i8_gemm(c_type, M, N, K, alpha, A, lda, SA, B, ldb, SB, beta, C, ldc, workspace=0, workspace_bytes=0,
                  stream=0) -> int:
    """C <- alpha*diag(SA)*A*B^T*diag(SB) + beta*C on 8-bit integers.  Returns the status code."""
    return _load_i8().sgemm_i8_gemm(c_type, M, N, K, alpha, A, lda, SA, B, ldb, SB, beta, C, ldc, workspace,
                                    workspace_bytes, stream)


def sgemm_i8_gemm_plan(M, N, K, aligned=1):
    """Host-only query: (status, kernel_id, tiles_m, tiles_n, splits, workspace_bytes)."""
    kid = ctypes.c_int(0)
    tm, tn, sp, nb = (ctypes.c_int64(0) for _ in range(4))
    st = _load_i8().sgemm_i8_gemm_plan(M, N, K, aligned, ctypes.byref(kid), ctypes.byref(tm), ctypes.byref(tn),
                                       ctypes.byref(sp), ctypes.byref(nb))
    return st, kid.value, tm.value, tn.value, sp.value, nb.value


def sgemm_i8_gemm_workspace(M, N, K, aligned=1):
    """Host-only query: (status, workspace_bytes) with which the product is fastest."""
    nb = ctypes.c_int64(0)
    st = _load_i8().sgemm_i8_gemm_workspace(M, N, K, aligned, ctypes.byref(nb))
    return st, nb.value


def sgemm_i8_quantize(x_type, rows, cols, X, ldx, Q, ldq, S, stream=0) -> int:
    """Rows of X -> 8-bit integers and a scale each.  Returns the status code."""
    return _load_i8().sgemm_i8_quantize(x_type, rows, cols, X, ldx, Q, ldq, S, stream)


# ---------------------------------------------------------------- over torch tensors

def i8_gemm(A, SA, B, SB, C, alpha=1.0, beta=0.0, workspace=None, stream=None):
    """C <- alpha*diag(SA)*A*B^T*diag(SB) + beta*C, in place; returns C.

    A (M, K) and B (N, K) are int8, SA (M) and SB (N) their float32 scales (a
    token's and a channel's each), C (M, N) is float32, float16 or bfloat16; rows
    may be strided.  The sums over k are exact; K is at most 131071.
    ``workspace``: a contiguous device tensor lent for partial sums where there are
    few output tiles, and for operands whose rows do not start on 16-byte
    boundaries (sgemm_i8_gemm_workspace says how many bytes serve; the call takes
    the fastest way that fits, with the same result).
    """
    check(tensors().i8_gemm(A, SA, B, SB, C, alpha, beta, workspace, stream))
    return C


def i8_quantize(X, Q, S, stream=None):
    """X (rows, cols; float32, float16 or bfloat16) -> Q (rows, cols; int8) with one
    scale per row in S (rows, float32): Q is 127 * X / max|X| of the row to the
    nearest integer, ties to even, and Q * S is about X."""
    check(tensors().i8_quantize(X, Q, S, stream))
