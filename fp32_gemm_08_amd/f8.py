"""ctypes binding of the 8-bit block-scaled family (argument marshalling only).

The ``sgemm_f8_*`` functions keep the C names and arguments of
``include/sgemm_f8.h``; pointers are plain integers (device addresses, 0 for
NULL) and ``stream`` is a hipStream_t as an integer.  ``f8_gemm``,
``f8_quantize``, ``rmsnorm`` and ``rmsnorm_backward`` are the same calls over
torch tensors: outputs are the caller's tensors, written in place, leading
dimensions are row strides, and the stream is torch's current one.  torch is
used for device memory and streams only; there is no fallback.

The tensor functions are no part of torch's gradient tracking: inputs that require
gradients are taken as they are, outputs carry no history, and writing them does not
move their version counters, so torch does not notice when a tensor that it saved for
a backward pass is overwritten.  A program that trains calls the backward functions
itself (or wraps both directions in a torch.autograd.Function) and keeps what they read.
"""
from __future__ import annotations

import ctypes

from .sgemm import SGEMM_OK, SgemmError, load, sgemm_f32_status_string

F8_FORMAT = {"e4m3": 1, "e5m2": 2}
F8_BLOCK = {"row": 0, "tile": 1}
TYPE = {"f32": 0, "fp16": 1, "bf16": 2}
RMSNORM_MAX_COLS = 32768

# Symbols declared in include/sgemm_f8.h.
F8_EXPORTS = ("sgemm_f8_gemm", "sgemm_f8_gemm_plan", "sgemm_f8_gemm_workspace", "sgemm_f8_quantize",
              "sgemm_f8_rmsnorm", "sgemm_f8_rmsnorm_bwd", "sgemm_f8_rmsnorm_bwd_plan")

_f8 = None


def _load_f8():
    global _f8
    if _f8 is None:
        lib = load()
        i64, f32, vp, ci = ctypes.c_int64, ctypes.c_float, ctypes.c_void_p, ctypes.c_int
        pi, pl = ctypes.POINTER(ci), ctypes.POINTER(i64)
        for name, args in (
                ("sgemm_f8_gemm", [ci, ci, ci, ci, i64, i64, i64, f32, vp, i64, vp, i64, vp, i64, vp, i64, f32, vp,
                                   i64, vp, i64, vp]),
                ("sgemm_f8_gemm_plan", [ci, i64, i64, i64, ci, pi, pl, pl, pl, pl]),
                ("sgemm_f8_gemm_workspace", [ci, i64, i64, i64, ci, pl]),
                ("sgemm_f8_quantize", [ci, ci, ci, i64, i64, vp, i64, vp, i64, vp, i64, vp, i64, vp, i64, vp]),
                ("sgemm_f8_rmsnorm", [ci, ci, i64, i64, vp, i64, vp, i64, vp, f32, vp, i64, vp, i64, vp, i64, vp, i64,
                                      vp, vp]),
                ("sgemm_f8_rmsnorm_bwd", [ci, ci, i64, i64, vp, i64, vp, i64, vp, vp, vp, i64, vp, i64, vp, vp, i64,
                                          vp]),
                ("sgemm_f8_rmsnorm_bwd_plan", [i64, i64, pl])):
            fn = getattr(lib, name)
            fn.restype, fn.argtypes = ci, args
        _f8 = lib
    return _f8


def sgemm_f8_gemm(format_a, format_b, b_block, c_type, M, N, K, alpha, A, lda, SA, ldsa, B, ldb, SB, ldsb, beta, C,
                  ldc, workspace=0, workspace_bytes=0, stream=0) -> int:
    """C <- alpha*A*B^T + beta*C on 8-bit operands with block scales.  Returns the status code."""
    return _load_f8().sgemm_f8_gemm(format_a, format_b, b_block, c_type, M, N, K, alpha, A, lda, SA, ldsa, B, ldb, SB,
                                    ldsb, beta, C, ldc, workspace, workspace_bytes, stream)


def sgemm_f8_gemm_plan(b_block, M, N, K, aligned=1):
    """Host-only query: (status, kernel_id, tiles_m, tiles_n, splits, workspace_bytes)."""
    kid = ctypes.c_int(0)
    tm, tn, sp, nb = (ctypes.c_int64(0) for _ in range(4))
    st = _load_f8().sgemm_f8_gemm_plan(b_block, M, N, K, aligned, ctypes.byref(kid), ctypes.byref(tm),
                                       ctypes.byref(tn), ctypes.byref(sp), ctypes.byref(nb))
    return st, kid.value, tm.value, tn.value, sp.value, nb.value


def sgemm_f8_gemm_workspace(b_block, M, N, K, aligned=1):
    """Host-only query: (status, workspace_bytes) with which the product is fastest."""
    nb = ctypes.c_int64(0)
    st = _load_f8().sgemm_f8_gemm_workspace(b_block, M, N, K, aligned, ctypes.byref(nb))
    return st, nb.value


def sgemm_f8_quantize(block, format, x_type, rows, cols, X, ldx, Q, ldq, S, lds, QT=0, ldqt=0, ST=0, ldst=0,
                      stream=0) -> int:
    """X -> its 8-bit values and scales, and (QT) those of X^T.  Returns the status code."""
    return _load_f8().sgemm_f8_quantize(block, format, x_type, rows, cols, X, ldx, Q, ldq, S, lds, QT, ldqt, ST, ldst,
                                        stream)


def sgemm_f8_rmsnorm(type, w_type, rows, cols, X, ldx, R, ldr, W, eps, H, ldh, Y, ldy, Q, ldq, S, lds, rstd,
                     stream=0) -> int:
    """Norm of x + r with outputs in x's type and in 8 bits.  Returns the status code."""
    return _load_f8().sgemm_f8_rmsnorm(type, w_type, rows, cols, X, ldx, R, ldr, W, eps, H, ldh, Y, ldy, Q, ldq, S,
                                       lds, rstd, stream)


def sgemm_f8_rmsnorm_bwd(type, w_type, rows, cols, DY, lddy, H, ldh, W, rstd, DH, lddh, DX, lddx, DW, workspace,
                         workspace_bytes, stream=0) -> int:
    """Backward pass of the norm.  Returns the status code."""
    return _load_f8().sgemm_f8_rmsnorm_bwd(type, w_type, rows, cols, DY, lddy, H, ldh, W, rstd, DH, lddh, DX, lddx,
                                           DW, workspace, workspace_bytes, stream)


def sgemm_f8_rmsnorm_bwd_plan(rows, cols):
    """Host-only query: (status, workspace_bytes)."""
    nb = ctypes.c_int64(0)
    st = _load_f8().sgemm_f8_rmsnorm_bwd_plan(rows, cols, ctypes.byref(nb))
    return st, nb.value


# ---------------------------------------------------------------- over torch tensors

_FORMAT_OF = None  # torch dtype -> sgemm_f8_format; -> sgemm_type; FP32 alone
_TYPE_OF = None
_F32 = None
_raw_stream = _current_device = None


def _tables():
    global _FORMAT_OF, _TYPE_OF, _F32, _raw_stream, _current_device
    import torch

    _raw_stream, _current_device = torch._C._cuda_getCurrentRawStream, torch.cuda.current_device
    _TYPE_OF = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}
    _F32 = {torch.float32: 0}
    # last: another thread's first call takes it as the sign that all are there
    _FORMAT_OF = {torch.float8_e4m3fn: 1, torch.float8_e5m2: 2}


def _matrix(name, t, table, device):
    """(id of the element type, rows, cols, address, leading dimension) of a
    2-D device tensor with unit stride along its rows."""
    kind = table.get(t.dtype)
    if kind is None or t.dim() != 2 or t.device != device:
        raise TypeError(f"{name}: a 2-D {' / '.join(str(k)[6:] for k in table)} tensor on the call's device is needed")
    rows, cols = t.shape
    ld, step = t.stride()
    if step != 1 and cols > 1:
        raise ValueError(f"{name} must have unit stride along its last dimension")
    if ld < cols or ld == 0:
        if rows > 1 and cols > 0:
            raise ValueError(f"{name} rows overlap (row stride below the row length)")
        ld = cols or 1
    elif rows <= 1:
        ld = cols or 1
    return kind, rows, cols, t.data_ptr(), ld


def _scale(name, t, shape, device):
    """(address, leading dimension) of an FP32 array of scales of that shape."""
    _, rows, cols, p, ld = _matrix(name, t, _F32, device)
    if rows != shape[0] or cols != shape[1]:
        raise ValueError(f"{name} has shape {(rows, cols)}, not {shape}")
    return p, ld


def _vector(name, t, n, device, types):
    kind = types.get(t.dtype)
    if kind is None or t.dim() != 1 or t.device != device:
        raise TypeError(f"{name}: a 1-D {' / '.join(str(k)[6:] for k in types)} tensor on the call's device is needed")
    if t.shape[0] != n or (n > 1 and t.stride(0) != 1):
        raise ValueError(f"{name} must hold {n} consecutive values")
    return kind, t.data_ptr()


def _workspace(t, device):
    if t is None:
        return 0, 0
    if t.device != device or not t.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on the call's device")
    return t.data_ptr(), t.numel() * t.element_size()


def _blocks(n):
    return (n + 127) // 128


def _scale_shape(block, rows, cols):
    return (_blocks(cols), rows) if block == 0 else (_blocks(rows), _blocks(cols))


def _device(t):
    """The device of a call: that of its first tensor, which must be a GPU."""
    if _FORMAT_OF is None:
        _tables()
    dev = t.device
    if dev.type != "cuda":
        raise TypeError("tensors on a GPU are needed")
    return dev


def _run(device, stream, fn, args):
    # the raw handle of torch's current stream: the Stream object around it
    # costs 2 us, as much as the launch itself
    raw = _raw_stream(device.index) if stream is None else stream.cuda_stream
    if _current_device() == device.index:
        st = fn(*args, raw)
    else:
        import torch

        with torch.cuda.device(device):
            st = fn(*args, raw)
    if st != SGEMM_OK:
        raise SgemmError(st, sgemm_f32_status_string(st))


def f8_gemm(A, SA, B, SB, C, alpha=1.0, beta=0.0, b_scale="tile", workspace=None, stream=None):
    """C <- alpha*A*B^T + beta*C, in place; returns C.

    A (M, K) and B (N, K) are float8_e4m3fn or float8_e5m2 (each its own), C
    (M, N) is float32, float16 or bfloat16; rows may be strided.  SA
    (ceil(K/128), M) holds A's scales, one per 128 values of a row; SB holds
    B's: (ceil(N/128), ceil(K/128)) with ``b_scale`` "tile" (weights), or
    (ceil(K/128), N) with "row".  ``workspace``: a contiguous device tensor lent
    for partial sums where there are few output tiles, and for operands whose rows
    do not start on 16-byte boundaries (sgemm_f8_gemm_workspace says how many
    bytes serve; the call takes the fastest way that fits).
    """
    dev = _device(C)
    block = F8_BLOCK[b_scale]
    fa, M, K, pa, lda = _matrix("A", A, _FORMAT_OF, dev)
    fb, N, kb, pb, ldb = _matrix("B", B, _FORMAT_OF, dev)
    ct, mc, nc, pc, ldc = _matrix("C", C, _TYPE_OF, dev)
    if kb != K or mc != M or nc != N:
        raise ValueError(f"shape mismatch: A {(M, K)}, B {(N, kb)}, C {(mc, nc)}")
    psa, ldsa = _scale("SA", SA, (_blocks(K), M), dev)
    psb, ldsb = _scale("SB", SB, _scale_shape(block, N, K), dev)
    pw, nw = _workspace(workspace, dev)
    _run(dev, stream, _load_f8().sgemm_f8_gemm,
         (fa, fb, block, ct, M, N, K, alpha, pa, lda, psa, ldsa, pb, ldb, psb, ldsb, beta, pc, ldc, pw, nw))
    return C


def f8_quantize(X, Q=None, S=None, QT=None, ST=None, block="row", stream=None):
    """X (rows, cols; float32, float16 or bfloat16) -> 8-bit values with scales.

    Q (rows, cols) and S receive X, QT (cols, rows) and ST receive X^T; either
    pair may be left out.  ``block`` "row": one scale per 128 values of a row of
    the output, S (ceil(cols/128), rows), ST (ceil(rows/128), cols); "tile": one
    per 128 x 128, S (ceil(rows/128), ceil(cols/128)), ST its transpose.  The
    format is Q's (and QT's) type.
    """
    dev = _device(X)
    b = F8_BLOCK[block]
    xt, rows, cols, px, ldx = _matrix("X", X, _TYPE_OF, dev)
    fmt = fq = fqt = 0
    pq = ldq = ps = lds = pqt = ldqt = pst = ldst = 0
    if Q is not None:
        fq, r, c, pq, ldq = _matrix("Q", Q, _FORMAT_OF, dev)
        if (r, c) != (rows, cols):
            raise ValueError(f"Q has shape {(r, c)}, not {(rows, cols)}")
        if S is None:
            raise ValueError("Q needs S")
        ps, lds = _scale("S", S, _scale_shape(b, rows, cols), dev)
    if QT is not None:
        fqt, r, c, pqt, ldqt = _matrix("QT", QT, _FORMAT_OF, dev)
        if (r, c) != (cols, rows):
            raise ValueError(f"QT has shape {(r, c)}, not {(cols, rows)}")
        if ST is None:
            raise ValueError("QT needs ST")
        pst, ldst = _scale("ST", ST, _scale_shape(b, cols, rows), dev)
    fmt = fq or fqt
    if fmt == 0:
        raise ValueError("neither Q nor QT is given")
    if fq and fqt and fq != fqt:
        raise TypeError("Q and QT must have the same format")
    _run(dev, stream, _load_f8().sgemm_f8_quantize,
         (b, fmt, xt, rows, cols, px, ldx, pq, ldq, ps, lds, pqt, ldqt, pst, ldst))


def rmsnorm(X, W, eps=1e-6, residual=None, H=None, Y=None, Q=None, S=None, rstd=None, stream=None):
    """h = X + residual, y = h / sqrt(mean(h^2) + eps) * W, row by row.

    X, residual, H and Y are (rows, cols) of one type (float32, float16 or
    bfloat16); W (cols) is of that type or float32.  Written where given: H <- h
    (may be X or residual itself), Y <- y, Q (float8_e4m3fn) with S
    (ceil(cols/128), rows) <- y in 8 bits, rstd (rows, float32) for the backward
    pass.
    """
    dev = _device(X)
    t, rows, cols, px, ldx = _matrix("X", X, _TYPE_OF, dev)
    wt, pw = _vector("W", W, cols, dev, _TYPE_OF)
    if wt != t and wt != 0:
        raise TypeError("W must be of X's type or float32")

    def like(name, m):
        if m is None:
            return 0, 0
        k, r, c, p, ld = _matrix(name, m, _TYPE_OF, dev)
        if k != t or (r, c) != (rows, cols):
            raise ValueError(f"{name} must be of X's type and shape")
        return p, ld

    pr, ldr = like("residual", residual)
    ph, ldh = like("H", H)
    py, ldy = like("Y", Y)
    pq = ldq = ps = lds = prs = 0
    if Q is not None:
        fq, r, c, pq, ldq = _matrix("Q", Q, _FORMAT_OF, dev)
        if fq != 1 or (r, c) != (rows, cols):
            raise ValueError("Q must be float8_e4m3fn of X's shape")
        if S is None:
            raise ValueError("Q needs S")
        ps, lds = _scale("S", S, (_blocks(cols), rows), dev)
    if rstd is not None:
        prs = _vector("rstd", rstd, rows, dev, _F32)[1]
    _run(dev, stream, _load_f8().sgemm_f8_rmsnorm,
         (t, wt, rows, cols, px, ldx, pr, ldr, pw, eps, ph, ldh, py, ldy, pq, ldq, ps, lds, prs))


def rmsnorm_backward(dY, H, W, rstd, dX, dW=None, workspace=None, dH=None, stream=None):
    """Gradients of the norm: dX (of X and of the residual alike) and dW.

    dY is the gradient of y, H and rstd are what the forward pass kept, dH the
    gradient that reaches h along the residual path (or None).  dX may be dY,
    dH or H itself.  dW (cols, float32) needs a ``workspace`` of
    sgemm_f8_rmsnorm_bwd_plan's bytes.
    """
    dev = _device(dY)
    t, rows, cols, pdy, lddy = _matrix("dY", dY, _TYPE_OF, dev)
    wt, pw = _vector("W", W, cols, dev, _TYPE_OF)
    if wt != t and wt != 0:
        raise TypeError("W must be of dY's type or float32")

    def like(name, m):
        if m is None:
            return 0, 0
        k, r, c, p, ld = _matrix(name, m, _TYPE_OF, dev)
        if k != t or (r, c) != (rows, cols):
            raise ValueError(f"{name} must be of dY's type and shape")
        return p, ld

    ph, ldh = like("H", H)
    pdh, lddh = like("dH", dH)
    pdx, lddx = like("dX", dX)
    prs = _vector("rstd", rstd, rows, dev, _F32)[1]
    pdw = _vector("dW", dW, cols, dev, _F32)[1] if dW is not None else 0
    pws, nws = _workspace(workspace, dev)
    _run(dev, stream, _load_f8().sgemm_f8_rmsnorm_bwd,
         (t, wt, rows, cols, pdy, lddy, ph, ldh, pw, prs, pdh, lddh, pdx, lddx, pdw, pws, nws))
