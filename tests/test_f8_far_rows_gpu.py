"""The norm, its backward pass, the transposed quantisation and tile scales where rows
lie so far apart that offsets pass 2^31 elements, every output compared.

The tolerances are those of test_f8_gpu.py, where they are derived."""
import numpy as np
import pytest

import fp32_gemm_08_amd as lib
from oracle import oracle_f8 as o8

from test_f8_gpu import HALF, TINY, U, check_q, codes, data, f64, need_gpu, operand, put, rounded, tt  # noqa: F401

pytestmark = pytest.mark.gpu
ROWS, COLS, LD = 300, 136, 1 << 23                        # the last rows start past 2^31 elements


def far(dtype, x=None, rows=ROWS, cols=COLS, ld=LD):
    import torch

    t = torch.empty(rows * ld, dtype=dtype, device="cuda").view(rows, ld)[:, :cols]
    return t if x is None else put(t, x)


@pytest.mark.parametrize("in_place", [None, "x", "r"])
def test_norm_forward(in_place):
    import torch

    rng = np.random.default_rng(61)
    x, r = data(rng, ROWS, COLS, "bf16"), data(rng, ROWS, COLS, "bf16")
    w = rounded(1 + 0.3 * rng.standard_normal(COLS), "bf16")
    X, R, Y = far(torch.bfloat16, x), far(torch.bfloat16, r), far(torch.bfloat16)
    H = {"x": X, "r": R}.get(in_place)
    H = far(torch.bfloat16) if H is None else H
    Q = far(torch.uint8).view(tt("e4m3"))
    S = torch.empty(2 * (1 << 31), device="cuda").view(2, 1 << 31)[:, :ROWS]
    rs = torch.empty(ROWS, device="cuda")
    lib.rmsnorm(X, torch.from_numpy(w).cuda().to(torch.bfloat16), 1e-6, residual=R, H=H, Y=Y, Q=Q, S=S, rstd=rs)
    h, rstd, y = o8.rmsnorm(x, r, w, 1e-6)
    assert np.all(np.abs(f64(H) - h) <= U * np.abs(h) * 2 + HALF["bf16"] * np.abs(h) + TINY["bf16"])
    assert np.all(np.abs(f64(Y) - y) <= 64 * U * np.abs(y) + HALF["bf16"] * np.abs(y) * (1 + 64 * U) + TINY["bf16"])
    assert np.all(np.abs(f64(rs) - rstd) <= 48 * U * rstd)
    check_q(codes(Q), S.cpu().numpy(), y)


@pytest.mark.parametrize("in_place", [None, "dy", "h", "dh"])
def test_norm_backward(in_place):
    import torch

    rng = np.random.default_rng(62)
    h, dy, dh = (data(rng, ROWS, COLS, "bf16") for _ in range(3))
    w = rounded(1 + 0.3 * rng.standard_normal(COLS), "bf16")
    rstd = (1.0 / np.sqrt((h.astype(np.float64) ** 2).mean(axis=1) + 1e-6)).astype(np.float32)
    H, DY, DH = far(torch.bfloat16, h), far(torch.bfloat16, dy), far(torch.bfloat16, dh)
    DX = {"dy": DY, "h": H, "dh": DH}.get(in_place)
    DX = far(torch.bfloat16) if DX is None else DX
    dwt = torch.empty(COLS, device="cuda")
    need = lib.sgemm_f8_rmsnorm_bwd_plan(ROWS, COLS)[1]
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    lib.rmsnorm_backward(DY, H, torch.from_numpy(w).cuda().to(torch.bfloat16), torch.from_numpy(rstd).cuda(), DX, dwt,
                         ws, dH=DH)
    dx, dw = o8.rmsnorm_backward(dy, h, w, rstd, dh)
    n, g = h.astype(np.float64) * rstd.astype(np.float64)[:, None], dy.astype(np.float64) * w
    tol = 80 * U * rstd[:, None].astype(np.float64) * (np.abs(g) + np.abs(n) * np.abs(g * n).mean(axis=1, keepdims=True))
    tol = tol + 2 * U * np.abs(dx)
    assert np.all(np.abs(f64(DX) - dx) <= tol + HALF["bf16"] * (np.abs(dx) + tol) + TINY["bf16"])
    groups = max(1, need // (4 * COLS))
    depth = -(-ROWS // groups) + groups / 32 + 36
    assert np.all(np.abs(f64(dwt) - dw) <= 2 * depth * U * np.abs(dy.astype(np.float64) * n).sum(axis=0))


@pytest.mark.parametrize("block", ["row", "tile"])
def test_transposed_quantisation(block):
    import torch

    rng = np.random.default_rng(63)
    x = data(rng, ROWS, COLS, "bf16")
    X = far(torch.bfloat16, x)
    QT = far(torch.uint8, rows=COLS, cols=ROWS, ld=1 << 24)
    shape = (o8.blocks(ROWS), COLS) if block == "row" else (o8.blocks(COLS), o8.blocks(ROWS))
    ST = torch.empty(shape[0] * (1 << 31), device="cuda").view(shape[0], 1 << 31)[:, :shape[1]]
    lib.f8_quantize(X, QT=QT.view(tt("e4m3")), ST=ST, block=block)
    q, s = o8.quantize(np.ascontiguousarray(x.T), block, "e4m3")
    assert np.array_equal(QT.cpu().numpy(), q) and np.array_equal(ST.cpu().numpy(), s)


@pytest.mark.parametrize("N,pad", [(300, 1), (300, 8), (100, 8)])
def test_products_with_tile_scales_far_apart(N, pad):
    """ldsb at which a 32-bit offset of a second row of scales would wrap to the first."""
    import torch

    M, K, ldsb = 260, 520, 1 << 30
    rng = np.random.default_rng(N + pad)
    A, SA, a = operand(rng, M, K, "row", "e4m3", pad, 0)
    B, SB, b = operand(rng, N, K, "tile", "e4m3", pad, 0)
    far_sb = torch.empty(SB.shape[0] * ldsb, device="cuda").view(-1, ldsb)[:, :SB.shape[1]]
    far_sb.copy_(SB)
    C = torch.empty(M, N, device="cuda")
    W = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
    lib.f8_gemm(A, SA, B, far_sb, C, workspace=W)
    D, size = o8.gemm_f8(a, b)
    tol = size * 2 * U * (130 + o8.blocks(K)) + 4 * U * np.abs(D)
    assert np.all(np.abs(f64(C) - D) <= tol + HALF["f32"] * (np.abs(D) + tol) + TINY["f32"])
