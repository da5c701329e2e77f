"""The norm over more rows than 2^22 (a norm per head of many tokens): the first, the
last and some rows between against the formula in FP64, the others against the same
call on a part of the rows."""
import pytest

import fp32_gemm_08_amd as lib

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.mark.parametrize("cols", [128, 40])
def test_rows_past_2_to_the_22(cols):
    import torch

    rows = (1 << 22) + 37
    g = torch.Generator(device="cuda").manual_seed(cols)
    X = torch.randn(rows, cols, generator=g, device="cuda").to(torch.bfloat16)
    W = (1 + 0.1 * torch.randn(cols, generator=g, device="cuda")).to(torch.bfloat16)

    def call(x):
        n = x.shape[0]
        y, rs = torch.empty_like(x), torch.empty(n, device="cuda")
        q, s = torch.empty(n, cols, dtype=torch.float8_e4m3fn, device="cuda"), torch.empty(1, n, device="cuda")
        lib.rmsnorm(x, W, 1e-6, Y=y, Q=q, S=s, rstd=rs)
        return y, q.view(torch.uint8), s, rs

    y, q, s, rs = call(X)
    pick = torch.cat([torch.arange(64), torch.arange(12345, rows, 65521), torch.arange(rows - 64, rows)]).cuda()
    x = X[pick].double()
    want = 1 / torch.sqrt((x * x).mean(1) + 1e-6)
    # a sum of `cols` products and the steps after it; bf16 rounds by half a step of 2^-8
    assert bool(((rs[pick] - want).abs() <= 64 * U * want).all())
    want = x * want[:, None] * W.double()
    assert bool(((y[pick].double() - want).abs() <= (64 * U + 2.0 ** -8) * want.abs()).all())
    for lo in range(0, rows, 1 << 20):                            # (a workgroup's rows stay together)
        hi = min(lo + (1 << 20), rows)
        y1, q1, s1, rs1 = call(X[lo:hi])
        assert torch.equal(y[lo:hi], y1) and torch.equal(q[lo:hi], q1)
        assert torch.equal(s[:, lo:hi], s1) and torch.equal(rs[lo:hi], rs1)
