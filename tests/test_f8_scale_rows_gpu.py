"""C <- beta * C, the product left out, where C has more rows than workgroups and more
than 2^31 elements apart."""
import pytest

import fp32_gemm_08_amd as lib

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("beta", [0.0, -0.5])
@pytest.mark.parametrize("M,N,ld", [((1 << 24) + 5, 3, 130), ((1 << 20) - 1, 5, 6), ((1 << 20) + 1, 300, 301)])
def test_many_rows(M, N, ld, beta):
    import torch

    g = torch.Generator(device="cuda").manual_seed(M)
    held = torch.randn(M, ld, generator=g, device="cuda", dtype=torch.float32).to(torch.bfloat16)
    want = held.clone()
    want[:, :N] = want[:, :N] * beta if beta else 0           # a power of two: exact
    f8 = torch.float8_e4m3fn
    A, B = torch.empty(M, 0, dtype=f8, device="cuda"), torch.empty(N, 0, dtype=f8, device="cuda")
    SA, SB = torch.empty(0, M, device="cuda"), torch.empty(0, N, device="cuda")
    lib.f8_gemm(A, SA, B, SB, held[:, :N], beta=beta, b_scale="row")
    assert torch.equal(held, want)
