"""C <- beta * C, the product left out, of more rows than one launch has workgroups of
256 work-items for (no GPU): taken, as the product over so many rows is."""
import os

import pytest

import fp32_gemm_08_amd as lib

NO_DEVICE = 3
P = {name: (i + 1) << 44 for i, name in enumerate("A SA B SB C".split())}


@pytest.mark.parametrize("M", [(1 << 24) - 1, 1 << 24, 1 << 26])
@pytest.mark.parametrize("K,alpha", [(0, 1.0), (256, 0.0), (256, 1.0)])
def test_rows_with_and_without_a_product(M, K, alpha):
    if not os.path.exists(lib.LIB_PATH):
        pytest.skip("libsgemm_f32.so not built")
    torch = pytest.importorskip("torch")
    if torch.cuda.is_available():
        pytest.skip("a GPU is here, and the addresses are made up")
    N = 64
    assert lib.sgemm_f8_gemm(1, 1, 0, 2, M, N, K, alpha, P["A"], max(K, 1), P["SA"], M, P["B"], max(K, 1), P["SB"], N,
                             0.5, P["C"], N, 0, 0, 0) == NO_DEVICE
