"""How many rows the norm takes in one call (no GPU): as many as one launch of the
row's own class has work-items for, its backward pass any number."""
import os

import pytest

import fp32_gemm_08_amd as lib

INVALID, NO_DEVICE = 1, 3
P = {name: (i + 1) << 44 for i, name in enumerate("X W Y S H DY DX RS".split())}


@pytest.fixture(autouse=True)
def without_a_device():
    if not os.path.exists(lib.LIB_PATH):
        pytest.skip("libsgemm_f32.so not built")
    torch = pytest.importorskip("torch")
    if torch.cuda.is_available():
        pytest.skip("a GPU is here, and the addresses are made up")


def norm(rows, cols):
    return lib.sgemm_f8_rmsnorm(2, 2, rows, cols, P["X"], cols, 0, 0, P["W"], 1e-6, 0, 0, P["Y"], cols, 0, 0, 0, 0, 0)


# columns, and the work-items that hold a row of so many
LANES = [(1, 16), (64, 16), (128, 16), (129, 32), (256, 32), (257, 64), (512, 64), (513, 64), (1024, 64), (1025, 256),
         (4096, 256), (4097, 512), (8192, 512), (8193, 1024), (16384, 1024), (16385, 1024), (32768, 1024)]


@pytest.mark.parametrize("cols,lanes", LANES)
def test_rows_of_one_launch(cols, lanes):
    wg = max(256, lanes)
    most = ((1 << 32) - 1) // wg * (wg // lanes)
    assert norm(most, cols) == NO_DEVICE
    assert norm(most + 1, cols) == INVALID
    assert norm(1, cols) == NO_DEVICE


def test_a_norm_per_head_goes_both_ways():
    rows, cols = 65536 * 64, 128
    assert norm(rows, cols) == NO_DEVICE
    assert lib.sgemm_f8_rmsnorm_bwd(2, 2, rows, cols, P["DY"], cols, P["H"], cols, P["W"], P["RS"], 0, 0, P["DX"], cols,
                                    0, 0, 0) == NO_DEVICE
