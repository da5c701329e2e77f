"""The backward pass of the norms around a block: who sums what, without a GPU (fake
addresses; no call reaches a launch)."""
import itertools

import pytest

import fp32_gemm_08_amd as lib

from test_block_boundary_cpu import NO_DEVICE, OK, bwd, built  # noqa: F401

# gates of the least and most rows that share a workspace's size, on both sides of every
# change of geometry
SHAPES = [(rows, cols, gate_rows) for cols in (8, 130, 300, 513, 1000, 1024, 1500, 4096, 8192, 9001, 32768)
          for rows, gate_rows in ((1, 1), (7, 2), (129, 1), (258, 2), (300, 2), (1000, 7), (1000, 5), (1030, 3), (2048, 16),
                                  (5000, 1), (5000, 40), (70000, 9), (70000, 400), (200000, 1))]


@pytest.mark.parametrize("rows,cols,gate_rows", SHAPES)
def test_the_planned_workspace_serves_whatever_is_asked_for(rows, cols, gate_rows):
    """The bytes of the call's own gate_rows, for every subset of its outputs."""
    torch = pytest.importorskip("torch")
    if torch.cuda.is_available():
        pytest.skip("a GPU is here")
    st, need = lib.sgemm_block_norm_bwd_plan(rows, cols, gate_rows)
    assert st == OK
    for outs in itertools.chain.from_iterable(itertools.combinations(("DX", "DO", "DW", "DWP", "DG"), n) for n in range(1, 6)):
        absent = {k: 0 for k in ("DX", "DO", "DW", "DWP", "DG") if k not in outs}
        assert bwd(rows=rows, cols=cols, gate_rows=gate_rows, wb=need, **absent) == NO_DEVICE, outs
