"""The norms around a block without rows, at the C ABI (no GPU; no call reaches a launch): a gate
per channel is gate_rows = rows, which is then 0."""
import pytest

from test_block_boundary_cpu import INVALID, NO_DEVICE, OK, bwd, built, norm  # noqa: F401


def test_a_gate_per_channel_without_rows():
    sums = dict(DW=0, DWP=0, DG=0)
    assert norm(rows=0, gate_rows=0) == OK and norm(rows=0, gate_rows=3) == OK
    assert bwd(rows=0, gate_rows=0, **sums) == OK and bwd(rows=0, gate_rows=3, **sums) == OK
    assert norm(rows=0, gate_rows=-1) == INVALID and bwd(rows=0, gate_rows=-1, **sums) == INVALID
    assert norm(gate_rows=0) == INVALID and bwd(gate_rows=0) == INVALID


def test_its_sums_are_still_set():
    torch = pytest.importorskip("torch")
    if torch.cuda.is_available():
        pytest.skip("a GPU is here")
    assert bwd(rows=0, gate_rows=0, ws=0, wb=0) == NO_DEVICE
