"""Forms of the operators around a block that need large or many-gated calls: the requantisation
with four wavefronts a workgroup, the norms' backward pass with several gates a walker where a
work-item has two or four pieces of a row, and with many gates of fp16 rows.  Tolerances: those
of test_block_gpu.py, whose checks these are."""
import pytest

import fp32_gemm_08_amd as lib

from test_block_gpu import run_bwd, run_requantize
from test_f8_gpu import need_gpu  # noqa: F401

pytestmark = pytest.mark.gpu


def blocks(n, size):
    return -(-n // size)


# 128 x 256 tiles enough for four wavefronts a workgroup; wavefronts of 64 columns that the last
# workgroup of a row of tiles has too many: 3, 2, 1, 0
@pytest.mark.parametrize("rows,cols,surplus", [(4100, 2050, 3), (130, 65400, 2), (257, 32677, 1), (16290, 512, 0)])
@pytest.mark.parametrize("fx,fmt", [("e4m3", "e4m3"), ("e5m2", "e4m3"), ("e4m3", "e5m2"), ("e5m2", "e5m2")])
def test_requantize_four_wavefronts(rows, cols, surplus, fx, fmt):
    assert blocks(rows, 128) * blocks(cols, 256) >= 256 and -blocks(cols, 64) % 4 == surplus
    run_requantize(rows, cols, fx, fmt, (0, 0, 0) if fx == fmt else (3, 5, 1))


# more than 64 gates; walkers of two rows: gates shorter than, as long as and longer than that,
# and a last gate that is not full
@pytest.mark.parametrize("cols", [8193, 9001, 16384, 16385, 20000, 32768])
@pytest.mark.parametrize("gate_rows", [1, 2, 3, 4])
@pytest.mark.parametrize("kept", [False, True])
def test_bwd_several_gates_of_wide_rows(cols, gate_rows, kept):
    t = ("bf16", "f32", "fp16")[(cols + gate_rows + kept) % 3]
    run_bwd(299, cols, t, kept=kept, gate_rows=gate_rows, alpha=0.75)


@pytest.mark.parametrize("kw", [dict(post=False), dict(dh=False), dict(dy=False), dict(sums=False), dict(outs="x"), dict(outs="o"),
                                dict(outs=""), dict(wt="f32", pads=(1, 3, 5)), dict(in_place=("xdy", "odh"))])
@pytest.mark.parametrize("cols", [9001, 20000])
def test_bwd_several_gates_of_wide_rows_variants(cols, kw):
    run_bwd(150, cols, "bf16", kept=cols > 16384, gate_rows=2, **kw)


@pytest.mark.parametrize("rows,cols", [(1300, 40), (1300, 300), (1300, 700), (700, 1500), (300, 4000), (300, 8000)])
@pytest.mark.parametrize("gate_rows", [1, 3])
@pytest.mark.parametrize("kept", [False, True])
def test_bwd_many_gates_of_fp16_rows(rows, cols, gate_rows, kept):
    run_bwd(rows, cols, "fp16", kept=kept, gate_rows=gate_rows)


@pytest.mark.parametrize("rows,cols,gate_rows", [(258, 1000, 2), (1000, 700, 7)])
def test_bwd_sums_of_w_alone_with_a_gate_in_the_planned_workspace(rows, cols, gate_rows):
    """Nothing that is asked for reads the gate: the sums of a call without one."""
    import torch

    g = torch.Generator(device="cuda").manual_seed(rows)
    dy, h = (torch.randn(rows, cols, generator=g, device="cuda") for _ in range(2))
    W, rstd = (torch.rand(n, generator=g, device="cuda") + 0.5 for n in (cols, rows))
    gate = torch.randn(blocks(rows, gate_rows), cols, generator=g, device="cuda")
    got = []
    for kw, plan in ((dict(gate=gate, gate_rows=gate_rows), gate_rows), ({}, 0)):
        ws = torch.full((lib.sgemm_block_norm_bwd_plan(rows, cols, plan)[1],), 0xA5, dtype=torch.uint8, device="cuda")
        dx, dw = torch.empty_like(dy), torch.empty(cols, device="cuda")
        lib.block_norm_backward(dy, h, None, W, rstd, dx, None, dW=dw, workspace=ws, **kw)
        got.append((dx, dw))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
