"""The norms around a block without rows, over torch tensors: a gate of every form is taken, and
the sums over rows are 0."""
import pytest

import fp32_gemm_08_amd as lib

from gpu_helpers import say
from test_f8_gpu import need_gpu  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("gate_shape,gate_rows", [((40,), None), ((40,), 0), ((0, 40), None), ((0, 40), 1), ((1, 40), None),
                                                  ((3, 40), None), ((3, 40), 7)])
@pytest.mark.parametrize("pad", [0, 5])
def test_gates_without_rows(gate_shape, gate_rows, pad):
    import torch

    say(f"no rows, gate {gate_shape}, gate_rows={gate_rows}, pad={pad}")
    e, r = torch.empty(0, 40, device="cuda"), torch.empty(0, device="cuda")
    W, gate = torch.ones(40, device="cuda"), torch.randn(gate_shape, device="cuda")
    lib.block_norm(e, e, W, w_post=W, gate=gate, gate_rows=gate_rows, H=e, rstd=r, rstd_post=r)
    dW, dWP = (torch.full((40,), 7.0, device="cuda") for _ in range(2))
    held = torch.full((max(len(gate), 1), 40 + pad), 7.0, device="cuda")
    dG = (held[:len(gate)] if gate.dim() == 2 else held[0])[..., :40]
    lib.block_norm_backward(e, e, e, W, r, e, e, w_post=W, rstd_post=r, gate=gate, gate_rows=gate_rows, dW=dW, dW_post=dWP,
                            dGate=dG)
    torch.cuda.synchronize()
    assert bool((dW == 0).all()) and bool((dWP == 0).all()) and bool((dG == 0).all())
    held[:, :40] = 7.0
    lib.block_norm_backward(e, e, e, W, r, e, e, w_post=W, rstd_post=r, gate=gate, gate_rows=gate_rows, dGate=dG)   # alone
    assert bool((dG == 0).all()) and bool((held[:, 40:] == 7).all())


def test_negative_gate_rows_without_rows():
    import torch

    e = torch.empty(0, 40, device="cuda")
    with pytest.raises(ValueError):
        lib.block_norm(e, e, torch.ones(40, device="cuda"), gate=torch.ones(40, device="cuda"), gate_rows=-1, H=e)
