"""The 8-bit layer of examples/f8_layer.py against the same layer in FP32.

Bounds, from the roundings on the way (relative, independent from value to value,
so that they add in squares and pass through a product at their own size): an e4m3
value is off by at most half a step of 2^-3 of it, an e5m2 value of 2^-2, hence by
2^-4 and 2^-3.
  out       activations and weights: sqrt(2) 2^-4 = 0.089, and bf16's 2^-8
  dweight   gradients and activations: sqrt(2^-6 + 2^-8) = 0.140
  dx        gradients and weights: 0.140, of the part that comes through the norm;
            bf16's roundings of dy and dx, 2 * 2^-8
  dgain     dy and the normed rows: 0.140
"""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    spec = importlib.util.spec_from_file_location("f8_layer", os.path.join(ROOT, "examples", "f8_layer.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.parametrize("tokens,width,out", [(512, 512, 768), (300, 257, 130), (1, 640, 640), (1000, 1024, 384)])
def test_layer(example, tokens, width, out):
    errors, us = example.run(tokens, width, out, steps=2)
    print(f"{tokens}x{width}->{out}: {errors} {us:.1f} us", flush=True)
    assert errors["out"] <= 0.089 + 2.0 ** -8
    assert errors["dweight"] <= 0.140 + 2.0 ** -8
    assert errors["dx"] <= 0.140 + 2 * 2.0 ** -8
    assert errors["dgain"] <= 0.140 + 2.0 ** -8


def test_weight_gradient_accumulates(example):
    import torch

    layer = example.F8Layer(256, 256, 256)
    x = torch.randn(256, 256, device="cuda").to(torch.bfloat16)
    g = (torch.randn(256, 256, device="cuda") * 1e-3).to(torch.bfloat16)
    layer.forward(x, x)
    layer.backward(g)
    once = layer.dweight.clone()
    layer.backward(g, accumulate=True)
    # the second product and its addition: one FP32 rounding of a value and of the sum
    assert bool((layer.dweight - 2 * once).abs().max() <= 4 * 2.0 ** -24 * once.abs().max())
