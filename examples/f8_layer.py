"""One layer trained in 8 bits: out = norm(x + r) W^T, forward and backward.

    python examples/f8_layer.py [--tokens 8192] [--width 4096] [--out 4096] [--steps 20]

The forward pass is one norm (which adds the residual and writes its output in 8
bits with a scale for each 128 values) and one product; the backward pass is one
quantisation of the gradient (along its rows for the input's gradient and along
the tokens for the weight's), one of the normed activations along the tokens, two
products and the norm's backward pass.  The weight is quantised once per update,
in 128 x 128 tiles, for both products that read it.  The results are compared with
the same layer in FP32, and the time of a step is printed.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import fp32_gemm_08_amd as lib  # noqa: E402

BF16, F32, E4M3, E5M2 = torch.bfloat16, torch.float32, torch.float8_e4m3fn, torch.float8_e5m2
EPS = 1e-6


def blocks(n):
    return (n + 127) // 128


class F8Layer:
    """The layer's weight in FP32, its 8-bit forms, and the buffers of a step."""

    def __init__(self, tokens, width, out, device="cuda", seed=0):
        g = torch.Generator(device=device).manual_seed(seed)

        def new(*shape, dtype=F32):
            return torch.empty(*shape, dtype=dtype, device=device)

        self.weight = torch.randn(out, width, generator=g, device=device) * width ** -0.5
        self.gain = torch.ones(width, dtype=F32, device=device)
        self.w8, self.sw = new(out, width, dtype=E4M3), new(blocks(out), blocks(width))
        self.wt8, self.swt = new(width, out, dtype=E4M3), new(blocks(width), blocks(out))
        # forward
        self.h, self.y = new(tokens, width, dtype=BF16), new(tokens, width, dtype=BF16)
        self.y8, self.sy, self.rstd = new(tokens, width, dtype=E4M3), new(blocks(width), tokens), new(tokens)
        self.out = new(tokens, out, dtype=BF16)
        # backward: the gradient along its rows and along the tokens, the activations along the tokens
        self.g8, self.sg = new(tokens, out, dtype=E5M2), new(blocks(out), tokens)
        self.gt8, self.sgt = new(out, tokens, dtype=E5M2), new(blocks(tokens), out)
        self.yt8, self.syt = new(width, tokens, dtype=E4M3), new(blocks(tokens), width)
        self.dy, self.dx = new(tokens, width, dtype=BF16), new(tokens, width, dtype=BF16)
        self.dweight, self.dgain = torch.zeros(out, width, device=device), new(width)
        # one workspace, as large as the neediest call wants it
        need = [lib.sgemm_f8_rmsnorm_bwd_plan(tokens, width)[1]]
        for block, m, n, k in (("tile", tokens, out, width), ("tile", tokens, width, out), ("row", out, width, tokens)):
            aligned = int(k % 16 == 0)
            need.append(lib.sgemm_f8_gemm_workspace(lib.F8_BLOCK[block], m, n, k, aligned)[1])
        self.workspace = new(max(max(need), 16), dtype=torch.uint8)
        self.requantize()

    def requantize(self):
        """After an update of the weight."""
        lib.f8_quantize(self.weight, self.w8, self.sw, self.wt8, self.swt, block="tile")

    def forward(self, x, residual):
        lib.rmsnorm(x, self.gain, EPS, residual=residual, H=self.h, Y=self.y, Q=self.y8, S=self.sy, rstd=self.rstd)
        return lib.f8_gemm(self.y8, self.sy, self.w8, self.sw, self.out, workspace=self.workspace)

    def backward(self, grad, grad_h=None, accumulate=False):
        """grad: of the output; grad_h: what reaches x + r along the residual path.
        Returns the gradient of x (and of the residual), in dx; dweight and dgain are set."""
        lib.f8_quantize(grad, self.g8, self.sg, self.gt8, self.sgt)
        lib.f8_quantize(self.y, QT=self.yt8, ST=self.syt)
        lib.f8_gemm(self.g8, self.sg, self.wt8, self.swt, self.dy, workspace=self.workspace)
        lib.f8_gemm(self.gt8, self.sgt, self.yt8, self.syt, self.dweight, beta=1.0 if accumulate else 0.0, b_scale="row",
                    workspace=self.workspace)
        lib.rmsnorm_backward(self.dy, self.h, self.gain, self.rstd, self.dx, self.dgain, self.workspace, dH=grad_h)
        return self.dx


def in_fp32(layer, x, residual, grad, grad_h):
    """The same step by its formulas in FP32: out, dx, dweight, dgain."""
    h = x.float() + residual.float()
    rstd = torch.rsqrt(h.square().mean(1, keepdim=True) + EPS)
    n = h * rstd
    y, g = n * layer.gain, grad.float()
    dy = g @ layer.weight
    p = dy * layer.gain
    dx = rstd * (p - n * (p * n).mean(1, keepdim=True)) + grad_h.float()
    return y @ layer.weight.t(), dx, g.t() @ y, (dy * n).sum(0)


def run(tokens=8192, width=4096, out=4096, steps=20, seed=1):
    """Relative errors (2-norm) of a step's results against FP32, and its time in us."""
    g = torch.Generator(device="cuda").manual_seed(seed)

    def random(*shape, scale=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * scale).to(BF16)

    layer = F8Layer(tokens, width, out)
    x, r = random(tokens, width), random(tokens, width)
    grad, grad_h = random(tokens, out, scale=1e-3), random(tokens, width, scale=1e-3)

    def step():
        layer.forward(x, r)
        layer.backward(grad, grad_h)

    step()
    got = (layer.out, layer.dx, layer.dweight, layer.dgain)
    errors = {name: float((a.float() - b).norm() / b.norm())
              for name, a, b in zip(("out", "dx", "dweight", "dgain"), got, in_fp32(layer, x, r, grad, grad_h))}
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    for _ in range(3):
        step()
    begin.record()
    for _ in range(steps):
        step()
    end.record()
    torch.cuda.synchronize()
    return errors, 1e3 * begin.elapsed_time(end) / max(steps, 1)


if __name__ == "__main__":
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    for name, value in (("tokens", 8192), ("width", 4096), ("out", 4096), ("steps", 20)):
        p.add_argument("--" + name, type=int, default=value)
    a = p.parse_args()
    errors, us = run(a.tokens, a.width, a.out, a.steps)
    flops = 6 * a.tokens * a.width * a.out
    print(f"{a.tokens} tokens, {a.width} -> {a.out}: {us:.1f} us a step, {flops / us * 1e-6:.0f} TFLOP/s of products")
    print("relative error against FP32: " + ", ".join(f"{k} {v:.4f}" for k, v in errors.items()))
