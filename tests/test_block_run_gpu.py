"""The operators around a block together, as a layer uses them: serving through 8-bit integers,
training with the activations kept in 8 bits; eager, captured and replayed, and from several
threads at once.

Each step is held to its definition on what the steps before it left on the device; the end of
the serving chain also to the FP64 chain from the inputs: an integer is off by half a step of
its scale and by y's own error, whose bound test_block_gpu.py derives."""
import threading

import numpy as np
import pytest

import fp32_gemm_08_amd as lib
from oracle import oracle_block as ob
from oracle import oracle_f8 as o8

from gpu_helpers import say
from test_block_gpu import check_blocks
from test_f8_gpu import HALF, TINY, U, codes, data, f64, need_gpu, rounded, tt  # noqa: F401

pytestmark = pytest.mark.gpu
EPS = 1e-6


def new(*shape, t):
    import torch

    return torch.empty(*shape, dtype=t if isinstance(t, torch.dtype) else tt(t), device="cuda")


def on_gpu(x, t):
    import torch

    return torch.from_numpy(np.ascontiguousarray(x)).to(tt(t)).cuda()


# ------------------------------------------------------------------ serving

@pytest.mark.parametrize("rows,cols,out", [(1, 512, 384), (1, 1017, 999), (5, 4096, 640), (70, 520, 300), (300, 1040, 260)])
def test_tokens_through_a_layer_of_integers(rows, cols, out):
    import torch

    say(f"serving {rows} x {cols} -> {out}")
    rng = np.random.default_rng(rows + cols)
    x, o = (data(rng, rows, cols, "bf16") for _ in range(2))
    w, wp = (rounded(1 + 0.3 * rng.standard_normal(cols), "bf16") for _ in range(2))
    layer = (0.05 * rng.standard_normal((out, cols))).astype(np.float32)
    X, O, W, WP = (on_gpu(v, "bf16") for v in (x, o, w, wp))
    B, SB = new(out, cols, t=torch.int8), new(out, t="f32")
    lib.i8_quantize(on_gpu(layer, "f32"), B, SB)
    Q, S, C = new(rows, cols, t=torch.int8), new(rows, t="f32"), new(rows, out, t="bf16")
    ws = new(max(lib.sgemm_i8_gemm_workspace(rows, out, cols, al)[1] for al in (0, 1)) + 16, t=torch.uint8)
    lib.block_norm(X, O, W, EPS, w_post=WP, H=X, Q=Q, S=S)          # the residual stream is updated in place
    lib.i8_gemm(Q, S, B, SB, C, workspace=ws)
    torch.cuda.synchronize()
    h, y, rstd, _, z = ob.block_norm(x, o, w, EPS, wp)
    eh = 54 * U * (np.abs(x) + np.abs(z))
    assert np.all(np.abs(f64(X) - h) <= eh + HALF["bf16"] * (np.abs(h) + eh) + TINY["bf16"])
    # on what is on the device: exact sums, four roundings and half a step
    b, sb = B.cpu().numpy(), SB.cpu().numpy()
    qb, sb1 = ob.quantize_rows_i8(layer)
    assert np.array_equal(b, qb) and np.array_equal(sb, sb1)
    D, s = ob.gemm_i8(Q.cpu().numpy(), S.cpu().numpy(), b, sb)
    tol = 5.1 * U * np.abs(D)
    assert np.all(np.abs(f64(C) - D) <= tol + HALF["bf16"] * (np.abs(D) + tol) + TINY["bf16"])
    # from the inputs
    rho = (np.abs(h) * eh).sum(axis=1) / (h * h).sum(axis=1) + 48 * U
    ey = np.abs(rstd[:, None] * w) * eh + np.abs(y) * (rho[:, None] + 3 * U)
    wide = b.astype(np.float64) * sb[:, None].astype(np.float64)
    step = (np.abs(y).max(axis=1) + ey.max(axis=1)) / 127 * (1 + 4 * U)
    off = (0.5 * step[:, None] + 2 * ey + 8 * U * np.abs(y).max(axis=1, keepdims=True)) @ np.abs(wide).T
    E = y @ wide.T
    tol = off + 5.1 * U * (np.abs(E) + off)
    assert np.all(np.abs(f64(C) - E) <= tol + HALF["bf16"] * (np.abs(E) + tol) + TINY["bf16"])


# ------------------------------------------------------------------ training

class Layer:
    """norms around a block -> product in 8 bits; the backward pass from what is kept: the
    product's two gradients, the weight's from the requantised activations, and the norms'."""

    def __init__(self, rows, cols, out, gates, alpha=0.75):
        import torch

        self.rows, self.cols, self.out, self.gates, self.alpha = rows, cols, out, gates, alpha
        self.gate_rows = -(-rows // gates)
        kb, rb, ob_ = o8.blocks(cols), o8.blocks(rows), o8.blocks(out)
        self.blocks = kb, rb, ob_
        self.X, self.O, self.DY, self.DH = (new(*s, t="bf16") for s in ((rows, cols), (rows, cols), (rows, out), (rows, cols)))
        self.G = new(gates, cols, t="bf16")
        self.W, self.WP = new(cols, t="bf16"), new(cols, t="bf16")
        self.B, self.SB = new(out, cols, t="e4m3"), new(ob_, kb, t="f32")
        self.BT, self.SBT = new(cols, out, t="e4m3"), new(kb, ob_, t="f32")
        g = torch.Generator(device="cuda").manual_seed(9)
        lib.f8_quantize(torch.randn(out, cols, generator=g, device="cuda") * 0.05, self.B, self.SB, self.BT, self.SBT, block="tile")

    def fill(self, seed):
        import torch

        g = torch.Generator(device="cuda").manual_seed(seed)
        for t in (self.X, self.O, self.DY, self.DH, self.G):
            t.copy_(torch.randn(t.shape, generator=g, device="cuda"))
        for t in (self.W, self.WP):
            t.copy_(1 + 0.3 * torch.randn(t.shape, generator=g, device="cuda"))

    def buffers(self):
        import torch

        rows, cols, out = self.rows, self.cols, self.out
        kb, rb, ob_ = self.blocks
        need = max(lib.sgemm_block_norm_bwd_plan(rows, cols, self.gate_rows)[1], 16 << 20)
        return dict(H=new(rows, cols, t="bf16"), Q=new(rows, cols, t="e4m3"), S=new(kb, rows, t="f32"),
                    H8=new(rows, cols, t="e4m3"), SH=new(kb, rows, t="f32"), O8=new(rows, cols, t="e4m3"),
                    SO=new(kb, rows, t="f32"), rs=new(rows, t="f32"), rp=new(rows, t="f32"), C=new(rows, out, t="bf16"),
                    D8=new(rows, out, t="e5m2"), SD=new(ob_, rows, t="f32"), DT=new(out, rows, t="e5m2"),
                    SDT=new(rb, out, t="f32"), QT=new(cols, rows, t="e4m3"), SQT=new(rb, cols, t="f32"),
                    dQ=new(rows, cols, t="bf16"), dB=new(out, cols, t="f32"), dX=new(rows, cols, t="bf16"),
                    dO=new(rows, cols, t="bf16"), dW=new(cols, t="f32"), dWP=new(cols, t="f32"),
                    dG=new(self.gates, cols, t="f32"), ws=new(need, t=torch.uint8))

    def step(self, b):
        lib.block_norm(self.X, self.O, self.W, EPS, w_post=self.WP, gate=self.G, gate_rows=self.gate_rows, alpha=self.alpha,
                       H=b["H"], Q=b["Q"], S=b["S"], H8=b["H8"], SH=b["SH"], O8=b["O8"], SO=b["SO"], rstd=b["rs"],
                       rstd_post=b["rp"])
        lib.f8_gemm(b["Q"], b["S"], self.B, self.SB, b["C"], workspace=b["ws"])
        lib.f8_quantize(self.DY, b["D8"], b["SD"], b["DT"], b["SDT"])
        lib.f8_gemm(b["D8"], b["SD"], self.BT, self.SBT, b["dQ"], workspace=b["ws"])
        lib.f8_requantize(b["Q"], b["S"], b["QT"], b["SQT"])
        lib.f8_gemm(b["DT"], b["SDT"], b["QT"], b["SQT"], b["dB"], b_scale="row", workspace=b["ws"])
        lib.block_norm_backward(b["dQ"], b["H8"], b["O8"], self.W, b["rs"], b["dX"], b["dO"], SH=b["SH"], SO=b["SO"],
                                w_post=self.WP, rstd_post=b["rp"], gate=self.G, gate_rows=self.gate_rows, alpha=self.alpha,
                                dH=self.DH, dW=b["dW"], dW_post=b["dWP"], dGate=b["dG"], workspace=b["ws"])


def same(a, b):
    import torch

    return [k for k in a if k != "ws" and not torch.equal(a[k].view(torch.uint8), b[k].view(torch.uint8))]


@pytest.mark.parametrize("rows,cols,out,gates", [(300, 272, 200, 2), (130, 520, 264, 1), (257, 333, 129, 5)])
def test_a_layer_trained_from_what_it_keeps_in_8_bits(rows, cols, out, gates):
    import torch

    say(f"training {rows} x {cols} -> {out}, {gates} gates")
    layer = Layer(rows, cols, out, gates)
    layer.fill(1)
    b = layer.buffers()
    layer.step(b)
    torch.cuda.synchronize()
    x, o, w, wp, gate, dh = (f64(t) for t in (layer.X, layer.O, layer.W, layer.WP, layer.G, layer.DH))
    h, y, rstd, rpost, z = ob.block_norm(x, o, w, EPS, wp, gate, layer.gate_rows, layer.alpha)
    eh = 54 * U * (np.abs(layer.alpha * x) + np.abs(ob.gate_of_rows(gate, layer.gate_rows, rows) * z))
    rho = (np.abs(h) * eh).sum(axis=1) / (h * h).sum(axis=1) + 48 * U
    ey = np.abs(rstd[:, None] * w) * eh + np.abs(y) * (rho[:, None] + 3 * U)
    check_blocks(codes(b["Q"]), b["S"].cpu().numpy(), y, ey)
    check_blocks(codes(b["H8"]), b["SH"].cpu().numpy(), h, eh)

    def kept(q, s, fmt="e4m3"):
        return o8.values(codes(b[q]), b[s].cpu().numpy(), "row", fmt)

    # the weight's gradient: requantised exactly as defined; then FP32 sums of its product
    q8 = o8.decode(codes(b["Q"]), "e4m3").astype(np.float32) * o8.spread(b["S"].cpu().numpy().T, "row", rows, cols)
    c, s = o8.quantize(q8.T, "row", "e4m3")
    assert np.array_equal(codes(b["QT"]), c) and np.array_equal(b["SQT"].cpu().numpy(), s)
    dt, qt = kept("DT", "SDT", "e5m2").astype(np.float64), kept("QT", "SQT").astype(np.float64)
    D, size = dt @ qt.T, np.abs(dt) @ np.abs(qt).T
    assert np.all(np.abs(f64(b["dB"]) - D) <= size * 2 * U * (130 + layer.blocks[1]) + 5 * U * np.abs(D))
    # the norms' gradients on the gradient that reached them
    e = ob.block_norm_backward(f64(b["dQ"]), dh, kept("H8", "SH"), kept("O8", "SO"), w, f64(b["rs"]), wp, f64(b["rp"]), gate,
                               layer.gate_rows, layer.alpha)
    for name, ref, depth in (("dX", "dx", 82), ("dO", "do", 150)):
        tol = depth * U * e[ref + "_size"]
        assert np.all(np.abs(f64(b[name]) - e[ref]) <= tol + HALF["bf16"] * (np.abs(e[ref]) + tol) + TINY["bf16"]), name
    # a sum over the rows has at most that many additions, and its terms 90 u
    for name, ref in (("dW", "dw"), ("dWP", "dw_post"), ("dG", "dgate")):
        assert np.all(np.abs(f64(b[name]) - e[ref]) <= (2 * rows + 90) * U * e[ref + "_size"]), name


def test_a_layer_captured_and_replayed():
    """Replays on new inputs, with the same calls made eagerly between them."""
    import torch

    layer = Layer(300, 272, 200, 2)
    held, eager = layer.buffers(), layer.buffers()
    layer.fill(0)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        layer.step(held)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer.step(held)
    for seed in (1, 2, 3, 4):
        layer.fill(seed)
        graph.replay()
        torch.cuda.synchronize()
        layer.step(eager)
        torch.cuda.synchronize()
        assert not same(held, eager), (seed, same(held, eager))


@pytest.mark.parametrize("rows,cols,out", [(1, 4096, 4096), (24, 520, 2000), (200, 272, 300)])
def test_tokens_captured_and_replayed(rows, cols, out):
    """Serving in a graph, a k-split's partial sums in a workspace that only it uses."""
    import torch

    B, SB = new(out, cols, t=torch.int8), new(out, t="f32")
    lib.i8_quantize(torch.randn(out, cols, device="cuda"), B, SB)
    X, O = new(rows, cols, t="bf16"), new(rows, cols, t="bf16")
    W = torch.ones(cols, dtype=torch.bfloat16, device="cuda")
    need = lib.sgemm_i8_gemm_workspace(rows, out, cols)[1] + 16

    def buffers():
        return dict(H=new(rows, cols, t="bf16"), Q=new(rows, cols, t=torch.int8), S=new(rows, t="f32"), C=new(rows, out, t="bf16"),
                    Q2=new(rows, out, t=torch.int8), S2=new(rows, t="f32"), ws=new(need, t=torch.uint8))

    def step(b):
        lib.block_norm(X, O, W, EPS, w_post=W, H=b["H"], Q=b["Q"], S=b["S"])
        lib.i8_gemm(b["Q"], b["S"], B, SB, b["C"], workspace=b["ws"])
        lib.i8_quantize(b["C"], b["Q2"], b["S2"])

    def fill(seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        for t in (X, O):
            t.copy_(torch.randn(t.shape, generator=g, device="cuda"))

    held, eager = buffers(), buffers()
    fill(0)
    step(held)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(held)
    for seed in (1, 2, 3):
        fill(seed)
        graph.replay()
        torch.cuda.synchronize()
        step(eager)
        torch.cuda.synchronize()
        assert not same(held, eager), (seed, same(held, eager))


# ------------------------------------------------------------------ streams and threads

def test_layers_on_streams_of_their_own_from_threads():
    """Four threads, a stream and buffers each, the same bits as each alone."""
    import torch

    layers = [Layer(*s) for s in ((300, 272, 200, 2), (130, 520, 264, 1), (257, 333, 129, 5), (64, 1024, 128, 1))]
    alone, got, errors = [], [], []
    for i, layer in enumerate(layers):
        layer.fill(20 + i)
        alone.append(layer.buffers())
        layer.step(alone[i])
        got.append([layer.buffers() for _ in range(4)])
    torch.cuda.synchronize()
    start = threading.Barrier(len(layers))

    def work(i):
        try:
            s = torch.cuda.Stream()
            start.wait()
            with torch.cuda.stream(s):
                for b in got[i]:
                    layers[i].step(b)
            s.synchronize()
        except BaseException as e:  # reported by the main thread
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(layers))]
    for t in threads:
        t.start()
    for t in threads:
        t.join(timeout=100)
    assert not any(t.is_alive() for t in threads)
    if errors:
        raise errors[0]
    torch.cuda.synchronize()
    for i, runs in enumerate(got):
        for b in runs:
            assert not same(alone[i], b), (i, same(alone[i], b))


def test_a_stream_that_is_named():
    import torch

    rows, cols = 70, 520
    s = torch.cuda.Stream()
    g = torch.Generator(device="cuda").manual_seed(3)
    X, O = (torch.randn(rows, cols, generator=g, device="cuda").bfloat16() for _ in range(2))
    W = torch.ones(cols, dtype=torch.bfloat16, device="cuda")

    def run(stream):
        b = dict(H=new(rows, cols, t="bf16"), H8=new(rows, cols, t="e4m3"), SH=new(5, rows, t="f32"), rs=new(rows, t="f32"),
                 Q=new(rows, cols, t=torch.int8), S=new(rows, t="f32"), QT=new(cols, rows, t="e4m3"), SQT=new(1, cols, t="f32"),
                 Q2=new(rows, cols, t=torch.int8), S2=new(rows, t="f32"), dX=new(rows, cols, t="bf16"), dW=new(cols, t="f32"))
        ws = new(lib.sgemm_block_norm_bwd_plan(rows, cols)[1], t=torch.uint8)
        torch.cuda.synchronize()
        lib.block_norm(X, O, W, EPS, H=b["H"], H8=b["H8"], SH=b["SH"], Q=b["Q"], S=b["S"], rstd=b["rs"], stream=stream)
        lib.f8_requantize(b["H8"], b["SH"], b["QT"], b["SQT"], stream=stream)
        lib.i8_quantize(b["H"], b["Q2"], b["S2"], stream=stream)
        lib.block_norm_backward(O, b["H"], None, W, b["rs"], b["dX"], None, dW=b["dW"], workspace=ws, stream=stream)
        torch.cuda.synchronize()
        return b

    assert not same(run(None), run(s))


def test_padded_rows_behind_the_last_sequence_stay():
    """A batch whose last rows hold no tokens: calls on the rows before them leave them as they are."""
    import torch

    rows, used, cols, out = 40, 27, 264, 136
    X, O = (torch.randn(rows, cols, device="cuda").bfloat16() for _ in range(2))
    X[used:], O[used:] = float("nan"), float("inf")
    W = torch.ones(cols, dtype=torch.bfloat16, device="cuda")
    H, Q, S, C = X.clone(), new(rows, cols, t=torch.int8).fill_(5), new(rows, t="f32").fill_(7), new(rows, out, t="bf16").fill_(9)
    B, SB = new(out, cols, t=torch.int8), new(out, t="f32")
    lib.i8_quantize(torch.randn(out, cols, device="cuda"), B, SB)
    lib.block_norm(X[:used], O[:used], W, EPS, w_post=W, H=H[:used], Q=Q[:used], S=S[:used])
    lib.i8_gemm(Q[:used], S[:used], B, SB, C[:used])
    assert bool((Q[used:] == 5).all()) and bool((S[used:] == 7).all()) and bool((C[used:] == 9).all())
    assert bool(H[used:].isnan().all()) and bool(torch.isfinite(H[:used]).all()) and bool(torch.isfinite(C[:used]).all())
    # gradients: the padding's are not part of the sums
    rs, dW = torch.ones(rows, device="cuda"), new(cols, t="f32")
    dX = new(rows, cols, t="bf16").fill_(3)
    ws = new(lib.sgemm_block_norm_bwd_plan(used, cols)[1], t=torch.uint8)
    lib.block_norm_backward(X[:used], H[:used], None, W, rs[:used], dX[:used], None, dW=dW, workspace=ws)
    assert bool(torch.isfinite(dW).all()) and bool((dX[used:] == 3).all()) and bool(torch.isfinite(dX[:used]).all())


@pytest.mark.parametrize("cols,gates", [(9001, 4), (20000, 3), (16384, 7)])
@pytest.mark.parametrize("kept", [False, True])
def test_gates_of_wide_rows(cols, gates, kept):
    from test_block_gpu import run_bwd

    run_bwd(20, cols, "bf16", kept=kept, gate_rows=-(-20 // gates))
