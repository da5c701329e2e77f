"""The norms around a block, what they keep in 8 bits and its use, on the GPU against the
FP64 oracle.

Tolerances, derived from the definitions (u = 2^-24, half an FP32 step):
  rstd_post  48 u, as the other norm's (a mean square of at most 32 values a work-item, 6
             wavefront and 16 workgroup additions, halved by the root, a few roundings).
  h          z: 48 u and two products; gate: one; one fused addition: 54 u of
             |alpha x| + |gate z|, and half a step of H's type on the rounded result.
  rstd       48 u and what h's error makes of the mean square: sum |h| E_h / sum h^2.
  y          |rstd w| E_h + |y| (rstd's + 3 u).
  8 bits     the scale within the largest error of its block and 4 u; a code within half a
             step of value / scale and the value's error over the scale.
  d          at most 54 additions for mean(g n), products and the kept values' own
             rounding: 80 u of rstd (|g| + |n| mean|g n|) + |dh|; dx one more product.
  do         p: d's and two products; its mean 54 additions more: 150 u of the formula
             with absolute values throughout.
  sums       as many additions as the longest chain has (rows of a walker, 16 rows side by
             side, workgroups / 32 and 33 in the second kernel), each u on the sum of
             absolute values, and the terms' own 90 u.
"""
import numpy as np
import pytest

import fp32_gemm_08_amd as lib
from oracle import oracle_block as ob
from oracle import oracle_f8 as o8

from gpu_helpers import say
from test_f8_gpu import (HALF, TINY, U, codes, data, f64, need_gpu, put, rounded, strided, tt)  # noqa: F401

pytestmark = pytest.mark.gpu


def check_blocks(q, s, v, err):
    """e4m3 codes with row blocks against values that the kernel holds within `err`."""
    rows, cols = v.shape
    top = np.maximum(o8._block_max(np.abs(v), "row").astype(np.float64), float(o8.FLOOR))
    worst = o8._block_max(err, "row").astype(np.float64) * (1 + 4 * U)
    assert np.all(np.abs(s.T * 448.0 - top) <= worst + 4 * U * top)
    per = o8.spread(s.T.astype(np.float64), "row", rows, cols)
    got, t = o8.decode(q, "e4m3"), v / per
    slack = err / per + 4 * U * np.abs(t)
    assert np.all(np.abs(got - t) <= np.maximum(2.0 ** -4 * (np.abs(t) + slack), 2.0 ** -10) + slack)


def check_i8(q, s, v, err):
    a = np.maximum(np.abs(v).max(axis=1), float(o8.FLOOR))
    assert np.all(np.abs(s * 127.0 - a) <= err.max(axis=1) + 4 * U * a)
    t = v / s[:, None].astype(np.float64)
    assert np.all(np.abs(q - t) <= 0.5 + err / s[:, None] + 4 * U * 127)


def run_norm(rows, cols, t, wt=None, block=True, post=True, gate_rows=None, alpha=1.0, q="e4m3", outs="HYQkrp", eps=1e-6,
             pads=(0, 0, 0), in_place=None, x=None, o=None):
    """gate_rows None: no gate."""
    import torch

    wt = wt or t
    rng = np.random.default_rng(rows * 31 + cols)
    say(f"block norm {rows}x{cols} {t} w {wt} block={block} post={post} gate_rows={gate_rows} alpha={alpha} q={q} "
        f"outs={outs} pads={pads} in_place={in_place}")
    px, po, pq = pads
    x = data(rng, rows, cols, t) if x is None else x
    o = (data(rng, rows, cols, t) if o is None else o) if block else None
    w = rounded(1 + 0.3 * rng.standard_normal(cols), wt)
    wp = rounded(1 + 0.3 * rng.standard_normal(cols), wt) if block and post else None
    gate = rounded(rng.standard_normal((-(-rows // gate_rows), cols)), wt) if block and gate_rows else None
    X = put(strided(rows, cols, tt(t), cols + px)[0], x)
    O = put(strided(rows, cols, tt(t), cols + px)[0], o) if block else None
    G = put(strided(len(gate), cols, tt(wt), cols + px)[0], gate) if gate is not None else None
    W, WP = (None if v is None else torch.from_numpy(v).to(tt(wt)).cuda() for v in (w, wp))
    kb = o8.blocks(cols)
    H, kh = strided(rows, cols, tt(t), cols + po)
    Y, ky = strided(rows, cols, tt(t), cols + po)
    Q, kq = strided(rows, cols, torch.int8 if q == "i8" else tt("e4m3"), cols + pq)
    S, ks = strided(*((1, rows) if q == "i8" else (kb, rows)), torch.float32, rows + pq)
    H8, kh8 = strided(rows, cols, tt("e4m3"), cols + pq)
    O8, ko8 = strided(rows, cols, tt("e4m3"), cols + pq)
    SH, ksh = strided(kb, rows, torch.float32, rows + pq)
    SO, kso = strided(kb, rows, torch.float32, rows + pq)
    rs, rp = (torch.full((rows,), float("nan"), device="cuda") for _ in range(2))
    H = {"x": X, "o": O}.get(in_place, H)
    kw = dict(H=H if "H" in outs else None, Y=Y if "Y" in outs else None, rstd=rs if "r" in outs else None)
    if "Q" in outs:
        kw.update(Q=Q, S=S[0] if q == "i8" else S)
    if "k" in outs:
        kw.update(H8=H8, SH=SH)
        if block:
            kw.update(O8=O8, SO=SO)
    if "p" in outs and wp is not None:
        kw.update(rstd_post=rp)
    lib.block_norm(X, O, W, eps, w_post=WP, gate=G, gate_rows=gate_rows if gate is not None else None, alpha=alpha, **kw)
    torch.cuda.synchronize()
    assert kh() and ky() and kq() and ks() and kh8() and ko8() and ksh() and kso()
    h, y, rstd, rstd_post, z = ob.block_norm(x, o, w, eps, wp, gate, gate_rows, alpha)
    size = np.abs(alpha * x.astype(np.float64))
    if block:
        size = size + np.abs(ob.gate_of_rows(gate, gate_rows, rows) * z)
    eh = 54 * U * size
    rho = (np.abs(h) * eh).sum(axis=1) / np.maximum((h * h).sum(axis=1), 1e-300) + 48 * U
    ey = np.abs(rstd[:, None] * w) * eh + np.abs(y) * (rho[:, None] + 3 * U)
    if "H" in outs:
        assert np.all(np.abs(f64(H) - h) <= eh + HALF[t] * (np.abs(h) + eh) + TINY[t])
    if "Y" in outs:
        assert np.all(np.abs(f64(Y) - y) <= ey + HALF[t] * (np.abs(y) + ey) + TINY[t])
    if "r" in outs:
        assert np.all(np.abs(f64(rs) - rstd) <= rho * rstd)
    if "Q" in outs:
        if q == "i8":
            check_i8(Q.cpu().numpy().astype(np.float64), S[0].cpu().numpy(), y, ey)
        else:
            check_blocks(codes(Q), S.cpu().numpy(), y, ey)
    if "k" in outs:
        check_blocks(codes(H8), SH.cpu().numpy(), h, eh)
        if block:
            c, s = o8.quantize(o, "row", "e4m3")
            assert np.array_equal(codes(O8), c) and np.array_equal(SO.cpu().numpy(), s)
    if "rstd_post" in kw:
        assert np.all(np.abs(f64(rp) - rstd_post) <= 48 * U * rstd_post)


NORM = [(1, 1), (1, 8), (3, 100), (2, 128), (5, 513), (1, 4096), (9, 1000), (4, 2048), (2, 4097), (3, 8192), (2, 9001),
        (2, 16384), (2, 20000), (1, 32768), (300, 264)]


@pytest.mark.parametrize("rows,cols", NORM)
@pytest.mark.parametrize("t", ["bf16", "f32", "fp16"])
def test_norm(rows, cols, t):
    run_norm(rows, cols, t, gate_rows=rows)
    run_norm(rows, cols, t, gate_rows=max(rows // 2, 1), alpha=0.75, q="i8")


@pytest.mark.parametrize("rows,cols", [(1, 100), (40, 130), (7, 1500)])
@pytest.mark.parametrize("kw", [dict(block=False), dict(block=False, alpha=-1.5, q="i8"), dict(post=False),
                                dict(post=False, gate_rows=1), dict(gate_rows=1), dict(gate_rows=3), dict(alpha=0.0),
                                dict(wt="f32", gate_rows=2), dict(wt="f32", post=False, alpha=2.5, q="i8")])
def test_norm_forms(rows, cols, kw):
    run_norm(rows, cols, "bf16", **kw)
    run_norm(rows, cols, "f32", **kw)


@pytest.mark.parametrize("outs", ["H", "Y", "Q", "k", "r", "p", "HQ", "Yr", "Hk"])
@pytest.mark.parametrize("q", ["e4m3", "i8"])
def test_norm_single_outputs(outs, q):
    run_norm(5, 700, "bf16", gate_rows=5, outs=outs, q=q)


@pytest.mark.parametrize("pads", [(8, 8, 8), (1, 0, 3), (0, 5, 16), (16, 3, 1)])
def test_norm_strides(pads):
    for t in ("bf16", "f32"):
        for q in ("e4m3", "i8"):
            run_norm(6, 640, t, wt="f32", gate_rows=2, pads=pads, q=q)


@pytest.mark.parametrize("where", ["x", "o"])
def test_norm_in_place(where):
    run_norm(6, 1100, "bf16", gate_rows=6, in_place=where)
    run_norm(3, 5000, "f32", gate_rows=1, in_place=where)


def test_norm_zero_rows_and_special_values():
    import torch

    rng = np.random.default_rng(1)
    x, o = data(rng, 5, 300), data(rng, 5, 300)
    o[1] = 0.0
    x[2], o[2] = 0.0, 0.0
    for q in ("e4m3", "i8"):
        run_norm(5, 300, "f32", gate_rows=5, x=x, o=o, q=q)
    X, O = torch.from_numpy(x).cuda(), torch.from_numpy(o).cuda()
    X[3, 5], O[4, 7] = float("nan"), float("inf")
    W = torch.ones(300, device="cuda")
    for dtype in (torch.int8, tt("e4m3")):
        H, Q = torch.empty_like(X), torch.zeros(5, 300, dtype=dtype, device="cuda")
        S = torch.empty(5 if dtype == torch.int8 else (3, 5), device="cuda")
        H8, SH = torch.empty(5, 300, dtype=tt("e4m3"), device="cuda"), torch.empty(3, 5, device="cuda")
        lib.block_norm(X, O, W, 1e-6, w_post=W, H=H, Q=Q, S=S, H8=H8, SH=SH)
        v = Q.float() * (S[:, None] if dtype == torch.int8 else S.t().repeat_interleave(128, 1)[:, :300])
        assert bool(torch.isfinite(v[:3]).all()) and bool((v[2] == 0).all())
        assert bool(torch.isnan(v[3]).all()) and bool(torch.isnan(v[4]).any())
        k = H8.float() * SH.t().repeat_interleave(128, 1)[:, :300]
        assert bool(torch.isfinite(k[:3]).all()) and bool(torch.isnan(k[3, :128]).all()) and bool(torch.isfinite(k[3, 128:]).all())


def test_norm_of_large_and_small_values():
    rng = np.random.default_rng(2)
    big, small = ((data(rng, 3, 500) * f).astype(np.float32) for f in (1e15, 1e-15))
    run_norm(3, 500, "f32", x=big, o=big, gate_rows=3)
    run_norm(3, 500, "f32", x=small, o=small, eps=0.0, gate_rows=3, q="i8")


# ------------------------------------------------------------------ backward

def run_bwd(rows, cols, t, wt=None, kept=False, post=True, gate_rows=None, alpha=1.0, dy=True, dh=True, sums=True,
            outs="xo", pads=(0, 0, 0), in_place=()):
    import torch

    wt = wt or t
    rng = np.random.default_rng(rows * 17 + cols)
    say(f"block norm backward {rows}x{cols} {t} w {wt} kept={kept} post={post} gate_rows={gate_rows} alpha={alpha} "
        f"dy={dy} dh={dh} sums={sums} outs={outs} pads={pads} in_place={in_place}")
    pi, po, pk = pads
    h, o, gy, gh = (data(rng, rows, cols, t) for _ in range(4))
    w, wp = (rounded(1 + 0.3 * rng.standard_normal(cols), wt) for _ in range(2))
    gate = rounded(rng.standard_normal((-(-rows // gate_rows), cols)), wt) if gate_rows else None
    rstd, rstd_post = ((1.0 / np.sqrt((v.astype(np.float64) ** 2).mean(axis=1) + 1e-6)).astype(np.float32) for v in (h, o))
    DY, DH = (put(strided(rows, cols, tt(t), cols + pi)[0], v) for v in (gy, gh))
    SH = SO = None
    if kept:
        (qh, sh), (qo, so) = (o8.quantize(v, "row", "e4m3") for v in (h, o))
        h, o = o8.values(qh, sh, "row", "e4m3"), o8.values(qo, so, "row", "e4m3")
        H, O = (put(strided(rows, cols, tt("e4m3"), cols + pk)[0], v) for v in (qh, qo))
        SH, SO = (put(strided(*v.shape, torch.float32, rows + pk)[0], v) for v in (sh, so))
    else:
        H, O = (put(strided(rows, cols, tt(t), cols + pi)[0], v) for v in (h, o))
    W, WP = (torch.from_numpy(v).to(tt(wt)).cuda() for v in (w, wp))
    G = put(strided(len(gate), cols, tt(wt), cols + pi)[0], gate) if gate is not None else None
    RS, RP = torch.from_numpy(rstd).cuda(), torch.from_numpy(rstd_post).cuda()
    DX, kx = strided(rows, cols, tt(t), cols + po)
    DO, ko = strided(rows, cols, tt(t), cols + po)
    for name in in_place:                                 # "xdy": DX is DY, and so on
        at = {"dy": DY, "dh": DH, "h": H, "o": O}[name[1:]]
        DX, DO = (at, DO) if name[0] == "x" else (DX, at)
    dw, kw = strided(1, cols, torch.float32)
    dwp, kwp = strided(1, cols, torch.float32)
    dg, kg = strided(1 if gate is None else len(gate), cols, torch.float32, cols + po)
    need = lib.sgemm_block_norm_bwd_plan(rows, cols, gate_rows or 0)[1]
    ws = torch.full((max(need, 16),), 0xA5, dtype=torch.uint8, device="cuda")
    has_gate = sums and gate is not None
    lib.block_norm_backward(DY if dy else None, H if dy else None, O if post or has_gate else None, W if dy else None,
                            RS if dy else None, DX if "x" in outs else None, DO if "o" in outs else None, SH=SH, SO=SO,
                            w_post=WP if post else None, rstd_post=RP if post else None, gate=G, gate_rows=gate_rows,
                            alpha=alpha, dH=DH if dh else None, dW=dw[0] if sums else None,
                            dW_post=dwp[0] if sums and post else None, dGate=dg if has_gate else None,
                            workspace=ws if sums else None)
    torch.cuda.synchronize()
    assert kx() and ko() and kw() and kwp() and kg()
    e = ob.block_norm_backward(gy if dy else None, gh if dh else None, h, o, w, rstd, wp if post else None, rstd_post, gate,
                               gate_rows, alpha)
    if "x" in outs:
        tol = 82 * U * e["dx_size"]
        assert np.all(np.abs(f64(DX) - e["dx"]) <= tol + HALF[t] * (np.abs(e["dx"]) + tol) + TINY[t])
    if "o" in outs:
        tol = 150 * U * e["do_size"]
        assert np.all(np.abs(f64(DO) - e["do"]) <= tol + HALF[t] * (np.abs(e["do"]) + tol) + TINY[t])
    if sums:
        groups = max(lib.sgemm_block_norm_bwd_plan(rows, cols, 0)[1] // (8 * cols), 1)
        walkers = (need // (4 * cols) - 2 * groups) // 2 if gate_rows and gate_rows < rows else groups
        depth = -(-rows // groups) + 16 + max(groups, walkers) / 32 + 34
        if dy:
            assert np.all(np.abs(f64(dw[0]) - e["dw"]) <= (depth + 6) * U * e["dw_size"])
        else:
            assert bool((dw == 0).all())
        if post:
            assert np.all(np.abs(f64(dwp[0]) - e["dw_post"]) <= (2 * depth + 90) * U * e["dw_post_size"])
        if gate is not None:
            assert np.all(np.abs(f64(dg) - e["dgate"]) <= (depth + 90) * U * e["dgate_size"])


@pytest.mark.parametrize("rows,cols", NORM + [(5000, 72), (3000, 700), (2500, 1030), (1200, 4096)])
@pytest.mark.parametrize("t", ["bf16", "f32", "fp16"])
@pytest.mark.parametrize("kept", [False, True])
def test_bwd(rows, cols, t, kept):
    run_bwd(rows, cols, t, kept=kept, gate_rows=rows, alpha=0.75)
    run_bwd(rows, cols, t, kept=kept, gate_rows=-(-rows // 3))


@pytest.mark.parametrize("gate_rows", [1, 2, 3, 5, 7, 64, 200, 1299, 1300])
@pytest.mark.parametrize("rows,cols", [(1300, 40), (1300, 300), (1300, 1500), (1301, 8000)])
def test_bwd_gates_of_several_rows(rows, cols, gate_rows):
    run_bwd(rows, cols, "bf16", gate_rows=gate_rows, kept=True)


def test_bwd_gates_that_cross_the_walkers():
    # 14 rows of 8 columns for each of 12288 walkers: gates shorter and longer than that, that
    # end inside of a walker's rows
    for gate_rows in (1, 9, 13, 14, 15, 28, 1001, 60000):
        run_bwd(160000, 8, "f32", gate_rows=gate_rows)


@pytest.mark.parametrize("kw", [dict(post=False), dict(post=False, gate_rows=130), dict(post=False, gate_rows=9),
                                dict(dh=False), dict(dy=False), dict(dy=False, gate_rows=11), dict(sums=False),
                                dict(sums=False, gate_rows=3), dict(sums=False, post=False, gate_rows=3), dict(outs="x"),
                                dict(outs="o"), dict(outs="", gate_rows=4), dict(wt="f32", gate_rows=4),
                                dict(pads=(8, 8, 8), gate_rows=4), dict(pads=(1, 3, 5), gate_rows=4),
                                dict(pads=(0, 1, 16), gate_rows=4)])
@pytest.mark.parametrize("kept", [False, True])
def test_bwd_variants(kw, kept):
    run_bwd(130, 800, "bf16", kept=kept, **kw)
    run_bwd(1100, 130, "f32", kept=kept, **kw)


@pytest.mark.parametrize("in_place", [("xdy",), ("xdh",), ("xh",), ("ody",), ("odh",), ("oo",), ("xdy", "oo"),
                                      ("xh", "odh"), ("xdh", "ody")])
def test_bwd_in_place(in_place):
    for rows, cols, t in ((130, 800, "bf16"), (70, 5000, "f32"), (600, 100, "fp16")):
        run_bwd(rows, cols, t, gate_rows=7, in_place=in_place)
        if not {"xh", "oo"} & set(in_place):
            run_bwd(rows, cols, t, gate_rows=7, in_place=in_place, kept=True)


def test_bwd_no_rows():
    import torch

    W, dw, dwp = torch.ones(40, device="cuda"), torch.full((40,), 7.0, device="cuda"), torch.full((40,), 7.0, device="cuda")
    e, r = torch.empty(0, 40, device="cuda"), torch.empty(0, device="cuda")
    dg = torch.full((1, 40), 7.0, device="cuda")
    lib.block_norm_backward(e, e, e, W, r, e, e, w_post=W, rstd_post=r, gate=torch.empty(0, 40, device="cuda"), gate_rows=4,
                            dW=dw, dW_post=dwp, dGate=dg[:0], workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    assert bool((dw == 0).all()) and bool((dwp == 0).all()) and bool((dg == 7).all())


def test_bwd_against_differences_of_the_forward():
    """The gradient of sum(y * v + h * u) by central differences of the FP32 forward kernel, for
    every input.  A difference is off by its own truncation, which FP64 gives, and by the
    rounding of y and h over the step."""
    import torch

    rows, cols, d, alpha, gate_rows = 4, 24, 2.0 ** -7, 0.75, 2
    rng = np.random.default_rng(5)
    v, u = (rng.standard_normal((rows, cols)).astype(np.float32) for _ in range(2))
    at = dict(x=rng.standard_normal((rows, cols)), o=rng.standard_normal((rows, cols)), w=1 + 0.3 * rng.standard_normal(cols),
              wp=1 + 0.3 * rng.standard_normal(cols), gate=rng.standard_normal((2, cols)))
    at = {k: x.astype(np.float32) for k, x in at.items()}

    def exact(p):
        h, y, rstd, rp, z = ob.block_norm(p["x"], p["o"], p["w"], 1e-3, p["wp"], p["gate"], gate_rows, alpha)
        return (y * v + h * u).sum(), np.abs(y * v).sum() + np.abs(h * u).sum()

    def kernel(p):
        t = {k: torch.from_numpy(x).cuda() for k, x in p.items()}
        H, Y = torch.empty_like(t["x"]), torch.empty_like(t["x"])
        lib.block_norm(t["x"], t["o"], t["w"], 1e-3, w_post=t["wp"], gate=t["gate"], alpha=alpha, H=H, Y=Y)
        return float((f64(Y) * v + f64(H) * u).sum())

    t = {k: torch.from_numpy(x).cuda() for k, x in at.items()}
    H, rs, rp = torch.empty_like(t["x"]), torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    lib.block_norm(t["x"], t["o"], t["w"], 1e-3, w_post=t["wp"], gate=t["gate"], alpha=alpha, H=H, rstd=rs, rstd_post=rp)
    got = dict(x=torch.empty_like(H), o=torch.empty_like(H), w=torch.empty(cols, device="cuda"),
               wp=torch.empty(cols, device="cuda"), gate=torch.empty(2, cols, device="cuda"))
    ws = torch.empty(lib.sgemm_block_norm_bwd_plan(rows, cols, gate_rows)[1], dtype=torch.uint8, device="cuda")
    lib.block_norm_backward(torch.from_numpy(v).cuda(), H, t["o"], t["w"], rs, got["x"], got["o"], w_post=t["wp"], rstd_post=rp,
                            gate=t["gate"], alpha=alpha, dH=torch.from_numpy(u).cuda(), dW=got["w"], dW_post=got["wp"],
                            dGate=got["gate"], workspace=ws)
    h, y, rstd, rpost, z = ob.block_norm(at["x"], at["o"], at["w"], 1e-3, at["wp"], at["gate"], gate_rows, alpha)
    e = ob.block_norm_backward(v, u, h, at["o"], at["w"], rstd, at["wp"], rpost, at["gate"], gate_rows, alpha)
    formula = dict(x=e["dx"], o=e["do"], w=e["dw"], wp=e["dw_post"], gate=e["dgate"])
    size = exact(at)[1]
    for name in at:
        g = f64(got[name])
        for i in np.ndindex(*at[name].shape):
            up, down = ({k: x.copy() for k, x in at.items()} for _ in range(2))
            up[name][i] += d
            down[name][i] -= d
            step = float(up[name][i]) - float(down[name][i])
            slope = (exact(up)[0] - exact(down)[0]) / step
            cut = abs(slope - formula[name][i])           # the difference's own truncation
            diff = (kernel(up) - kernel(down)) / step
            assert abs(diff - g[i]) <= cut + 2 * 130 * U * 2 * size / step + 400 * U * size, (name, i)


# ------------------------------------------------------------------ requantisation

@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 128), (1, 129), (2, 127), (3, 5), (128, 128), (127, 255), (129, 257),
                                       (200, 1000), (333, 64), (1000, 1017)])
@pytest.mark.parametrize("fx,fmt", [("e4m3", "e4m3"), ("e5m2", "e4m3"), ("e4m3", "e5m2"), ("e5m2", "e5m2")])
def test_requantize(rows, cols, fx, fmt):
    for pads in ((0, 0, 0), (3, 5, 1), (16, 8, 4)):
        run_requantize(rows, cols, fx, fmt, pads)


def run_requantize(rows, cols, fx, fmt, pads=(0, 0, 0), change=None):
    import torch

    px, pq, ps = pads
    say(f"requantize {rows}x{cols} {fx} -> {fmt} pads={pads}")
    rng = np.random.default_rng(rows * 1000 + cols)
    q, s = o8.quantize(data(rng, rows, cols), "row", fx)
    if change:
        change(q, s)
    X = put(strided(rows, cols, tt(fx), cols + px)[0], q)
    SX = put(strided(*s.shape, torch.float32, rows + ps)[0], s)
    QT, kq = strided(cols, rows, tt(fmt), rows + pq)
    ST, ks = strided(o8.blocks(rows), cols, torch.float32, cols + ps)
    lib.f8_requantize(X, SX, QT, ST)
    torch.cuda.synchronize()
    assert kq() and ks()
    with np.errstate(all="ignore"):
        x = o8.decode(q, fx).astype(np.float32) * o8.spread(s.T, "row", rows, cols)   # one FP32 product
    want, st = o8.quantize(x.T, "row", fmt)
    got = codes(QT)
    nan = np.isnan(o8.decode(want, fmt))
    assert np.array_equal(nan, np.isnan(o8.decode(got, fmt))) and np.array_equal(got[~nan], want[~nan])
    assert np.array_equal(ST.cpu().numpy(), st, equal_nan=True)


def test_requantize_special_values():
    def change(q, s):
        q[3, 5] = 0x7f                                    # NaN
        s[0, 7], s[1, 9] = np.inf, np.nan
        s[2, 11] = 1e-45                                  # a subnormal scale
        q[200:, :] = 0

    run_requantize(300, 400, "e4m3", "e4m3", change=change)
    run_requantize(300, 400, "e5m2", "e5m2", change=change)


# ------------------------------------------------------------------ offsets, streams, refusals

def test_rows_past_32_bit_offsets():
    import torch

    rows, cols, ld = 300, 136, 1 << 23                    # the last rows start past 2^31 elements
    rng = np.random.default_rng(6)
    x, o = data(rng, rows, cols, "bf16"), data(rng, rows, cols, "bf16")

    def far(v=None, dtype=torch.bfloat16, ld=ld):
        t = torch.empty(rows * ld, dtype=dtype, device="cuda").view(rows, ld)[:, :cols]
        return t if v is None else put(t, v)

    X, O, H = far(x), far(o), far()
    H8, O8 = far(dtype=torch.uint8, ld=2 * ld).view(tt("e4m3")), far(dtype=torch.uint8, ld=2 * ld).view(tt("e4m3"))
    W = torch.ones(cols, dtype=torch.bfloat16, device="cuda")
    SH, SO = torch.empty(2, rows, device="cuda"), torch.empty(2, rows, device="cuda")
    rs, rp = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    lib.block_norm(X, O, W, 1e-6, w_post=W, H=H, H8=H8, SH=SH, O8=O8, SO=SO, rstd=rs, rstd_post=rp)
    h, _, rstd, rpost, z = ob.block_norm(x, o, np.ones(cols), 1e-6, np.ones(cols))
    eh = 54 * U * (np.abs(x) + np.abs(z))
    assert np.all(np.abs(f64(H) - h) <= eh + HALF["bf16"] * (np.abs(h) + eh) + TINY["bf16"])
    assert np.array_equal(codes(O8), o8.quantize(o, "row", "e4m3")[0])
    check_blocks(codes(H8), SH.cpu().numpy(), h, eh)
    k = [o8.values(codes(q), s.cpu().numpy(), "row", "e4m3") for q, s in ((H8, SH), (O8, SO))]
    DX, DO = far(), far()
    lib.block_norm_backward(X, H8, O8, W, rs, DX, DO, SH=SH, SO=SO, w_post=W, rstd_post=rp, dH=O)
    e = ob.block_norm_backward(x, o, k[0], k[1], np.ones(cols), f64(rs), np.ones(cols), f64(rp))
    for got, name, f in ((DX, "dx", 82), (DO, "do", 150)):
        tol = f * U * e[name + "_size"]
        assert np.all(np.abs(f64(got) - e[name]) <= tol + HALF["bf16"] * (np.abs(e[name]) + tol) + TINY["bf16"])
    QT, ST = torch.empty(cols, rows, dtype=tt("e4m3"), device="cuda"), torch.empty(3, cols, device="cuda")
    lib.f8_requantize(H8, SH, QT, ST)
    with np.errstate(all="ignore"):
        v = o8.decode(codes(H8), "e4m3").astype(np.float32) * o8.spread(SH.cpu().numpy().T, "row", rows, cols)
    assert np.array_equal(codes(QT), o8.quantize(v.T, "row", "e4m3")[0])


def test_wrappers_refuse_what_does_not_fit():
    import torch

    x, w, e = torch.randn(6, 256, device="cuda"), torch.ones(256, device="cuda"), torch.empty(6, 256, device="cuda")
    r = torch.ones(6, device="cuda")
    q, s = torch.empty(6, 256, dtype=tt("e4m3"), device="cuda"), torch.ones(2, 6, device="cuda")
    lib.block_norm(x, x.clone(), w, H=e, Q=q, S=s)
    for kw, err in ((dict(w_post=w.half()), TypeError), (dict(gate=torch.ones(4, 256, device="cuda")), ValueError),
                    (dict(gate=torch.ones(4, 256, device="cuda"), gate_rows=2), ValueError), (dict(Q=q), ValueError),
                    (dict(Q=q, S=s.t()), ValueError), (dict(Q=q, S=r), TypeError),
                    (dict(Q=q.view(torch.int8), S=s), TypeError), (dict(H8=q), ValueError), (dict(H8=e, SH=s), TypeError),
                    (dict(Y=e[:, :255]), ValueError), (dict(rstd=r[:5]), ValueError), (dict(rstd_post=r), ValueError)):
        with pytest.raises(err):
            lib.block_norm(x, x.clone(), w, **{"H": e, **kw})
    for kw in (dict(Y=x), dict(H=x[:, :255], Y=e[:, :255])):
        with pytest.raises((lib.SgemmError, ValueError)):
            lib.block_norm(x, x.clone(), w, **kw)
    with pytest.raises(ValueError):
        lib.block_norm(x, None, w, w_post=w, H=e)
    with pytest.raises(ValueError):
        lib.block_norm(x, x.clone(), None, Y=e)
    with pytest.raises(TypeError):
        lib.block_norm_backward(x, x, q, w, r, e, None, SO=s, w_post=w, rstd_post=r)   # one of them in 8 bits
    with pytest.raises(ValueError):
        lib.block_norm_backward(x, q, None, w, r, e, None)                             # no scales
    with pytest.raises(ValueError):
        lib.block_norm_backward(x, x, None, w, r, e, None, w_post=w, rstd_post=r)
    with pytest.raises(ValueError):
        lib.block_norm_backward(None, None, None, None, None, e, None)
    with pytest.raises(lib.SgemmError):
        lib.block_norm_backward(x, x, None, w, r, e, None, dW=torch.empty(256, device="cuda"))   # no workspace
    with pytest.raises(ValueError):
        lib.f8_requantize(q, s, q, s)
