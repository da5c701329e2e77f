"""The 8-bit products tile by tile, split by split and at other alignments, and the
norm's rows by 16 to 1024 lanes, against the FP64 oracle.

The tolerances are those of test_f8_gpu.py, where they are derived.  A product
split over k adds one FP32 rounding per part (at most 16): the bound there counts
130 + k-blocks roundings of a whole step each, which covers it.
"""
import numpy as np
import pytest

import fp32_gemm_08_amd as lib
from oracle import oracle_f8 as o8

from gpu_helpers import say
from test_f8_gpu import GUARD, HALF, TINY, U, data, f64, operand, run_bwd, run_norm, run_quantize, rounded, strided, tt

pytestmark = pytest.mark.gpu

SKINNY, ANY, S, N, M, L = 80, 81, 82, 83, 84, 85


@pytest.fixture(scope="module", autouse=True)
def need_gpu():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    assert lib.sgemm_f32_version()


def product(m, n, k, block="tile", ct="bf16", fa="e4m3", fb="e4m3", pad=None, beta=0.0, room=None, offset=0):
    """One product against the oracle; `room`: bytes of workspace (None: those that serve)."""
    import torch

    rng = np.random.default_rng(m + 3 * n + 7 * k)
    pad = -k % 16 if pad is None else pad
    aligned = int((k + pad) % 16 == 0 and offset % 16 == 0)
    if room is None:
        room = lib.sgemm_f8_gemm_workspace(lib.F8_BLOCK[block], m, n, k, aligned)[1]
    say(f"f8 product {m}x{n}x{k} {fa}*{fb} {block} -> {ct} pad={pad} beta={beta} room={room} offset={offset}")
    A, SA, a = operand(rng, m, k, "row", fa, pad, offset)
    B, SB, b = operand(rng, n, k, block, fb, pad, offset)
    C, kept = strided(m, n, tt(ct), n + 5)
    c = rounded(rng.standard_normal((m, n)) * 10, ct)
    C.copy_(torch.from_numpy(c))
    W = torch.full((room + 64,), GUARD, dtype=torch.uint8, device="cuda")
    lib.f8_gemm(A, SA, B, SB, C, beta=beta, b_scale=block, workspace=W[:room] if room else None)
    torch.cuda.synchronize()
    assert kept(), "written outside C"
    assert bool((W[room:] == GUARD).all()), "written past the workspace"
    D, size = o8.gemm_f8(a, b, 1.0, beta, c)
    tol = size * 2 * U * (130 + o8.blocks(k)) + 4 * U * (np.abs(D) + abs(beta) * np.abs(c))
    if ct != "f32":
        tol = tol + size * 7 * 2.0 ** -13
    tol = tol + HALF[ct] * (np.abs(D) + tol) + TINY[ct]
    got = f64(C)
    if ct == "fp16":
        # what rounds past the largest fp16 value is infinite; it is checked here and then set to D
        over = np.abs(D) - tol >= 65520
        assert np.all(got[over] == np.copysign(np.inf, D[over]))
        got = np.where(over | (np.isinf(got) & (np.abs(D) + tol >= 65520)), D, got)
    assert np.all(np.abs(got - D) <= tol), f"max {np.max(np.abs(got - D) / tol):.3g} of the bound"
    if ct != "f32":
        assert np.linalg.norm(got - D) <= HALF[ct] * np.linalg.norm(D) + 2.0 ** -12 * np.linalg.norm(D - beta * c)
    return C


def plan(m, n, k, block="tile", aligned=1):
    st, kid, _, _, splits, nbytes = lib.sgemm_f8_gemm_plan(lib.F8_BLOCK[block], m, n, k, aligned)
    assert st == 0
    return kid, splits, nbytes


# shapes that the plan gives to each tile, ragged in every dimension
TILES = [(S, 1, 1000, 1017, 640), (S, 1, 65, 70, 100), (N, 1, 500, 4000, 300), (N, 1, 257, 5401, 129),
         (M, 1, 2000, 2040, 272), (M, 1, 1025, 4000, 150), (L, 1, 2900, 3100, 160), (L, 1, 3333, 3000, 1050)]


@pytest.mark.parametrize("kid,splits,m,n,k", TILES)
@pytest.mark.parametrize("block", ["tile", "row"])
@pytest.mark.parametrize("ct", ["bf16", "f32"])
def test_tiles(kid, splits, m, n, k, block, ct):
    assert plan(m, n, k, block)[:2] == (kid, splits)
    product(m, n, k, block, ct)


@pytest.mark.parametrize("k", [1, 15, 16, 17, 112, 127, 128, 129, 256, 383])
@pytest.mark.parametrize("m,n", [(70, 90), (300, 9000), (2040, 2040), (3000, 3000)])
def test_last_values_of_rows(m, n, k):
    """Rows end anywhere in a stage; the padding behind them holds NaN codes."""
    product(m, n, k)
    product(m, n, k, ct="f32", block="row", fa="e5m2", pad=16 + -k % 16)


def test_every_tile_and_every_kind_is_planned():
    assert {plan(*t[2:])[0] for t in TILES} == {S, N, M, L}
    assert plan(64, 500, 500)[0] == SKINNY and plan(16, 500, 500, aligned=0)[0] == SKINNY
    assert plan(17, 500, 500, aligned=0)[0] == ANY and plan(65, 1, 500)[0] == ANY


@pytest.mark.parametrize("m,n,k", [(128, 512, 8000), (256, 256, 4096), (100, 600, 16400), (1000, 1000, 8100)])
@pytest.mark.parametrize("block,ct,beta", [("tile", "bf16", 0.0), ("row", "f32", 1.0), ("tile", "fp16", -0.5)])
def test_splits(m, n, k, block, ct, beta):
    kid, splits, nbytes = plan(m, n, k, block)
    assert splits > 1 and nbytes == 4 * splits * m * n
    a = product(m, n, k, block, ct, beta=beta)
    import torch

    assert torch.equal(a, product(m, n, k, block, ct, beta=beta))       # the same order every time
    product(m, n, k, block, ct, beta=beta, room=nbytes - 1)             # a part less, or none
    product(m, n, k, block, ct, beta=beta, room=0)


@pytest.mark.parametrize("m,n,k", [(2048, 2048, 2047), (600, 4100, 4095), (1500, 1300, 3001)])
@pytest.mark.parametrize("block,ct", [("tile", "bf16"), ("row", "f32")])
def test_operands_laid_out_anew(m, n, k, block, ct):
    nbytes = lib.sgemm_f8_gemm_workspace(lib.F8_BLOCK[block], m, n, k, 0)[1]
    assert nbytes >= (m + n) * -(-k // 128) * 128
    product(m, n, k, block, ct, pad=0)
    product(m, n, k, block, ct, pad=0, offset=3, room=nbytes - 1)       # too little: through registers
    product(m, n, k, block, ct, pad=1, offset=5)


@pytest.mark.parametrize("m", [1, 2, 15, 16, 17, 31, 33, 48, 63, 64])
@pytest.mark.parametrize("n", [16, 500, 8200, 16500])
def test_few_rows(m, n):
    product(m, n, 400)
    product(m, n, 1400, ct="f32", fa="e5m2")
    product(m, n, 333, pad=0, offset=1)
    if n <= 500:
        product(m, n, 2100, block="row", ct="fp16")


@pytest.mark.parametrize("m,n,k", [(300, 1, 500), (5000, 1, 129), (2, 1, 70), (70, 2, 300)])
def test_one_column(m, n, k):
    product(m, n, k)
    product(m, n, k, block="row", ct="f32", pad=0)


@pytest.mark.parametrize("m,n", [(300, 300), (1100, 130)])
def test_rows_4_mb_apart(m, n):
    """The largest leading dimension of the fast kernels, and one beyond it."""
    import torch

    rng = np.random.default_rng(4)
    k = 272
    qa, sa = o8.quantize(data(rng, m, k), "row", "e4m3")
    qb, sb = o8.quantize(data(rng, n, k), "tile", "e4m3")
    D, size = o8.gemm_f8(o8.values(qa, sa, "row", "e4m3"), o8.values(qb, sb, "tile", "e4m3"))
    tol = size * (2 * U * 133 + 7 * 2.0 ** -13) + 4 * U * np.abs(D)
    e4 = torch.float8_e4m3fn
    for ld in (1 << 22, (1 << 22) + 16):
        A = torch.empty(m * ld, dtype=torch.uint8, device="cuda").view(m, ld)[:, :k]
        A.copy_(torch.from_numpy(qa))
        B = torch.empty(n * ld, dtype=torch.uint8, device="cuda").view(n, ld)[:, :k]
        B.copy_(torch.from_numpy(qb))
        C = torch.empty(m, n, dtype=torch.bfloat16, device="cuda")
        lib.f8_gemm(A.view(e4), torch.from_numpy(sa).cuda(), B.view(e4), torch.from_numpy(sb).cuda(), C)
        assert np.all(np.abs(f64(C) - D) <= tol + HALF["bf16"] * (np.abs(D) + tol) + TINY["bf16"])
        del A, B


def test_nan_and_infinity_stay_in_their_rows():
    import torch

    for m, n, k in ((1000, 1000, 300), (500, 4000, 300), (2000, 2040, 300), (2900, 3100, 300)):
        rng = np.random.default_rng(m)
        A, SA, _ = operand(rng, m, k, "row", "e4m3", 4)
        B, SB, _ = operand(rng, n, k, "tile", "e4m3", 4)
        A.view(torch.uint8)[m - 1, 299] = 0x7f
        SA[1, 3] = float("nan")
        SA[2, 7] = float("inf")
        A.view(torch.uint8)[7, 256:] = 0                  # infinity times zeros
        C = torch.zeros(m, n, dtype=torch.bfloat16, device="cuda")
        lib.f8_gemm(A, SA, B, SB, C)
        bad = torch.isnan(C)
        rows = torch.zeros(m, dtype=torch.bool, device="cuda")
        rows[[3, 7, m - 1]] = True
        assert bool(bad[rows].all()) and not bool(bad[~rows].any())


# ------------------------------------------------------------------ rows of the norm

ROWS = [(1, 5), (2, 7), (37, 100), (1000, 24), (17, 128), (33, 129), (13, 256), (9, 257), (130, 300), (5, 511), (6, 512),
        (2050, 513), (3, 1023), (70, 1024), (5, 1025), (3, 2047), (2, 2049), (800, 9), (4, 32761)]


@pytest.mark.parametrize("rows,cols", ROWS)
@pytest.mark.parametrize("t,wt", [("bf16", "bf16"), ("f32", "f32"), ("fp16", "f32")])
def test_norm_rows(rows, cols, t, wt):
    run_norm(rows, cols, t, wt=wt, pads=(0, 3, 1))
    run_bwd(rows, cols, t, wt=wt, pads=(1, 0))


@pytest.mark.parametrize("cols", [3, 9, 100, 301, 1017, 4099])
def test_norm_in_place_of_ragged_rows(cols):
    for t in ("bf16", "f32"):
        run_norm(50, cols, t, in_place="x")
        for where in ("dy", "h", "dh"):
            run_bwd(50, cols, t, in_place=where)


@pytest.mark.parametrize("cols", [1, 2, 3, 4, 5, 6, 7, 9, 15, 130, 133])
def test_quantize_short_pieces(cols):
    for t in ("bf16", "f32"):
        run_quantize(131, cols, "row", t, "e4m3", pads=(1, 3, 5, 1))
        run_quantize(cols, 131, "tile", t, "e5m2", pads=(3, 1, 1, 0))
