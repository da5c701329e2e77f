"""Products of 8-bit integers and the quantisation of rows on the GPU against the FP64 oracle.

The integer sums are exact.  D = alpha * ((float(s) * sa) * sb): four roundings of u = 2^-24
on the product, one more with beta on |D| + |beta c|, and half a step of C's type.  Quantised
integers are equal to the definition's; scales are one correctly rounded division."""
import numpy as np
import pytest

import fp32_gemm_08_amd as lib
from oracle import oracle_block as ob

from gpu_helpers import say
from test_f8_gpu import GUARD, HALF, TINY, U, data, f64, need_gpu, put, rounded, strided, tt  # noqa: F401

pytestmark = pytest.mark.gpu


def put_i8(t, q):
    import torch

    t.copy_(torch.from_numpy(np.ascontiguousarray(q)))
    return t


def operand(rng, rows, cols, pad, offset=0, extremes=False):
    """int8 values and scales that differ by row, on the device and on the host."""
    import torch

    q = rng.integers(-128, 128, (rows, cols)).astype(np.int8)
    if extremes:
        q = np.where(rng.random((rows, 1)) < 0.5, -128, 127).astype(np.int8) * np.ones((1, cols), np.int8)
    s = np.exp(rng.standard_normal(rows)).astype(np.float32)
    t, _ = strided(rows, cols, torch.int8, cols + pad, offset)
    if pad:
        torch.as_strided(t, (rows, cols + pad), (cols + pad, 1)).fill_(77)     # bytes past K must not count
    return put_i8(t, q), torch.from_numpy(s).cuda(), q, s


def run_gemm(M, N, K, ct="bf16", alpha=1.0, beta=0.0, pad=None, offset=0, ldc_pad=0, ws=True, stream=None, extremes=False):
    import torch

    rng = np.random.default_rng(M * 7 + N * 3 + K)
    pad = -K % 16 if pad is None else pad
    say(f"i8 gemm {M}x{N}x{K} -> {ct} alpha={alpha} beta={beta} pad={pad} offset={offset} ws={ws}")
    A, SA, a, sa = operand(rng, M, K, pad, offset, extremes)
    B, SB, b, sb = operand(rng, N, K, pad, offset, extremes)
    C, kc = strided(M, N, tt(ct), N + ldc_pad)
    c = rounded(rng.standard_normal((M, N)) * 1000, ct)
    if beta != 0.0:
        put(C, c)
    n = max(lib.sgemm_i8_gemm_workspace(M, N, K, al)[1] for al in (0, 1)) if ws is True else int(ws)
    W = torch.full((n,), GUARD, dtype=torch.uint8, device="cuda") if n else None
    if stream is not None:
        torch.cuda.synchronize()
    lib.i8_gemm(A, SA, B, SB, C, alpha=alpha, beta=beta, workspace=W, stream=stream)
    torch.cuda.synchronize()
    assert kc(), "written outside C"
    D, s = ob.gemm_i8(a, sa, b, sb, alpha, beta, c)
    got, p = f64(C), np.abs(alpha * s * sa.astype(np.float64)[:, None] * sb)
    tol = 4.01 * U * p + 1.01 * U * (np.abs(D) + abs(beta) * np.abs(c))
    tol = tol + HALF[ct] * (np.abs(D) + tol) + TINY[ct]
    if ct == "fp16":
        # what rounds past the largest fp16 value is infinite; it is checked here and then set to D
        over = np.abs(D) - tol >= 65520
        assert np.all(got[over] == np.copysign(np.inf, D[over]))
        got = np.where(over | (np.isinf(got) & (np.abs(D) + tol >= 65520)), D, got)
    far = np.abs(got - D)
    assert np.all(far <= tol), f"max {np.max(far / tol):.3g} of the bound at {np.unravel_index(np.argmax(far / tol), far.shape)}"
    return f64(C)


SHAPES = [(1, 1, 1), (1, 16, 128), (1, 200, 300), (2, 5, 127), (3, 129, 129), (16, 64, 256), (17, 250, 1000),
          (33, 128, 640), (64, 192, 384), (65, 65, 65), (100, 130, 2000), (128, 128, 128), (129, 257, 255),
          (200, 384, 512), (256, 256, 1024), (300, 520, 1040), (513, 300, 144)]


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_gemm_aligned(M, N, K):
    run_gemm(M, N, K, ct="f32")


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("offset", [0, 1, 3])
def test_gemm_any_alignment(M, N, K, offset):
    run_gemm(M, N, K, pad=1, offset=offset, ct="bf16")
    run_gemm(M, N, K, pad=0, offset=offset, ct="f32")


@pytest.mark.parametrize("M,N,K", [(1100, 1090, 300), (1030, 1030, 129), (2100, 600, 1), (1024, 1024, 512), (1020, 1000, 511),
                                   (70, 4000, 640), (33, 900, 100)])
def test_gemm_any_alignment_without_a_workspace(M, N, K):
    assert (-(-M // 64) * -(-N // 64) > 256) == ((M, N) in ((1100, 1090), (1030, 1030), (2100, 600)))   # both of its forms
    run_gemm(M, N, K, pad=1, offset=1, ws=0)


@pytest.mark.parametrize("ct", ["f32", "bf16", "fp16"])
@pytest.mark.parametrize("M,N,K", [(1, 70, 200), (5, 70, 200), (40, 100, 300), (150, 200, 272), (300, 300, 400)])
def test_gemm_types(ct, M, N, K):
    run_gemm(M, N, K, ct, alpha=0.75, beta=-1.5, ldc_pad=8)
    run_gemm(M, N, K, ct, alpha=-2.0 ** -8, beta=0.0, ldc_pad=3, pad=5)


@pytest.mark.parametrize("M,N,K", [(1, 4096, 4096), (4, 1000, 8192), (20, 512, 4096), (48, 2048, 2064), (64, 640, 7000),
                                   (64, 128, 16384), (96, 384, 16384), (512, 1024, 1024), (640, 768, 512), (1000, 1017, 999),
                                   (1024, 2048, 640), (2048, 1536, 384), (1100, 1300, 128)])
def test_gemm_larger_and_the_same_with_any_workspace(M, N, K):
    a = run_gemm(M, N, K)
    for ws in (0, 16, 1 << 20):
        assert np.array_equal(a, run_gemm(M, N, K, ws=ws))
    run_gemm(M, N, K, ct="f32", beta=1.0)
    run_gemm(M, N, K, ct="f32", pad=3, offset=1)


# (M, N, K, kernel, splits or 1): every kernel with k that ends within 16 bytes, within a k-block and
# on its end, one and two k-blocks, splits of unequal length, and edges in both directions
KERNELS = [(16, 1000, 16384, 90, 4), (3, 500, 12345, 90, 8), (9, 17000, 200, 90, 1), (31, 1000, 300, 90, 1),
           (32, 600, 8192, 90, 8), (25, 4090, 1111, 90, 1), (32, 4100, 200, 92, 1), (200, 200, 3000, 92, 4),
           (33, 1000, 8205, 92, 8), (700, 700, 128, 92, 1), (1000, 999, 129, 92, 1), (510, 4000, 4097, 93, 1),
           (500, 4090, 4080, 93, 1), (1000, 4000, 2049, 94, 1), (1010, 4090, 1920, 94, 1), (2047, 8100, 1000, 95, 1),
           (2040, 8190, 1040, 95, 1), (8100, 8000, 144, 95, 1)]


@pytest.mark.parametrize("M,N,K,kid,splits", KERNELS)
def test_gemm_every_kernel(M, N, K, kid, splits):
    plan = lib.sgemm_i8_gemm_plan(M, N, K, 1)
    assert plan[1] == kid and (plan[4] > 1) == (splits > 1), plan
    run_gemm(M, N, K)
    run_gemm(M, N, K, ct="f32", beta=-0.5, ldc_pad=5)


@pytest.mark.parametrize("M,N", [(1, 40), (20, 70), (70, 130), (300, 260)])
def test_gemm_largest_sums(M, N):
    # -128 times -128 in every place of the longest k: 131071 * 2^14, 16384 below 2^31
    run_gemm(M, N, 131071, ct="f32", extremes=True, pad=1)
    run_gemm(M, N, 131056, ct="f32", extremes=True)


def test_gemm_product_free():
    import torch

    A, B = (torch.zeros(r, 16, dtype=torch.int8, device="cuda")[:, :0] for r in (5, 7))
    SA, SB = torch.full((5,), float("nan"), device="cuda"), torch.ones(7, device="cuda")
    for ct in ("f32", "bf16", "fp16"):
        C = torch.full((5, 7), float("nan"), dtype=tt(ct), device="cuda")
        lib.i8_gemm(A, SA, B, SB, C)
        assert torch.all(C == 0)
        C.fill_(3.0)
        lib.i8_gemm(A, SA, B, SB, C, beta=-0.5)
        assert torch.all(C == -1.5)
    A, B = (torch.zeros(r, 200, dtype=torch.int8, device="cuda") for r in (5, 7))
    C = torch.full((5, 7), 3.0, device="cuda")
    lib.i8_gemm(A, SA, B, SB, C, alpha=0.0, beta=2.0)
    assert torch.all(C == 6)


def test_gemm_old_c_is_not_read_at_beta_zero_and_nan_stays_in_its_row():
    import torch

    for M, N, K in ((3, 70, 300), (40, 90, 304), (80, 90, 300), (300, 300, 320)):
        rng = np.random.default_rng(M)
        A, SA, _, _ = operand(rng, M, K, 4)
        B, SB, _, _ = operand(rng, N, K, 4)
        SA[1] = float("nan")
        SB[2] = float("inf")
        C = torch.full((M, N), float("nan"), device="cuda")
        lib.i8_gemm(A, SA, B, SB, C)
        bad = ~torch.isfinite(C)
        want = torch.zeros(M, N, dtype=torch.bool, device="cuda")
        want[1], want[:, 2] = True, True
        assert torch.equal(bad, want)


# ------------------------------------------------------------------ quantisation of rows

def run_quantize(rows, cols, xt, pads=(0, 0), x=None):
    import torch

    px, pq = pads
    say(f"i8 quantize {rows}x{cols} {xt} pads={pads}")
    x = data(np.random.default_rng(rows * 1000 + cols), rows, cols, xt) if x is None else x
    X = put(strided(rows, cols, tt(xt), cols + px)[0], x)
    Q, kq = strided(rows, cols, torch.int8, cols + pq)
    S, ks = strided(1, rows, torch.float32)
    lib.i8_quantize(X, Q, S[0])
    torch.cuda.synchronize()
    assert kq() and ks()
    q, s = ob.quantize_rows_i8(x)
    assert np.array_equal(Q.cpu().numpy(), q)
    assert np.array_equal(S[0].cpu().numpy(), s, equal_nan=True)


@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 8), (3, 100), (2, 128), (5, 513), (1, 4096), (9, 1000), (4, 2048), (2, 4097),
                                       (3, 8192), (2, 9001), (2, 16384), (2, 20000), (1, 32768), (300, 264), (2, 32769),
                                       (3, 70001), (1, 131071)])
@pytest.mark.parametrize("xt", ["bf16", "f32", "fp16"])
def test_quantize(rows, cols, xt):
    run_quantize(rows, cols, xt)
    run_quantize(rows, cols, xt, pads=(3, 5))


def test_quantize_middles_between_integers():
    # values that lie on the middle between two integers, and the nearest FP32 values on both
    # sides of it, for largest values that are no powers of two
    rng = np.random.default_rng(3)
    a = np.concatenate([[127.0, 254.0, 1.0], np.exp(rng.uniform(-20, 20, 61))]).astype(np.float32)
    i = np.arange(-127, 127) + 0.5
    x = (i[None, :] * a[:, None].astype(np.float64) / 127.0).astype(np.float32)
    x = np.concatenate([a[:, None], x, np.nextafter(x, np.float32(np.inf)), np.nextafter(x, np.float32(-np.inf))], axis=1)
    assert np.all(np.abs(x).max(axis=1) == a)
    run_quantize(*x.shape, "f32", x=x)
    run_quantize(*x.shape, "bf16", x=rounded(x, "bf16"))


def test_quantize_special_values():
    x = data(np.random.default_rng(9), 8, 400)
    x[0, 3], x[1, 300], x[2, 10] = np.nan, np.inf, -np.inf
    x[3] = 0.0
    x[4] = 1e-38                                          # far below the floor
    x[5, 7] = np.float32(3e38)
    x[6] = -0.0
    x[7] = np.float32(2.0 ** -89)
    run_quantize(8, 400, "f32", x=x)


# ------------------------------------------------------------------ offsets, streams, refusals

def test_rows_past_32_bit_offsets():
    import torch

    M, N, K, ld = 300, 160, 160, 1 << 24
    rng = np.random.default_rng(4)
    B, SB, b, sb = operand(rng, N, K, 0)
    for pad in (0, 1):                                    # aligned rows, and rows that start at any byte
        a = rng.integers(-128, 128, (M, K)).astype(np.int8)
        sa = np.exp(rng.standard_normal(M)).astype(np.float32)
        A = torch.empty(M * (ld + pad), dtype=torch.int8, device="cuda").view(M, ld + pad)[:, :K]
        put_i8(A, a)
        C = torch.empty(M * (ld // 2), dtype=torch.bfloat16, device="cuda").view(M, ld // 2)[:, :N]
        lib.i8_gemm(A, torch.from_numpy(sa).cuda(), B, SB, C)
        D, _ = ob.gemm_i8(a, sa, b, sb)
        assert np.all(np.abs(f64(C) - D) <= (5 * U + HALF["bf16"] * (1 + 5 * U)) * np.abs(D) + TINY["bf16"])
    x = data(rng, M, K, "bf16")
    X = torch.empty(M * (ld // 2), dtype=torch.bfloat16, device="cuda").view(M, ld // 2)[:, :K]
    Q, S = torch.empty(M * ld, dtype=torch.int8, device="cuda").view(M, ld)[:, :K], torch.empty(M, device="cuda")
    lib.i8_quantize(put(X, x), Q, S)
    q, s = ob.quantize_rows_i8(x)
    assert np.array_equal(Q.cpu().numpy(), q) and np.array_equal(S.cpu().numpy(), s)


def test_another_stream():
    import torch

    s = torch.cuda.Stream()
    for shape in ((1, 300, 528), (40, 300, 520), (200, 300, 520)):
        run_gemm(*shape, stream=s)


def test_wrappers_refuse_what_does_not_fit():
    import torch

    q, s, c = torch.ones(4, 256, dtype=torch.int8, device="cuda"), torch.ones(4, device="cuda"), torch.empty(4, 4, device="cuda")
    lib.i8_gemm(q, s, q, s, c)
    assert bool((c == 256).all())
    with pytest.raises(TypeError):
        lib.i8_gemm(q.view(torch.uint8), s, q, s, c)
    with pytest.raises(ValueError):
        lib.i8_gemm(q, s[:3], q, s, c)
    with pytest.raises(ValueError):
        lib.i8_gemm(q, s, q[:, :128], s, c)
    with pytest.raises(ValueError):
        lib.i8_gemm(q, s, q, s, c[:, :3])
    with pytest.raises(lib.SgemmError) as e:
        lib.i8_gemm(q, s, q, s, c, workspace=c.view(-1))
    assert e.value.status == 2
    with pytest.raises(lib.SgemmError) as e:
        z = torch.zeros(1, lib.I8_MAX_K + 1, dtype=torch.int8, device="cuda")
        lib.i8_gemm(z, s[:1], z.clone(), s[1:2], c[:1, :1])
    assert e.value.status == 1
    x = torch.randn(4, 256, device="cuda")
    with pytest.raises(TypeError):
        lib.i8_quantize(x.double(), q, s)
    with pytest.raises(ValueError):
        lib.i8_quantize(x, q[:, :255], s)
    with pytest.raises(ValueError):
        lib.i8_quantize(x, q, s[:3])
    with pytest.raises(TypeError):
        lib.i8_quantize(x, q.float(), s)
