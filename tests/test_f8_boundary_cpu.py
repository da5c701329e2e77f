"""The 8-bit family's C ABI without a GPU: declared symbols, refusals, quick
returns and the planning queries (fake addresses; no call reaches a launch)."""
import ctypes
import os
import re

import pytest

import fp32_gemm_08_amd as lib
from fp32_gemm_08_amd import f8

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, INVALID, ALIAS = 0, 1, 2
P = {name: (i + 1) << 40 for i, name in enumerate("A SA B SB C W X Q S QT ST R H Y RS DY DH DX DW".split())}


@pytest.fixture(scope="module", autouse=True)
def built():
    if not os.path.exists(lib.LIB_PATH):
        pytest.skip("libsgemm_f32.so not built")


def test_exports_every_declared_symbol():
    text = open(os.path.join(ROOT, "include", "sgemm_f8.h"), encoding="utf-8").read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    declared = sorted(set(re.findall(r"\b(sgemm_f8_\w+)\s*\(", text)))
    assert declared == sorted(f8.F8_EXPORTS)
    so = ctypes.CDLL(lib.LIB_PATH)
    for name in declared:
        assert hasattr(so, name), name


def gemm(fa=1, fb=1, block=1, ct=2, M=64, N=256, K=384, alpha=1.0, beta=0.0, W=0, wb=0, **kw):
    a = dict(A=P["A"], lda=K, SA=P["SA"], ldsa=max(M, 1), B=P["B"], ldb=K, SB=P["SB"],
             ldsb=max(N if block == 0 else -(-K // 128), 1), C=P["C"], ldc=max(N, 1))
    a.update(kw)
    return lib.sgemm_f8_gemm(fa, fb, block, ct, M, N, K, alpha, a["A"], a["lda"], a["SA"], a["ldsa"], a["B"],
                             a["ldb"], a["SB"], a["ldsb"], beta, a["C"], a["ldc"], W, wb, 0)


@pytest.mark.parametrize("kw", [
    dict(fa=0), dict(fb=3), dict(block=2), dict(block=-1), dict(ct=3), dict(ct=-1), dict(M=-1), dict(N=1 << 31),
    dict(K=-1), dict(lda=383), dict(ldb=383), dict(ldc=255), dict(ldsa=63), dict(ldsb=2), dict(block=0, ldsb=255),
    dict(A=0), dict(SA=0), dict(B=0), dict(SB=0), dict(C=0), dict(SA=P["SA"] + 2), dict(SB=P["SB"] + 1),
    dict(C=P["C"] + 1), dict(ct=0, C=P["C"] + 2), dict(wb=-1), dict(W=P["W"] + 8, wb=64),
    dict(lda=1 << 62), dict(M=1 << 30, N=1 << 30, ldc=1 << 30, ldsa=1 << 30),
    dict(K=0, lda=0), dict(alpha=0.0, beta=2.0, C=0)])
def test_gemm_refusals(kw):
    assert gemm(**kw) == INVALID


@pytest.mark.parametrize("kw", [dict(C=P["A"] + 8), dict(C=P["B"]), dict(C=P["SA"]), dict(C=P["SB"] + 4),
                                dict(W=P["A"], wb=64), dict(W=P["B"], wb=64), dict(W=P["C"], wb=64),
                                dict(W=P["C"] - 64, wb=80), dict(W=P["SB"], wb=16)])
def test_gemm_alias(kw):
    assert gemm(**kw) == ALIAS


def test_gemm_quick_returns():
    assert gemm(M=0) == OK and gemm(N=0) == OK and gemm(M=0, A=0, B=0, C=0, SA=0, SB=0) == OK
    assert gemm(alpha=0.0, beta=1.0, A=0, B=0, SA=0, SB=0) == OK
    assert gemm(K=0, lda=1, ldb=1, ldsb=1, beta=1.0, A=0, B=0) == OK


def test_gemm_plan():
    for block in (0, 1):
        for M, N, K in ((1, 1, 1), (1, 4096, 4096), (48, 16384, 4096), (100, 300, 20000), (512, 4096, 4096),
                        (8192, 8192, 8192), (1000, 1017, 999)):
            for al in (0, 1):
                st, kid, tm, tn, sp, nb = lib.sgemm_f8_gemm_plan(block, M, N, K, al)
                assert st == OK and kid >= 80 and tm >= 1 and tn >= 1 and sp >= 1
                assert (nb == 0) == (sp == 1) and (sp == 1 or nb >= 4 * sp * M * N)
    assert lib.sgemm_f8_gemm_plan(1, 0, 5, 5)[1] == 0 and lib.sgemm_f8_gemm_plan(1, 5, 5, 0)[1] == 0
    assert lib.sgemm_f8_gemm_plan(2, 5, 5, 5)[0] == INVALID
    assert lib.sgemm_f8_gemm_plan(1, -5, 5, 5)[0] == INVALID
    assert lib.sgemm_f8_gemm_plan(1, 5, 5, 5, 2)[0] == INVALID


def quant(block=0, fmt=1, xt=2, rows=200, cols=300, **kw):
    rb, cb = -(-rows // 128), -(-cols // 128)
    a = dict(X=P["X"], ldx=max(cols, 1), Q=P["Q"], ldq=max(cols, 1), S=P["S"], lds=max(rows if block == 0 else cb, 1),
             QT=P["QT"], ldqt=max(rows, 1), ST=P["ST"], ldst=max(cols if block == 0 else rb, 1))
    a.update(kw)
    return lib.sgemm_f8_quantize(block, fmt, xt, rows, cols, *(a[k] for k in
                                 ("X", "ldx", "Q", "ldq", "S", "lds", "QT", "ldqt", "ST", "ldst")), 0)


@pytest.mark.parametrize("kw", [dict(block=2), dict(fmt=0), dict(fmt=3), dict(xt=3), dict(rows=-1), dict(cols=1 << 31),
                                dict(ldx=299), dict(ldq=299), dict(lds=199), dict(ldqt=199), dict(ldst=299),
                                dict(block=1, lds=2), dict(block=1, ldst=1), dict(X=0), dict(S=0), dict(ST=0),
                                dict(X=P["X"] + 1), dict(S=P["S"] + 2), dict(xt=0, X=P["X"] + 2)])
def test_quantize_refusals(kw):
    assert quant(**kw) == INVALID


@pytest.mark.parametrize("kw", [dict(Q=P["X"]), dict(S=P["X"] + 4), dict(QT=P["X"] + 64), dict(ST=P["Q"]),
                                dict(QT=P["Q"] + 100), dict(ST=P["S"])])
def test_quantize_alias(kw):
    assert quant(**kw) == ALIAS


def test_quantize_quick_returns():
    assert quant(rows=0, X=0) == OK and quant(cols=0, X=0) == OK
    assert quant(Q=0, QT=0, X=0) == OK


def norm(t=2, wt=2, rows=7, cols=300, eps=1e-6, **kw):
    ld = max(cols, 1)
    a = dict(X=P["X"], ldx=ld, R=P["R"], ldr=ld, W=P["W"], H=P["H"], ldh=ld, Y=P["Y"], ldy=ld, Q=P["Q"], ldq=ld,
             S=P["S"], lds=max(rows, 1), rstd=P["RS"])
    a.update(kw)
    return lib.sgemm_f8_rmsnorm(t, wt, rows, cols, a["X"], a["ldx"], a["R"], a["ldr"], a["W"], eps, a["H"], a["ldh"],
                                a["Y"], a["ldy"], a["Q"], a["ldq"], a["S"], a["lds"], a["rstd"], 0)


@pytest.mark.parametrize("kw", [dict(t=3), dict(wt=1), dict(t=0, wt=2), dict(rows=-1), dict(cols=-1),
                                dict(cols=lib.RMSNORM_MAX_COLS + 1), dict(eps=-1.0), dict(eps=float("nan")),
                                dict(eps=float("inf")), dict(ldx=299), dict(ldr=299), dict(ldh=299), dict(ldy=299),
                                dict(ldq=299), dict(lds=6), dict(X=0), dict(W=0), dict(S=0), dict(X=P["X"] + 1),
                                dict(R=P["R"] + 1), dict(rstd=P["RS"] + 2), dict(wt=0, W=P["W"] + 2),
                                dict(rows=1 << 30)])
def test_norm_refusals(kw):
    assert norm(**kw) == INVALID


@pytest.mark.parametrize("kw", [dict(Y=P["X"]), dict(H=P["X"] + 2), dict(H=P["R"] + 600), dict(Q=P["X"]),
                                dict(H=P["X"], ldh=301), dict(rstd=P["W"]), dict(H=P["Y"]), dict(S=P["Q"] + 4),
                                dict(H=P["W"])])
def test_norm_alias(kw):
    assert norm(**kw) == ALIAS


def test_norm_quick_returns():
    assert norm(rows=0, X=0, W=0) == OK and norm(cols=0, X=0) == OK
    assert norm(H=0, Y=0, Q=0, rstd=0, X=0) == OK


def bwd(t=2, wt=2, rows=7, cols=300, wb=1 << 24, **kw):
    ld = max(cols, 1)
    a = dict(DY=P["DY"], lddy=ld, H=P["H"], ldh=ld, W=P["W"], rstd=P["RS"], DH=P["DH"], lddh=ld, DX=P["DX"], lddx=ld,
             DW=P["DW"], ws=P["A"])
    a.update(kw)
    return lib.sgemm_f8_rmsnorm_bwd(t, wt, rows, cols, a["DY"], a["lddy"], a["H"], a["ldh"], a["W"], a["rstd"],
                                    a["DH"], a["lddh"], a["DX"], a["lddx"], a["DW"], a["ws"], wb, 0)


@pytest.mark.parametrize("kw", [dict(t=-1), dict(wt=1), dict(rows=-1), dict(cols=lib.RMSNORM_MAX_COLS + 1),
                                dict(lddy=299), dict(ldh=299), dict(lddh=299), dict(lddx=299), dict(DY=0), dict(H=0),
                                dict(W=0), dict(rstd=0), dict(DX=0), dict(DY=P["DY"] + 1), dict(DW=P["DW"] + 2),
                                dict(ws=0), dict(ws=P["A"] + 4), dict(wb=-1)])
def test_bwd_refusals(kw):
    assert bwd(**kw) == INVALID


def test_bwd_needs_the_planned_workspace():
    need = lib.sgemm_f8_rmsnorm_bwd_plan(7, 300)[1]
    assert bwd(wb=need - 1) == INVALID
    assert bwd(wb=need - 1, ws=0) == INVALID


@pytest.mark.parametrize("kw", [dict(DX=P["DY"] + 2), dict(DX=P["H"], lddx=301), dict(DX=P["W"]), dict(DW=P["RS"]),
                                dict(DW=P["DX"]), dict(ws=P["DY"]), dict(ws=P["DX"]), dict(ws=P["DW"])])
def test_bwd_alias(kw):
    assert bwd(**kw) == ALIAS


def test_bwd_quick_returns_and_plan():
    assert bwd(cols=0, DY=0) == OK and bwd(rows=0, DW=0, DY=0) == OK
    st, nb = lib.sgemm_f8_rmsnorm_bwd_plan(7, 300)
    assert st == OK and nb > 0 and nb % 4 == 0
    st, nb = lib.sgemm_f8_rmsnorm_bwd_plan(16384, 4096)
    assert st == OK and 0 < nb <= 64 << 20
    assert lib.sgemm_f8_rmsnorm_bwd_plan(0, 300) == (OK, 0)
    assert lib.sgemm_f8_rmsnorm_bwd_plan(-1, 300)[0] == INVALID
    assert lib.sgemm_f8_rmsnorm_bwd_plan(1, lib.RMSNORM_MAX_COLS + 1)[0] == INVALID


def test_valid_calls_without_a_device_say_so():
    torch = pytest.importorskip("torch")
    if torch.cuda.is_available():
        pytest.skip("a GPU is here")
    assert gemm() == gemm(alpha=0.0, beta=2.0) == quant() == norm() == bwd() == 3  # SGEMM_ERR_NO_DEVICE
    assert norm(H=P["X"]) == norm(H=P["R"]) == bwd(DX=P["DY"]) == bwd(DX=P["H"]) == bwd(DX=P["DH"]) == 3


def test_tensor_wrappers_refuse_host_tensors():
    torch = pytest.importorskip("torch")
    x, w = torch.zeros(2, 8), torch.zeros(8)
    with pytest.raises(TypeError):
        lib.rmsnorm(x, w, Y=x)
    with pytest.raises(TypeError):
        lib.f8_quantize(x, torch.zeros(2, 8).to(torch.float8_e4m3fn), torch.zeros(1, 2))
    with pytest.raises(TypeError):
        lib.f8_gemm(x, x, x, x, x)
    with pytest.raises(TypeError):
        lib.rmsnorm_backward(x, x, w, w, x)


def test_gemm_workspace_query():
    for block in (0, 1):
        for M, N, K in ((1, 1, 1), (64, 4096, 4096), (128, 512, 8000), (512, 4096, 4096), (8192, 8192, 8192),
                        (1000, 1017, 999), (2048, 2048, 2047)):
            parts = lib.sgemm_f8_gemm_plan(block, M, N, K, 1)[5]
            assert lib.sgemm_f8_gemm_workspace(block, M, N, K, 1) == (OK, parts)
            st, nb = lib.sgemm_f8_gemm_workspace(block, M, N, K, 0)
            assert st == OK and (nb == 0 or nb >= (M + N) * K)
    assert lib.sgemm_f8_gemm_workspace(1, 4096, 4096, 4095, 0)[1] >= 8192 * 4096
    assert lib.sgemm_f8_gemm_workspace(1, 0, 5, 5) == (OK, 0) and lib.sgemm_f8_gemm_workspace(1, 5, 5, 0) == (OK, 0)
    big = (1 << 31) - 1025
    assert lib.sgemm_f8_gemm_workspace(1, big, big, big, 0)[0] == OK
    assert lib.sgemm_f8_gemm_workspace(1, big + 1, 1, 1)[0] == INVALID
    assert lib.sgemm_f8_gemm_workspace(2, 5, 5, 5)[0] == INVALID
    assert lib.sgemm_f8_gemm_workspace(1, 5, 5, 5, 3)[0] == INVALID
