"""The C ABIs of the norms around a block, of the products of 8-bit integers and of the
requantisation without a GPU: declared symbols, refusals, quick returns and the planning
queries (fake addresses; no call reaches a launch)."""
import ctypes
import os
import re

import pytest

import fp32_gemm_08_amd as lib

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, INVALID, ALIAS, NO_DEVICE = 0, 1, 2, 3
P = {name: (i + 1) << 40 for i, name in enumerate(
    "A SA B SB C WS X O W WP G H Y Q S H8 SH O8 SO RS RP DY DH DX DO DW DWP DG QT ST".split())}
BIG = (1 << 31) - 1025


@pytest.fixture(scope="module", autouse=True)
def built():
    if not os.path.exists(lib.LIB_PATH):
        pytest.skip("libsgemm_f32.so not built")


@pytest.mark.parametrize("header,prefix,exports", [("sgemm_i8.h", "sgemm_i8_", lib.I8_EXPORTS),
                                                   ("sgemm_norm.h", "sgemm_block_norm", lib.NORM_EXPORTS)])
def test_exports_every_declared_symbol(header, prefix, exports):
    text = open(os.path.join(ROOT, "include", header), encoding="utf-8").read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    declared = sorted(set(re.findall(r"\b(%s\w*)\s*\(" % prefix, text)))
    assert declared == sorted(exports)
    so = ctypes.CDLL(lib.LIB_PATH)
    for name in declared:
        assert hasattr(so, name), name


# ------------------------------------------------------------------ products of 8-bit integers

def gemm(ct=2, M=64, N=256, K=384, alpha=1.0, beta=0.0, W=0, wb=0, **kw):
    a = dict(A=P["A"], lda=max(K, 1), SA=P["SA"], B=P["B"], ldb=max(K, 1), SB=P["SB"], C=P["C"], ldc=max(N, 1))
    a.update(kw)
    return lib.sgemm_i8_gemm(ct, M, N, K, alpha, a["A"], a["lda"], a["SA"], a["B"], a["ldb"], a["SB"], beta, a["C"],
                             a["ldc"], W, wb, 0)


@pytest.mark.parametrize("kw", [
    dict(ct=3), dict(ct=-1), dict(M=-1), dict(N=1 << 31), dict(K=-1), dict(K=lib.I8_MAX_K + 1), dict(lda=383), dict(ldb=383),
    dict(ldc=255), dict(A=0), dict(SA=0), dict(B=0), dict(SB=0), dict(C=0), dict(SA=P["SA"] + 2), dict(SB=P["SB"] + 1),
    dict(C=P["C"] + 1), dict(ct=0, C=P["C"] + 2), dict(wb=-1), dict(W=P["WS"] + 8, wb=64), dict(lda=1 << 62),
    dict(M=1 << 30, N=1 << 30, ldc=1 << 30), dict(K=0, lda=0), dict(alpha=0.0, beta=2.0, C=0)])
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
    assert gemm(K=0, beta=1.0, A=0, B=0) == OK


def test_gemm_plans():
    for M, N, K in ((1, 1, 1), (1, 4096, 4096), (48, 16384, 4096), (64, 1024, 16384), (100, 300, 20000), (512, 4096, 4096),
                    (8192, 8192, 8192), (1000, 1017, 999), (2048, 2048, 2047)):
        for al in (0, 1):
            st, kid, tm, tn, sp, nb = lib.sgemm_i8_gemm_plan(M, N, K, al)
            assert st == OK and kid >= 90 and tm >= 1 and tn >= 1 and sp >= 1
            assert (nb == 0) == (sp == 1) and (sp == 1 or nb >= 4 * sp * M * N)
            st, room = lib.sgemm_i8_gemm_workspace(M, N, K, al)
            assert st == OK and (al == 0 or room == nb)
    assert lib.sgemm_i8_gemm_plan(0, 5, 5)[1] == 0 and lib.sgemm_i8_gemm_plan(5, 5, 0)[1] == 0
    assert lib.sgemm_i8_gemm_plan(-5, 5, 5)[0] == INVALID and lib.sgemm_i8_gemm_plan(5, 5, lib.I8_MAX_K + 1)[0] == INVALID
    assert lib.sgemm_i8_gemm_plan(5, 5, 5, 2)[0] == INVALID and lib.sgemm_i8_gemm_workspace(5, 5, 5, 2)[0] == INVALID
    assert lib.sgemm_i8_gemm_workspace(0, 5, 5) == (OK, 0)
    assert lib.sgemm_i8_gemm_workspace(BIG, BIG, lib.I8_MAX_K, 0)[0] == OK
    assert lib.sgemm_i8_gemm_workspace(BIG + 1, 1, 1, 1)[0] == INVALID


def quant(xt=2, rows=200, cols=300, **kw):
    a = dict(X=P["X"], ldx=max(cols, 1), Q=P["Q"], ldq=max(cols, 1), S=P["S"])
    a.update(kw)
    return lib.sgemm_i8_quantize(xt, rows, cols, a["X"], a["ldx"], a["Q"], a["ldq"], a["S"], 0)


def test_quantize_checks():
    for kw in (dict(xt=3), dict(rows=-1), dict(cols=1 << 31), dict(ldx=299), dict(ldq=299), dict(X=0), dict(Q=0), dict(S=0),
               dict(X=P["X"] + 1), dict(S=P["S"] + 2), dict(xt=0, X=P["X"] + 2), dict(rows=1 << 30)):
        assert quant(**kw) == INVALID, kw
    for kw in (dict(Q=P["X"] + 5), dict(S=P["X"] + 4), dict(S=P["Q"])):
        assert quant(**kw) == ALIAS, kw
    assert quant(rows=0, X=0) == OK and quant(cols=0, X=0) == OK


# ------------------------------------------------------------------ requantisation

def requant(fx=1, fmt=1, rows=200, cols=300, **kw):
    a = dict(X=P["X"], ldx=max(cols, 1), SX=P["S"], ldsx=max(rows, 1), QT=P["QT"], ldqt=max(rows, 1), ST=P["ST"],
             ldst=max(cols, 1))
    a.update(kw)
    return lib.sgemm_f8_requantize(fx, fmt, rows, cols, a["X"], a["ldx"], a["SX"], a["ldsx"], a["QT"], a["ldqt"], a["ST"],
                                   a["ldst"], 0)


def test_requantize_checks():
    for kw in (dict(fx=0), dict(fmt=3), dict(rows=-1), dict(cols=1 << 31), dict(ldx=299), dict(ldsx=199), dict(ldqt=199),
               dict(ldst=299), dict(X=0), dict(SX=0), dict(QT=0), dict(ST=0), dict(SX=P["S"] + 2), dict(ST=P["ST"] + 1),
               dict(rows=BIG, cols=BIG)):
        assert requant(**kw) == INVALID, kw
    for kw in (dict(QT=P["X"] + 5), dict(QT=P["S"]), dict(ST=P["X"]), dict(ST=P["S"] + 4), dict(ST=P["QT"])):
        assert requant(**kw) == ALIAS, kw
    assert requant(rows=0, X=0) == OK and requant(cols=0, X=0) == OK


# ------------------------------------------------------------------ the norms

def norm(t=2, wt=2, rows=8, cols=300, gate_rows=4, alpha=1.0, eps=1e-6, qf=1, **kw):
    ld, lr = max(cols, 1), max(rows, 1)
    a = dict(X=P["X"], ldx=ld, O=P["O"], ldo=ld, W=P["W"], WP=P["WP"], G=P["G"], ldg=ld, H=P["H"], ldh=ld, Y=P["Y"], ldy=ld,
             Q=P["Q"], ldq=ld, S=P["S"], lds=lr, H8=P["H8"], ldh8=ld, SH=P["SH"], ldsh=lr, O8=P["O8"], ldo8=ld, SO=P["SO"],
             ldso=lr, RS=P["RS"], RP=P["RP"])
    a.update(kw)
    return lib.sgemm_block_norm(t, wt, rows, cols, a["X"], a["ldx"], a["O"], a["ldo"], a["W"], a["WP"], a["G"], a["ldg"],
                                gate_rows, alpha, eps, a["H"], a["ldh"], a["Y"], a["ldy"], qf, a["Q"], a["ldq"], a["S"],
                                a["lds"], a["H8"], a["ldh8"], a["SH"], a["ldsh"], a["O8"], a["ldo8"], a["SO"], a["ldso"],
                                a["RS"], a["RP"], 0)


@pytest.mark.parametrize("kw", [
    dict(t=3), dict(wt=1), dict(t=0, wt=2), dict(rows=-1), dict(cols=-1), dict(cols=lib.RMSNORM_MAX_COLS + 1), dict(eps=-1.0),
    dict(eps=float("nan")), dict(eps=float("inf")), dict(alpha=float("nan")), dict(alpha=float("inf")), dict(gate_rows=0),
    dict(gate_rows=-3), dict(qf=2), dict(qf=0), dict(ldx=299), dict(ldo=299), dict(ldg=299), dict(ldh=299), dict(ldy=299),
    dict(ldq=299), dict(lds=7), dict(ldh8=299), dict(ldsh=7), dict(ldo8=299), dict(ldso=7), dict(X=0), dict(W=0), dict(S=0),
    dict(SH=0), dict(SO=0), dict(X=P["X"] + 1), dict(O=P["O"] + 1), dict(G=P["G"] + 1), dict(WP=P["WP"] + 1),
    dict(RS=P["RS"] + 2), dict(RP=P["RP"] + 1), dict(wt=0, G=P["G"] + 2), dict(S=P["S"] + 2), dict(qf=3, S=P["S"] + 2),
    dict(rows=1 << 30)])
def test_norm_refusals(kw):
    assert norm(**kw) == INVALID


@pytest.mark.parametrize("kw", [dict(Y=P["X"]), dict(Y=P["O"]), dict(H=P["X"] + 2), dict(H=P["O"], ldh=301), dict(Q=P["X"]),
                                dict(H=P["Y"]), dict(H8=P["O"]), dict(O8=P["O"]), dict(SH=P["G"]), dict(RS=P["WP"]),
                                dict(RS=P["RP"]), dict(O8=P["H8"]), dict(SO=P["SH"] + 8), dict(H=P["G"]), dict(S=P["Q"] + 4)])
def test_norm_alias(kw):
    assert norm(**kw) == ALIAS


def test_norm_quick_returns():
    none = dict(H=0, Y=0, Q=0, H8=0, O8=0, RS=0, RP=0)
    assert norm(rows=0, X=0, W=0) == OK and norm(cols=0, X=0) == OK and norm(X=0, **none) == OK
    assert norm(X=0, O=0, **dict(none, O8=P["O8"], RP=P["RP"])) == OK       # they belong to O


def bwd(t=2, wt=2, rows=8, cols=300, kept=0, gate_rows=4, alpha=1.0, wb=1 << 24, **kw):
    ld, lr = max(cols, 1), max(rows, 1)
    a = dict(DY=P["DY"], lddy=ld, DH=P["DH"], lddh=ld, H=P["H"], ldh=ld, SH=P["SH"], ldsh=lr, O=P["O"], ldo=ld, SO=P["SO"],
             ldso=lr, W=P["W"], WP=P["WP"], RS=P["RS"], RP=P["RP"], G=P["G"], ldg=ld, DX=P["DX"], lddx=ld, DO=P["DO"], lddo=ld,
             DW=P["DW"], DWP=P["DWP"], DG=P["DG"], lddg=ld, ws=P["WS"])
    a.update(kw)
    return lib.sgemm_block_norm_bwd(t, wt, rows, cols, a["DY"], a["lddy"], a["DH"], a["lddh"], kept, a["H"], a["ldh"], a["SH"],
                                    a["ldsh"], a["O"], a["ldo"], a["SO"], a["ldso"], a["W"], a["WP"], a["RS"], a["RP"], a["G"],
                                    a["ldg"], gate_rows, alpha, a["DX"], a["lddx"], a["DO"], a["lddo"], a["DW"], a["DWP"],
                                    a["DG"], a["lddg"], a["ws"], wb, 0)


@pytest.mark.parametrize("kw", [
    dict(t=-1), dict(wt=1), dict(rows=-1), dict(cols=lib.RMSNORM_MAX_COLS + 1), dict(kept=2), dict(kept=-1),
    dict(alpha=float("inf")), dict(gate_rows=0), dict(wb=-1), dict(DY=0, DH=0), dict(O=0), dict(WP=0), dict(G=0),
    dict(WP=0, DWP=0, O=0), dict(lddy=299), dict(lddh=299), dict(ldh=299), dict(ldo=299), dict(ldg=299), dict(lddx=299),
    dict(lddo=299), dict(lddg=299), dict(kept=1, ldsh=7), dict(kept=1, ldso=7), dict(kept=1, SH=0), dict(kept=1, SO=0),
    dict(kept=1, SO=P["SO"] + 2), dict(H=0), dict(W=0), dict(RS=0), dict(RP=0), dict(DY=P["DY"] + 1), dict(H=P["H"] + 1),
    dict(O=P["O"] + 1), dict(DX=P["DX"] + 1), dict(DW=P["DW"] + 2), dict(DG=P["DG"] + 1), dict(ws=0), dict(ws=P["WS"] + 4)])
def test_bwd_refusals(kw):
    assert bwd(**kw) == INVALID


def test_bwd_needs_the_planned_workspace():
    need = lib.sgemm_block_norm_bwd_plan(8, 300, 4)[1]
    assert bwd(wb=need - 1) == INVALID and bwd(wb=need - 1, ws=0) == INVALID
    assert bwd(rows=8, gate_rows=8, wb=lib.sgemm_block_norm_bwd_plan(8, 300, 8)[1] - 1) == INVALID


@pytest.mark.parametrize("kw", [dict(DX=P["DY"] + 2), dict(DX=P["H"], lddx=301), dict(DX=P["O"]), dict(DO=P["H"]),
                                dict(DX=P["W"]), dict(DO=P["G"]), dict(DW=P["RS"]), dict(DG=P["G"]), dict(DWP=P["DW"]),
                                dict(DO=P["DX"]), dict(DX=P["DY"], DO=P["DY"]), dict(kept=1, DX=P["H"]),
                                dict(kept=1, DO=P["O"]), dict(kept=1, DO=P["SO"]), dict(ws=P["DY"]), dict(ws=P["DG"])])
def test_bwd_alias(kw):
    assert bwd(**kw) == ALIAS


def test_bwd_quick_returns_and_plan():
    sums = dict(DW=0, DWP=0, DG=0)
    assert bwd(cols=0, DY=0) == OK and bwd(rows=0, DY=0, **sums) == OK and bwd(DX=0, DO=0, H=0, **sums) == OK
    plan = lib.sgemm_block_norm_bwd_plan
    for cols in (1, 128, 300, 1000, 2000, 4096, 8192, 16384, lib.RMSNORM_MAX_COLS):
        for rows in (1, 7, 1000, 16384, BIG):
            for gate_rows in (0, 1, 3, 2048, rows):
                st, nb = plan(rows, cols, gate_rows)
                assert st == OK and 0 < nb <= 128 << 20 and nb % (4 * cols) == 0
    assert plan(16384, 4096, 0) == plan(16384, 4096, 16384) == plan(16384, 4096, 1 << 40)
    assert plan(16384, 4096, 64)[1] > plan(16384, 4096, 2048)[1] > plan(16384, 4096, 0)[1]
    assert plan(0, 300, 5) == (OK, 0)
    assert plan(-1, 300, 0)[0] == INVALID and plan(1, lib.RMSNORM_MAX_COLS + 1, 0)[0] == INVALID and plan(1, 1, -1)[0] == INVALID


def test_valid_calls_without_a_device_say_so():
    torch = pytest.importorskip("torch")
    if torch.cuda.is_available():
        pytest.skip("a GPU is here")
    assert gemm() == gemm(alpha=0.0, beta=2.0) == quant() == requant() == norm() == bwd() == bwd(kept=1) == NO_DEVICE
    assert norm(H=P["X"]) == norm(H=P["O"]) == norm(O=0, WP=0) == norm(qf=3, lds=0) == norm(W=0, Y=0, Q=0) == NO_DEVICE
    assert norm(G=0, gate_rows=0) == norm(gate_rows=1 << 40) == NO_DEVICE
    assert bwd(DX=P["DY"], DO=P["O"]) == bwd(DX=P["H"], DO=P["DH"]) == bwd(kept=1, DX=P["DH"], DO=P["DY"]) == NO_DEVICE
    assert bwd(DY=0, H=0, W=0, RS=0) == bwd(DO=0, DWP=0, DG=0, O=0, WP=0, G=0, gate_rows=0) == NO_DEVICE
    assert bwd(WP=0, RP=0, DWP=0, DG=0, O=0) == bwd(DW=0, DWP=0, DG=0, ws=0, wb=0) == NO_DEVICE
    assert bwd(rows=0) == NO_DEVICE


def test_tensor_wrappers_refuse_host_tensors():
    torch = pytest.importorskip("torch")
    x, w = torch.zeros(2, 8), torch.zeros(8)
    q = torch.zeros(2, 8, dtype=torch.int8)
    for call in (lambda: lib.i8_gemm(q, x, q, x, x), lambda: lib.i8_quantize(x, q, w),
                 lambda: lib.f8_requantize(q.view(torch.float8_e4m3fn), x, q, x), lambda: lib.block_norm(x, x, w, H=x),
                 lambda: lib.block_norm_backward(x, x, x, w, w, x, x)):
        with pytest.raises(TypeError):
            call()
