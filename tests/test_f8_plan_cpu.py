"""The plan of an 8-bit product against the 32-bit offsets of the pipelined kernels
(no GPU).  They hold a row's offset within a tile (row * ld, the last k-blocks beside
it), the byte count of a tile's last rows (rows * ld) and the offset of a tile's second
row of tile scales (4 * ldsb) in 32 bits, out of range from 0xfffffff0 on; so leading
dimensions of operands, laid out anew or not, and of such scales end at 2^22.

The library's own planning functions are called by a small host program, with the
leading dimensions of a call; its numbers are checked here in Python's integers."""
import os
import subprocess

import pytest

import fp32_gemm_08_amd as lib
from fp32_gemm_08_amd import build as hipbuild

ALL = 0xFFFFFFF0
MAX_LD = 1 << 22
ANY, SKINNY = 81, 80
TILE = {82: (64, 64), 83: (128, 64), 84: (128, 128), 85: (256, 256)}
ROOM = 1 << 44
INVALID_VALUE = 1  # hipErrorInvalidValue

PROGRAM = r"""
#include "f8_internal.h"
#include <cstdio>
// plan:   row_b M N K rows_on_16 lda ldb ldsb room -> kid pack splits bytes
// launch: the same of a plan for 128 x 128 tiles (rows_on_16 = 0: operands laid out
//         anew) -> the launch's status
int main(int argc, char **argv)
{
    const bool launch = argv[1][0] == 'l';
    long long b, M, N, K, on16, lda, ldb, ldsb, room;
    while (scanf("%lld %lld %lld %lld %lld %lld %lld %lld %lld", &b, &M, &N, &K, &on16, &lda, &ldb, &ldsb, &room) == 9) {
        sgemm::F8GemmArgs a{};
        a.M = (int)M, a.N = (int)N, a.K = (int)K;
        a.lda = lda, a.ldb = ldb, a.ldsa = M, a.ldsb = ldsb, a.ldc = N;
        a.alpha = 1.0f;
        a.c_type = SGEMM_TYPE_BF16;
        if (launch) {
            sgemm::F8GemmPlan p;
            p.kid = sgemm::KID_F8_M;
            p.tiles_m = (M + 127) / 128, p.tiles_n = (N + 127) / 128;
            p.pack = p.bytes = on16 ? 0 : (M + N) * ((K + 127) / 128 * 128);
            printf("%d\n", (int)sgemm::launch_f8_gemm(a, p, 1, 1, b != 0, nullptr));
        } else {
            const sgemm::F8GemmPlan p = sgemm::f8_call_plan(a, on16 != 0, b != 0, room);
            printf("%d %lld %lld %lld\n", p.kid, (long long)p.pack, (long long)p.splits, (long long)p.bytes);
        }
    }
}
"""


@pytest.fixture(scope="module")
def planner(tmp_path_factory):
    if not os.path.exists(lib.LIB_PATH):
        pytest.skip("libsgemm_f32.so not built")
    try:
        hipcc = hipbuild.hipcc()
    except RuntimeError:
        pytest.skip("no hipcc")
    d = tmp_path_factory.mktemp("plan")
    src, exe = str(d / "plan.cpp"), str(d / "plan")
    with open(src, "w", encoding="utf-8") as f:
        f.write(PROGRAM)
    r = subprocess.run([hipcc] + hipbuild.common_flags() + ["-x", "hip", src, "-x", "none", lib.LIB_PATH, "-o", exe,
                       "-Wl,-rpath," + os.path.dirname(lib.LIB_PATH)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr

    def ask(mode, calls):
        text = "".join(" ".join(str(int(v)) for v in c) + "\n" for c in calls)
        r = subprocess.run([exe, mode], input=text, capture_output=True, text=True, timeout=120)
        assert r.returncode == 0, r.stderr
        return [tuple(int(v) for v in line.split()) for line in r.stdout.splitlines()]

    return ask


def packed(K):
    return -(-K // 128) * 128


def call(row_b, M, N, K, on16, lda=None, ldb=None, ldsb=None, room=ROOM):
    return (row_b, M, N, K, on16, lda or K, ldb or K, ldsb or (N if row_b else -(-K // 128)), room)


def within(c, got):
    """A planned call's largest 32-bit quantities, where its kernel holds such ones."""
    row_b, M, N, K, _, lda, ldb, ldsb, _ = c
    kid, pack, splits, nbytes = got
    if kid not in TILE:
        assert kid in (ANY, SKINNY) and pack == 0
        return
    bm, bn = TILE[kid]
    if pack:
        lda = ldb = packed(K)
        assert pack == (M + N) * lda
    for rows, tile, ld in ((M, bm, lda), (N, bn, ldb)):
        assert ld >= K and ld % 16 == 0
        assert (min(rows, tile) - 1) * ld + packed(K) < ALL     # the last row's offset, with k beside it
        assert (tile - 1) * ld < ALL                             # the count of a part-filled tile's rows
        assert (tile - 1) * ld + 112 < ALL                       # a lane's offset, rows past the matrix too
    if not row_b:
        assert 4 * ldsb * ((min(bn, N) - 1) // 128) < 1 << 32


SIZES = [(17, 17), (100, 100), (512, 512), (300, 4000), (4096, 4096), (8192, 257)]


def test_offsets_of_every_plan_fit(planner):
    calls = []
    for M, N in SIZES:
        for K in (999, MAX_LD - 200, MAX_LD - 17, MAX_LD - 16, MAX_LD, MAX_LD + 1, MAX_LD + 16, 2 * MAX_LD, 33818641,
                  40000001, (1 << 26) + 1, (1 << 27) - 1, (1 << 28) - 3, (1 << 31) - 1025):
            for row_b in (0, 1):
                calls.append(call(row_b, M, N, K, 0))
                calls.append(call(row_b, M, N, K, 1, lda=K + -K % 16, ldb=K + -K % 16))
                calls.append(call(row_b, M, N, K, 1, lda=max(MAX_LD, K + -K % 16), ldb=2 * MAX_LD + K + -K % 16))
        for K in (999, 4095, 4096):
            for ldsb in (MAX_LD, MAX_LD + 1, 1 << 28, 1 << 30, (1 << 30) + 64, 1 << 33):
                calls.append(call(0, M, N, K, 0, ldsb=ldsb))
                calls.append(call(0, M, N, K, 1, lda=K + -K % 16, ldb=K + -K % 16, ldsb=ldsb))
    for c, got in zip(calls, planner("plan", calls)):
        within(c, got)


def test_the_limits_are_where_they_are_said_to_be(planner):
    big = 1 << 23                                                # k-blocks are no reason to pack below
    calls = [call(1, 512, 512, MAX_LD - 1, 0), call(1, 512, 512, MAX_LD + 1, 0),
             call(1, 512, 512, MAX_LD, 1), call(1, 512, 512, MAX_LD + 16, 1),
             call(0, 4096, 4096, 4095, 0, ldsb=MAX_LD), call(0, 4096, 4096, 4095, 0, ldsb=MAX_LD + 1),
             call(1, 4096, 4096, 4095, 0, ldsb=big), call(0, 4096, 128, 4096, 1, ldsb=big),
             call(0, 4096, 129, 4096, 1, ldsb=big)]
    got = planner("plan", calls)
    assert [g[1] > 0 for g in got] == [True, False, False, False, True, False, True, False, False]
    assert [g[0] in TILE for g in got] == [True, False, True, False, True, False, True, True, False]


def test_the_query_asks_for_no_packing_past_the_limit():
    for block in (0, 1):
        for M, N, K in ((512, 512, 40000001), (17, 17, (1 << 28) - 3), (100, 100, (1 << 27) - 1),
                        (512, 512, (1 << 26) + 1), (512, 512, MAX_LD + 1)):
            assert lib.sgemm_f8_gemm_workspace(block, M, N, K, 0) == (0, 0)
            assert lib.sgemm_f8_gemm_workspace(block, M, N, K, 1) == (0, 0)  # rows cannot be that near
            assert lib.sgemm_f8_gemm_plan(block, M, N, K, 1)[1] == ANY
        assert lib.sgemm_f8_gemm_workspace(block, 512, 512, MAX_LD - 1, 0)[1] >= 1024 * MAX_LD


def test_the_launch_refuses_what_its_offsets_cannot_hold(planner):
    """The check right before the kernels, were a plan to forget (no kernel is launched)."""
    calls = [call(1, 512, 512, MAX_LD + 16, 0), call(1, 512, 512, 4096, 1, lda=MAX_LD + 16),
             call(1, 512, 512, 4096, 1, ldb=1 << 28), call(0, 512, 512, 4096, 1, ldsb=1 << 30),
             call(0, 512, 512, 4095, 0, ldsb=1 << 30)]
    assert planner("launch", calls) == [(INVALID_VALUE,)] * len(calls)
