"""Which gates the second kernel of the norms' backward pass joins (no GPU).  The library's own
numbers come from a small host program; who has which rows is worked out here."""
import os
import subprocess

import pytest

import fp32_gemm_08_amd as lib
from fp32_gemm_08_amd import build as hipbuild

PROGRAM = r"""
#include "norm_internal.h"
#include <cstdio>
// rows cols gate_rows -> team walkers chunk, gates looked at
int main()
{
    long long rows, cols, gate_rows;
    while (scanf("%lld %lld %lld", &rows, &cols, &gate_rows) == 3) {
        const sgemm::BlockNormSums n = sgemm::block_norm_sums(rows, cols, gate_rows);
        printf("%lld %lld %lld %lld\n", (long long)n.team, (long long)n.walkers, (long long)n.chunk,
               (long long)sgemm::block_norm_gates_to_join(n, rows, gate_rows));
    }
}
"""


@pytest.fixture(scope="module")
def ask(tmp_path_factory):
    if not os.path.exists(lib.LIB_PATH):
        pytest.skip("libsgemm_f32.so not built")
    try:
        hipcc = hipbuild.hipcc()
    except RuntimeError:
        pytest.skip("no hipcc")
    d = tmp_path_factory.mktemp("gates")
    src, exe = str(d / "gates.cpp"), str(d / "gates")
    with open(src, "w", encoding="utf-8") as f:
        f.write(PROGRAM)
    r = subprocess.run([hipcc] + hipbuild.common_flags() + ["-x", "hip", src, "-x", "none", lib.LIB_PATH, "-o", exe,
                       "-Wl,-rpath," + os.path.dirname(lib.LIB_PATH)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr

    def call(calls):
        text = "".join(" ".join(str(v) for v in c) + "\n" for c in calls)
        r = subprocess.run([exe], input=text, capture_output=True, text=True, timeout=120)
        assert r.returncode == 0, r.stderr
        return [tuple(int(v) for v in line.split()) for line in r.stdout.splitlines()]

    return call


def joined(rows, gate_rows, chunk, looked_at):
    """The gates that the kernel adds slots for (walkers of `chunk` consecutive rows): its own choice."""
    out = []
    for i in range(looked_at):
        g = i if gate_rows >= chunk else (min(rows, (i + 1) * chunk) - 1) // gate_rows
        first, end = g * gate_rows, min(rows, (g + 1) * gate_rows)
        walkers = first // chunk, (end - 1) // chunk
        if walkers[0] != walkers[1] and (gate_rows >= chunk or walkers[0] == i):
            out.append(g)
    return out


def test_gates_are_joined_once_and_none_is_looked_at_where_none_is_split(ask):
    calls = [(rows, cols, gate_rows) for cols in (8, 200, 300, 700, 2000, 4096, 9001, 20000)
             for rows in (300, 1030, 2048, 9000, 12345, 65536)
             for gate_rows in (1, 2, 3, 4, 5, 7, 8, 9, 16, 31, 32, 64, 100, 256) if gate_rows < rows]
    none = 0
    for (rows, cols, gate_rows), (team, walkers, chunk, looked_at) in zip(calls, ask(calls)):
        gates = -(-rows // gate_rows)
        if team:
            assert looked_at == gates
            continue
        assert walkers == -(-rows // chunk)
        split = [g for g in range(gates) if g * gate_rows // chunk != (min(rows, (g + 1) * gate_rows) - 1) // chunk]
        assert joined(rows, gate_rows, chunk, looked_at) == split, (rows, cols, gate_rows)
        if chunk % gate_rows == 0:
            none += 1
            assert not split and looked_at == 0, (rows, cols, gate_rows, chunk, looked_at)
    assert none > 20
