"""The native module of the tensor calls: what it refuses before it looks at a tensor, and
first calls from several threads (no GPU)."""
import subprocess
import sys
import threading

import pytest

from test_sanitizers_cpu import ROOT

torch = pytest.importorskip("torch")
NAMES = ("i8_gemm", "i8_quantize", "f8_requantize", "block_norm", "block_norm_backward")


def module():
    from fp32_gemm_08_amd.native import tensors

    return tensors()


@pytest.mark.parametrize("name", NAMES)
def test_refuses_other_argument_counts(name):
    call = getattr(module(), name)
    for n in (0, 1, 40):
        with pytest.raises(TypeError, match="arguments"):
            call(*[None] * n)


@pytest.mark.parametrize("what", [None, 1, "x", [1.0], object()])
def test_refuses_what_is_no_tensor(what):
    import fp32_gemm_08_amd as lib

    for call in (lambda: lib.i8_gemm(what, what, what, what, what), lambda: lib.i8_quantize(what, what, what),
                 lambda: lib.f8_requantize(what, what, what, what), lambda: lib.block_norm(what, what, what, H=what)):
        with pytest.raises((TypeError, ValueError)):
            call()


def test_bind_refuses_what_is_no_table_of_addresses():
    """In a process of its own: a failed bind() leaves the module unbound, and its calls say so."""
    code = ("import torch\n"
            "from fp32_gemm_08_amd import _tensors as t\n"
            "for args in ((), (1,), ((1, 2), None, None, None), ((), None, None, None)):\n"
            "    try:\n"
            "        t.bind(*args)\n"
            "    except (TypeError, ValueError):\n"
            "        pass\n"
            "    else:\n"
            "        raise SystemExit('bound')\n"
            "try:\n"
            "    t.i8_quantize(None, None, None, None)\n"
            "except RuntimeError as e:\n"
            "    print(e)\n")
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "bind()" in r.stdout, r.stdout + r.stderr


def test_first_calls_from_several_threads():
    import fp32_gemm_08_amd as lib
    from fp32_gemm_08_amd import native

    native._module = None
    x, q, s, got = torch.zeros(2, 8), torch.zeros(2, 8, dtype=torch.int8), torch.zeros(2), []
    start = threading.Barrier(8)

    def work():
        start.wait()
        try:
            lib.i8_quantize(x, q, s)
        except TypeError:
            got.append(1)

    threads = [threading.Thread(target=work) for _ in range(8)]
    for t in threads:
        t.start()
    for t in threads:
        t.join(60)
    assert len(got) == 8
