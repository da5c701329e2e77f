"""The argument checks, plans and queries of the operators around a block in the library built
with AddressSanitizer and UndefinedBehaviorSanitizer on the host side (no GPU; no call reaches
a launch)."""
import os
import subprocess
import sys

from test_sanitizers_cpu import ROOT, sanitized  # noqa: F401


def test_boundary_file_under_asan_and_ubsan(sanitized):  # noqa: F811
    runtime, lib, _ = sanitized
    env = dict(os.environ, LD_PRELOAD=runtime, SGEMM_F32_LIBRARY=lib, HIP_VISIBLE_DEVICES="-1",
               ASAN_OPTIONS="detect_leaks=0:abort_on_error=0:halt_on_error=1",
               UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-m", "not gpu", "-p", "no:cacheprovider",
                        os.path.join(ROOT, "tests", "test_block_boundary_cpu.py")],
                       cwd=ROOT, env=env, capture_output=True, text=True, timeout=600)
    out = r.stdout + r.stderr
    assert "AddressSanitizer" not in out and "runtime error:" not in out, out[-4000:]
    assert r.returncode == 0 and " passed" in r.stdout.splitlines()[-1], out[-4000:]
