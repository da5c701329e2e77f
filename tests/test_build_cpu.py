"""The build without and with torch (no GPU, no compiler run): the C library depends on neither
torch nor the module that calls it with torch tensors."""
import importlib.util
import os

import pytest

from fp32_gemm_08_amd import build as hipbuild


class Done:
    returncode, stdout, stderr = 0, "", ""


@pytest.fixture
def tools(tmp_path, monkeypatch):
    """Compilers that write an empty file and say what they were asked for."""
    ran = []

    def run(cmd, **kw):
        out = cmd[cmd.index("-o") + 1]
        ran.append(os.path.basename(out))
        open(out, "w").close()
        return Done()

    monkeypatch.setattr(hipbuild.subprocess, "run", run)
    monkeypatch.setattr(hipbuild, "hipcc", lambda: "hipcc")
    monkeypatch.setattr(hipbuild, "BUILD", str(tmp_path / "build"))
    monkeypatch.setattr(hipbuild, "LIB", str(tmp_path / "lib.so"))
    monkeypatch.setattr(hipbuild, "TENSORS", str(tmp_path / "_tensors.so"))
    return tmp_path, ran


def test_builds_both(tools):
    path, ran = tools
    assert hipbuild.build() == str(path / "lib.so")
    assert (path / "lib.so").exists() and (path / "_tensors.so").exists()


def test_builds_the_library_without_torch(tools, monkeypatch, capsys):
    path, ran = tools
    monkeypatch.setattr(importlib.util, "find_spec", lambda name: None)
    hipbuild.build(verbose=True)
    assert (path / "lib.so").exists() and not (path / "_tensors.so").exists()
    assert "torch" in capsys.readouterr().out


def test_a_failure_of_the_module_leaves_the_new_library(tools, monkeypatch):
    path, ran = tools
    good = hipbuild.subprocess.run

    class Failed:
        returncode, stdout, stderr = 1, "", "no such header"

    def run(cmd, **kw):
        return Failed() if any("tensors.cpp" in c for c in cmd) else good(cmd, **kw)

    monkeypatch.setattr(hipbuild.subprocess, "run", run)
    with pytest.raises(RuntimeError, match="no such header"):
        hipbuild.build()
    assert (path / "lib.so").exists()


def test_variants_build_no_module(tools, monkeypatch):
    path, ran = tools
    monkeypatch.setattr(hipbuild, "variant_path", lambda v: str(path / f"{v}.so"))
    hipbuild.build(variant="poison")
    assert (path / "poison.so").exists() and not (path / "_tensors.so").exists()

