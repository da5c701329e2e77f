"""The module of the tensor calls is used with the Python and the torch that it was compiled for,
whose tensors it reads, and with no other (no GPU)."""
import sys

import pytest

from fp32_gemm_08_amd import native

torch = pytest.importorskip("torch")


@pytest.fixture(autouse=True)
def unbound(monkeypatch):
    monkeypatch.setattr(native, "_module", None)


def test_says_what_it_was_built_for():
    from fp32_gemm_08_amd import _tensors

    python, version = _tensors.built_for.split()
    assert python == f"{sys.version_info.major}.{sys.version_info.minor}" and torch.__version__.startswith(version)
    assert native.tensors() is _tensors


def test_refuses_another_torch(monkeypatch):
    monkeypatch.setattr(torch, "__version__", "9.9.1+rocm")
    with pytest.raises(RuntimeError, match="9.9.1") as e:
        native.tensors()
    assert "build" in str(e.value) and native._module is None


def test_refuses_another_python(monkeypatch):
    from fp32_gemm_08_amd import _tensors

    monkeypatch.setattr(_tensors, "built_for", "3.1 " + torch.__version__.split("+")[0], raising=False)
    with pytest.raises(RuntimeError, match="3.1"):
        native.tensors()
