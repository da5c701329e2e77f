"""What the tensor calls say where their module is absent, or there but not for this Python or
this torch (no GPU)."""
import os
import sys

import pytest

from fp32_gemm_08_amd import native

pytest.importorskip("torch")


class Finder:
    """Puts an ImportError in the place of the module."""

    def find_spec(self, name, path=None, target=None):
        if name == "fp32_gemm_08_amd._tensors":
            raise ImportError("undefined symbol: _ZN5torch5movedEv")


@pytest.fixture
def unloadable(monkeypatch):
    import fp32_gemm_08_amd

    monkeypatch.setattr(native, "_module", None)
    monkeypatch.delitem(sys.modules, "fp32_gemm_08_amd._tensors", raising=False)
    monkeypatch.delattr(fp32_gemm_08_amd, "_tensors", raising=False)
    monkeypatch.setattr(sys, "meta_path", [Finder()] + sys.meta_path)


def test_a_module_that_does_not_load_is_not_called_missing(unloadable, monkeypatch, tmp_path):
    there = tmp_path / "_tensors.so"
    there.write_text("")
    monkeypatch.setattr(native, "MODULE", str(there), raising=False)
    with pytest.raises(RuntimeError) as e:
        native.tensors()
    assert "missing" not in str(e.value) and "undefined symbol" in str(e.value) and "build" in str(e.value)


def test_a_missing_module_is(unloadable, monkeypatch, tmp_path):
    monkeypatch.setattr(native, "MODULE", str(tmp_path / "_tensors.so"), raising=False)
    with pytest.raises(RuntimeError, match="missing"):
        native.tensors()


def test_it_is_where_the_build_puts_it():
    from fp32_gemm_08_amd import build

    assert os.path.abspath(native.MODULE) == build.TENSORS
