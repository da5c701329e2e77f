"""The module ``_tensors`` (csrc/tensors.cpp), which calls the library with torch tensors: it
checks them as ``f8`` does in Python and raises the same exceptions, in a few hundred
nanoseconds.  It is built next to the library; there is no other way to these calls.
"""
from __future__ import annotations

import ctypes
import os
import sys

from .sgemm import SGEMM_OK, SgemmError, load, sgemm_f32_status_string

# The C functions it calls, in the order of its bind().
CALLS = ("sgemm_i8_gemm", "sgemm_i8_quantize", "sgemm_f8_requantize", "sgemm_block_norm", "sgemm_block_norm_bwd")

MODULE = os.path.join(os.path.dirname(os.path.abspath(__file__)), "_tensors.so")
_module = None


def tensors():
    """The module, bound to the loaded library."""
    return _module or _bind()


def _bind():
    global _module
    import torch

    try:
        from . import _tensors
    except ImportError as e:
        if os.path.exists(MODULE):
            raise RuntimeError(f"_tensors.so does not load ({e}): it is built for one Python and one torch; build it again "
                               "(python -m fp32_gemm_08_amd.build)") from e
        raise RuntimeError("_tensors.so is missing: build it (python -m fp32_gemm_08_amd.build)") from e
    python, version = getattr(_tensors, "built_for", "? ?").split()
    if python != f"{sys.version_info.major}.{sys.version_info.minor}" or not torch.__version__.startswith(version):
        raise RuntimeError(f"_tensors.so is built for Python {python} and torch {version}, not for "
                           f"{sys.version_info.major}.{sys.version_info.minor} and {torch.__version__}: build it again "
                           "(python -m fp32_gemm_08_amd.build)")
    lib = load()
    _tensors.bind(tuple(ctypes.cast(getattr(lib, name), ctypes.c_void_p).value for name in CALLS),
                  torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice, torch._C._cuda_setDevice)
    _module = _tensors
    return _module


def check(status):
    if status != SGEMM_OK:
        raise SgemmError(status, sgemm_f32_status_string(status))
