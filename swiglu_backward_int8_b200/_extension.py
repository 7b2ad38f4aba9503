"""The extension module of csrc/marshal.cpp, where it fits the installed torch.

It is a shorter way to the calls of lowbit.py, which has all of them without it:
where it is missing, or was built against another torch, the package works and
its small calls take some microseconds longer on the host.
"""
from __future__ import annotations

import importlib.util
import os
import sys
import types
import warnings

_PKG = os.path.dirname(os.path.abspath(__file__))
MODULE = os.path.join(_PKG, "_marshal.so")
BUILT_FOR = os.path.join(_PKG, "_marshal.txt")   # what MODULE was built for, written by build.py
NAMES = ("rmsnorm_quant", "rmsnorm_backward", "quantize_fp4", "dequantize_fp4", "matmul_fp4")


def installed() -> str:
    """What the module depends on: torch's C++ interfaces, their ABI, and Python's."""
    import torch
    return f"torch {torch.__version__}, C++ ABI {int(torch._C._GLIBCXX_USE_CXX11_ABI)}, Python {sys.implementation.cache_tag}"


def built_for(module: str = MODULE, record: str = BUILT_FOR) -> str:
    """What the module was built for; empty where there is none, or no record of it."""
    if not (os.path.exists(module) and os.path.exists(record)):
        return ""
    with open(record) as f:
        return f.read().strip()


def _left_to_python(*args) -> int:
    """The stand-in for each function: the answer of a call that the short way does not make."""
    return -1


def load(addresses: tuple):
    """The extension module, bound to the library's entries, or its stand-in."""
    have, want = built_for(), installed()
    why = None
    if have == want:
        spec = importlib.util.spec_from_file_location(f"{__package__}._marshal", MODULE)
        try:
            module = importlib.util.module_from_spec(spec)
            spec.loader.exec_module(module)
            module.bind(*addresses)
            sys.modules[spec.name] = module
            return module
        except ImportError as e:
            why = str(e)
    elif have:
        why = f"it was built for {have}, and this is {want}"
    else:
        why = "it is missing, or has no record of what it was built for"
    warnings.warn(f"{MODULE} is not used: {why}.  Calls of the norm, the 4-bit quantizer and the 4-bit product take some "
                  "microseconds longer on the host; build it with __graft_entry__.build().", RuntimeWarning, stacklevel=2)
    return types.SimpleNamespace(**{name: _left_to_python for name in NAMES})
