"""Build the in-tree CUDA library ``libsdq.so`` for sm_100a.

    python swiglu_backward_int8_b200/build.py [--verbose]

(run it as a script: importing the package needs the library it builds)

nvcc compiles ``csrc/sdq_api.cu`` (host API + the fused kernel),
``csrc/fwd_api.cu`` (the forward-side SwiGLU + q8_1 kernel),
``csrc/norm_api.cu`` (the quantizing RMS norm) and ``csrc/fp4_api.cu`` (the
4-bit quantizer and product), each in a process of its own, and links them into
a shared library with a C ABI (``include/sdq.h``); the CUDA runtime is linked
statically and the driver's tensor-map encoder is looked up at run time, so
the library needs only the NVIDIA driver at load time.  ``csrc/marshal.cpp``, the
short way from torch tensors to the library's entries, becomes the extension
module ``_marshal.so`` against the installed torch, which ``_marshal.txt`` records.
The package works without it (_extension.py): where it cannot be compiled, that is
said and the build goes on.
"""
from __future__ import annotations

import concurrent.futures
import importlib.util
import os
import re
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libsdq.so")
MARSHAL = os.path.join(PKG, "_marshal.so")
MARSHAL_RECORD = os.path.join(PKG, "_marshal.txt")
MARSHAL_SOURCE = os.path.join(CSRC, "marshal.cpp")
OBJECTS = os.path.join(PKG, "_build")   # one object a source, kept for the next build
SOURCES = [os.path.join(CSRC, f) for f in ("sdq_api.cu", "fwd_api.cu", "norm_api.cu", "fp4_api.cu")]
DEPS = sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC)) + [os.path.join(INCLUDE, "sdq.h"), os.path.abspath(__file__)]

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
NVCC_FLAGS = ["-O3", "-std=c++17", *ARCH, "-lineinfo", "-Xcompiler", "-fPIC,-O2",
              "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _extension():
    """_extension.py, loaded by path: importing the package needs the library."""
    spec = importlib.util.spec_from_file_location("sdq_extension", os.path.join(PKG, "_extension.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def _run(cmd, verbose: bool) -> None:
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"compiling failed:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    if verbose:
        sys.stderr.write(r.stdout + r.stderr)


def _includes(path: str) -> set:
    """The source and the files of this repository that it includes."""
    found, todo = set(), [path]
    while todo:
        f = todo.pop()
        if f in found:
            continue
        found.add(f)
        with open(f) as src:
            for name in re.findall(r'^#include "([^"]+)"', src.read(), flags=re.M):
                todo += [p for d in (CSRC, INCLUDE) if os.path.exists(p := os.path.join(d, name))]
    return found


def _compile(source: str, obj: str, force: bool, verbose: bool) -> None:
    """Compile one source unless its object is newer than all that goes into it."""
    used = _includes(source) | {os.path.abspath(__file__)}
    if not force and os.path.exists(obj) and os.path.getmtime(obj) >= max(os.path.getmtime(f) for f in used):
        return
    tmp = f"{obj}.tmp{os.getpid()}"
    _run([nvcc(), *NVCC_FLAGS, *(["-Xptxas", "-v"] if verbose else []), "-c", source, "-o", tmp], verbose)
    os.replace(tmp, obj)


def _compile_marshal(verbose: bool) -> None:
    """The extension module: the host compiler, torch's headers and libraries."""
    import sysconfig
    import torch
    base = os.path.dirname(os.path.abspath(torch.__file__))
    cuda = os.path.dirname(os.path.dirname(nvcc()))
    includes = [INCLUDE, os.path.join(base, "include"), os.path.join(base, "include", "torch", "csrc", "api", "include"),
                os.path.join(cuda, "include"), sysconfig.get_paths()["include"]]
    lib = os.path.join(base, "lib")
    tmp = MARSHAL + f".tmp{os.getpid()}"
    _run([shutil.which("g++") or "g++", "-O2", "-std=c++17", "-fPIC", "-shared",
          f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
          *(f"-I{i}" for i in includes), MARSHAL_SOURCE, "-o", tmp, f"-L{lib}", "-ltorch_python", "-ltorch", "-ltorch_cpu",
          "-lc10_cuda", "-lc10", f"-Wl,-rpath,{lib}"], verbose)
    if os.path.exists(MARSHAL_RECORD):   # (a new module beside an old record would not be loaded)
        os.remove(MARSHAL_RECORD)
    os.replace(tmp, MARSHAL)
    with open(MARSHAL_RECORD, "w") as f:
        f.write(_extension().installed() + "\n")


def _newer(so: str) -> bool:
    """Whether a built file is there and newer than all sources."""
    return os.path.exists(so) and os.path.getmtime(so) >= max(os.path.getmtime(f) for f in DEPS)


def _marshal_fits() -> bool:
    """Whether _marshal.so is newer than the sources and was built for this torch."""
    if not _newer(MARSHAL):
        return False
    e = _extension()
    return e.built_for(MARSHAL, MARSHAL_RECORD) == e.installed()


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile libsdq.so if it is missing or older than the sources, and
    _marshal.so likewise, or if it was built for another torch."""
    todo = force or not _newer(LIB)
    marshal = force or not _marshal_fits()
    if not todo and not marshal:
        return LIB
    os.makedirs(OBJECTS, exist_ok=True)
    objects = [os.path.join(OBJECTS, os.path.basename(s) + ".o") for s in SOURCES]
    with concurrent.futures.ThreadPoolExecutor(len(SOURCES) + 1) as pool:
        short = pool.submit(_compile_marshal, verbose) if marshal else None
        if todo:
            for _ in pool.map(lambda so: _compile(*so, force, verbose), zip(SOURCES, objects)):
                pass
        try:
            if short:
                short.result()
        except Exception as e:   # no torch headers, no host compiler, ...
            for f in (MARSHAL, MARSHAL_RECORD):
                if os.path.exists(f):
                    os.remove(f)
            sys.stderr.write(f"{MARSHAL} was not built, the package goes without it:\n{e}\n")
    if todo:
        tmp = LIB + f".tmp{os.getpid()}"
        _run([nvcc(), *ARCH, "-shared", *objects, "-o", tmp], verbose)
        os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    build(force=True, verbose="--verbose" in sys.argv)
    print(LIB)
