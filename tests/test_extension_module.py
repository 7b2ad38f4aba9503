"""The package with and without its extension module, and what a build makes anew, on the CPU."""
from __future__ import annotations

import importlib.util
import os
import pathlib
import shutil
import subprocess
import sys

import pytest

ROOT = pathlib.Path(__file__).resolve().parent.parent
PKG = "swiglu_backward_int8_b200"

USE = """
import warnings
with warnings.catch_warnings(record=True) as told:
    warnings.simplefilter("always")
    import swiglu_backward_int8_b200 as sdq
import torch
from swiglu_backward_int8_b200 import lowbit
assert sdq.__file__.startswith({root!r}), sdq.__file__
assert sdq.sdq_validate(0, 0, 0, 0, 0, 0, 5, 256, 128) == sdq.Status.ERR_NULL      # the older entries
x = torch.zeros(4, 64, dtype=torch.bfloat16)
assert lowbit._marshal.rmsnorm_quant(x, *[None] * 12) == -1
for call in (lambda: sdq.rmsnorm_quant(x, torch.ones(64)), lambda: sdq.quantize_fp4(x),
             lambda: sdq.dequantize_fp4(x, x), lambda: sdq.matmul_fp4(x, x, x, x),
             lambda: sdq.rmsnorm_backward(x, x, x, x)):
    try:
        call()
    except ValueError as e:
        assert "CUDA" in str(e)
    else:
        raise AssertionError("a host tensor was taken")
print("told:", *[str(w.message) for w in told if w.category is RuntimeWarning])
"""


def _copy(tmp_path):
    """The package in a folder of its own, with the built files."""
    to = tmp_path / PKG
    to.mkdir()
    for f in (ROOT / PKG).iterdir():
        if f.suffix in (".py", ".so", ".txt"):
            shutil.copy2(f, to / f.name)
    return to


def _use(tmp_path):
    env = dict(os.environ, PYTHONPATH=str(tmp_path))
    r = subprocess.run([sys.executable, "-c", USE.format(root=str(tmp_path))], cwd=tmp_path, env=env, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
    return r.stdout


def test_package_with_its_module(tmp_path):
    _copy(tmp_path)
    assert _use(tmp_path).strip() == "told:"


@pytest.mark.parametrize("what", ["missing", "another torch", "no record", "not a module"])
def test_package_without_its_module(tmp_path, what):
    """Everything is there, and a warning says what is not used and why."""
    to = _copy(tmp_path)
    if what == "missing":
        (to / "_marshal.so").unlink()
    elif what == "another torch":
        (to / "_marshal.txt").write_text("torch 2.10.0, C++ ABI 1, Python cpython-312\n")
    elif what == "no record":
        (to / "_marshal.txt").unlink()
    else:
        (to / "_marshal.so").write_bytes(b"\x7fELF" + bytes(60))
    told = _use(tmp_path)
    assert "_marshal.so is not used" in told and "build it" in told
    if what == "another torch":
        assert "torch 2.10.0" in told


# ---- what a build makes anew: the compilers are replaced by a function that records them ----

@pytest.fixture
def tree(tmp_path):
    """A copy of the sources, and a function: build, and return the outputs made (by nvcc and g++)."""
    shutil.copytree(ROOT / PKG / "csrc", tmp_path / PKG / "csrc")
    shutil.copytree(ROOT / "include", tmp_path / "include")
    for f in ("build.py", "_extension.py"):
        shutil.copy2(ROOT / PKG / f, tmp_path / PKG / f)

    def build(fails=()):
        spec = importlib.util.spec_from_file_location("sdq_build_copy", tmp_path / PKG / "build.py")
        mod = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(mod)
        made = []

        def run(cmd, verbose):
            out = cmd[cmd.index("-o") + 1]
            name = os.path.basename(out).split(".tmp")[0]
            if name in fails:
                raise RuntimeError("no such header")
            made.append(name)
            pathlib.Path(out).write_bytes(b"")

        mod._run, mod.nvcc = run, lambda: "/usr/local/cuda/bin/nvcc"
        mod.build()
        return sorted(made)

    build.pkg = tmp_path / PKG
    return build


ALL = sorted(["_marshal.so", "libsdq.so"] + [f"{f}.cu.o" for f in ("sdq_api", "fwd_api", "norm_api", "fp4_api")])


def test_build_goes_on_without_the_module(tree, capfd):
    assert tree(fails=("_marshal.so",)) == [f for f in ALL if f != "_marshal.so"]
    assert (tree.pkg / "libsdq.so").exists() and not (tree.pkg / "_marshal.so").exists()
    assert "_marshal.so was not built" in capfd.readouterr().err
    assert tree() == ["_marshal.so"]                     # tried again, alone
    assert tree() == []


def test_build_makes_the_module_anew_for_another_torch(tree):
    assert tree() == ALL and tree() == []
    (tree.pkg / "_marshal.txt").write_text("torch 2.10.0, C++ ABI 1, Python cpython-312\n")
    assert tree() == ["_marshal.so"] and tree() == []
    (tree.pkg / "_marshal.txt").unlink()
    assert tree() == ["_marshal.so"] and tree() == []


def test_build_makes_all_anew_after_a_change_of_its_flags(tree):
    assert tree() == ALL
    later = os.path.getmtime(tree.pkg / "libsdq.so") + 10
    os.utime(tree.pkg / "build.py", (later, later))
    assert tree() == ALL
