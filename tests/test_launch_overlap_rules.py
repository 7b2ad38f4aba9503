"""Every kernel of the library may start before the kernel ahead of it in the stream has ended, and waits for that
one's end before it reads (griddepcontrol.wait).  What it reads then is not constant for its lifetime: the compiler may
move a load through the non-coherent path across the wait, and that path's cache may hold what was there before."""
from __future__ import annotations

import re

from tests.test_source_rules import _cuda_sources


def _code(text):
    return re.sub(r"//[^\n]*|/\*.*?\*/", "", text, flags=re.S)


def test_no_load_through_the_non_coherent_path():
    for p in _cuda_sources():
        found = re.findall(r"__ldg\b|ld\.global[.\w:]*\.nc\b|__restrict__", _code(p.read_text()))
        assert not found, (p.name, found)


def test_every_file_with_a_kernel_waits_for_the_kernel_before():
    files = [c for c in (_code(p.read_text()) for p in _cuda_sources()) if "__global__" in c]
    assert len(files) >= 5
    for code in files:
        assert re.search(r"(?<!void )grid_dependency_wait\(\);", code)
