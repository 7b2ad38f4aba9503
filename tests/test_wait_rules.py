"""Rules of the products' bounded waits, checked on the sources."""
from __future__ import annotations

import re

from tests.test_launch_overlap_rules import _code
from tests.test_source_rules import _cuda_sources


def _products():
    return {p.name: _code(p.read_text()) for p in _cuda_sources() if p.name.startswith("fp4_matmul")}


def _before(code, at):
    """The innermost condition of the code at `at`: "elect" inside a branch that one elected lane takes, else ""."""
    depth = 0
    for m in reversed(list(re.finditer(r"[{}]", code[:at]))):
        depth += 1 if m.group() == "}" else -1
        if depth < 0:
            depth = 0
            head = code[code.rfind("\n", 0, m.start()) + 1:m.start()]
            if "elect_one()" in head:
                return "elect"
    return ""


def test_a_warp_decides_together_whether_its_wait_ran_out():
    """A wait that may run out is called by one elected lane, or its answer goes through a vote: tcgen05.ld and the
    cluster's barriers, which take whole warps, follow."""
    calls = 0
    for name, code in _products().items():
        for m in re.finditer(r"(?<![\w])wait\(sync,", code):
            calls += 1
            line = code[code.rfind("\n", 0, m.start()) + 1:code.find("\n", m.start())]
            assert _before(code, m.start()) == "elect" or re.search(r"all_lanes\([^;]*wait\(sync", line), (name, line.strip())
    assert calls >= 7


def test_the_products_test_hook_refuses_before_any_launch():
    import pytest
    import swiglu_backward_int8_b200 as sdq
    from swiglu_backward_int8_b200 import _lib
    good = dict(a=1 << 20, ld_a=48, a_s=1 << 20, b=1 << 20, ld_b=48, b_s=1 << 20, out=1 << 20, ld_out=7, m=5, n=7, k=96,
                format=sdq.FMT_E8M0, rank=0, step=0, limit=10 ** 6, stream=None)
    for kw, status in ((dict(rank=-1), 3), (dict(step=-1), 3), (dict(limit=999), 3), (dict(limit=10 ** 9 + 1), 3),
                       (dict(format=0), 9), (dict(a=None), 1), (dict(ld_out=6), 10)):
        with pytest.raises(sdq.SdqError) as e:
            _lib.sdq_matmul_fp4_test_stall(*dict(good, **kw).values())
        assert e.value.status == status, kw
