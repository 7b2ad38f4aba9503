"""The 4-bit product's failure path: loads withheld by the test hook, waits that run out, a status, and a context that
goes on.  Nothing faults or hangs: every wait is bounded, and what is in flight lands before a CTA leaves."""
from __future__ import annotations

import time

import pytest
import torch

import swiglu_backward_int8_b200 as sdq
from swiglu_backward_int8_b200 import _lib

pytestmark = pytest.mark.gpu
_FMT = {"e8m0": sdq.FMT_E8M0, "e4m3": sdq.FMT_SCALE_E4M3}


def _operands(m, n, k, scales):
    gen = torch.Generator(device="cuda").manual_seed(m + k)
    a, b = (torch.randn(r, k, generator=gen, device="cuda").bfloat16() for r in (m, n))
    return (*sdq.quantize_fp4(a, scales), *sdq.quantize_fp4(b, scales))


def _stall(ops, out, scales, rank, step, limit_ns):
    a, a_s, b, b_s = ops
    stream = torch.cuda.current_stream().cuda_stream
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    _lib.sdq_matmul_fp4_test_stall(a.data_ptr(), a.stride(0), a_s.data_ptr(), b.data_ptr(), b.stride(0), b_s.data_ptr(),
                                   out.data_ptr(), out.stride(0), a.shape[0], b.shape[0], 2 * a.shape[1],
                                   _FMT[scales] | (sdq.FMT_OUT_F32 if out.dtype == torch.float32 else 0), rank, step, limit_ns,
                                   stream)
    status = sdq.sdq_device_status(stream)
    # the end waits for a second at most; what it waits for comes in microseconds, so it ends by itself
    assert time.perf_counter() - t0 < 0.5
    return status


def _then_right(ops, dtype, want):
    """The next calls, of either form, are right."""
    for _ in range(2):
        assert torch.equal(sdq.matmul_fp4(*ops, out_dtype=dtype), want)
    assert sdq.sdq_device_status() == sdq.Status.OK


@pytest.mark.parametrize("scales", ["e8m0", "e4m3"])
@pytest.mark.parametrize("m,n,k,rank,step", [(5, 300, 1024, 0, 0), (5, 300, 8192, 3, 1), (64, 300, 1024, 0, 2), (64, 300, 7168, 1, 5),
                                             (300, 500, 2048, 0, 7)])
def test_few_rows_with_loads_withheld(scales, m, n, k, rank, step):
    ops = _operands(m, n, k, scales)
    want = sdq.matmul_fp4(*ops)
    assert sdq.sdq_device_status() == sdq.Status.OK
    out = torch.empty_like(want)
    assert _stall(ops, out, scales, rank, step, 2_000_000) == sdq.Status.ERR_TIMEOUT
    _then_right(ops, torch.bfloat16, want)


@pytest.mark.parametrize("scales", ["e8m0", "e4m3"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rank", [0, 1])
@pytest.mark.parametrize("step", [0, 3, 8, 21])
def test_pairs_with_loads_withheld(scales, dtype, rank, step):
    """8 steps a tile and several tiles a pair: none, some or all stages full, the first or a later tile, the CTA that
    issues the products ahead of the other or behind it."""
    ops = _operands(2600, 4100, 2048, scales)
    want = sdq.matmul_fp4(*ops, out_dtype=dtype)
    assert sdq.sdq_device_status() == sdq.Status.OK
    out = torch.empty_like(want)
    assert _stall(ops, out, scales, rank, step, 2_000_000) == sdq.Status.ERR_TIMEOUT
    _then_right(ops, dtype, want)


def test_short_limits_and_calls_behind_one_another():
    """A limit of 50 us, other work queued behind the call that stops early."""
    ops, few = _operands(2600, 4100, 2048, "e8m0"), _operands(5, 300, 8192, "e8m0")
    want, want_few = sdq.matmul_fp4(*ops), sdq.matmul_fp4(*few)
    out = torch.empty_like(want)
    stream = torch.cuda.current_stream().cuda_stream
    for rank, step in ((0, 2), (1, 2), (0, 9), (1, 12)):
        a, a_s, b, b_s = ops
        _lib.sdq_matmul_fp4_test_stall(a.data_ptr(), a.stride(0), a_s.data_ptr(), b.data_ptr(), b.stride(0), b_s.data_ptr(),
                                       out.data_ptr(), out.stride(0), 2600, 4100, 2048, sdq.FMT_E8M0, rank, step, 50_000, stream)
        got_few, got = sdq.matmul_fp4(*few), sdq.matmul_fp4(*ops)
        assert sdq.sdq_device_status(stream) == sdq.Status.ERR_TIMEOUT
        assert torch.equal(got, want) and torch.equal(got_few, want_few)
    assert sdq.sdq_device_status() == sdq.Status.OK


def test_loads_that_are_never_reached_hold_nothing_up():
    ops = _operands(64, 300, 1024, "e8m0")
    out = torch.empty(64, 300, dtype=torch.bfloat16, device="cuda")
    assert _stall(ops, out, "e8m0", 0, 4, 2_000_000) == sdq.Status.OK
    assert torch.equal(out, sdq.matmul_fp4(*ops))


def test_refusals():
    ops = _operands(5, 300, 1024, "e8m0")
    out = torch.empty(5, 300, dtype=torch.bfloat16, device="cuda")
    for rank, step, limit in ((-1, 0, 10 ** 6), (0, -1, 10 ** 6), (0, 0, 999), (0, 0, 10 ** 9 + 1)):
        with pytest.raises(sdq.SdqError) as e:
            _stall(ops, out, "e8m0", rank, step, limit)
        assert e.value.status == sdq.Status.ERR_SHAPE
