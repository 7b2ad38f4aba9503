"""The norm, quantizer and product on the ways a call can take: through the
extension module or the Python checks, first met inside a graph capture, with
offsets past 32 bits, on a stream of their own."""
from __future__ import annotations

import os
import subprocess
import sys

import pytest
import torch

import swiglu_backward_int8_b200 as sdq
from swiglu_backward_int8_b200 import _marshal, lowbit

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
NAMES = ("rmsnorm_quant", "rmsnorm_backward", "quantize_fp4", "dequantize_fp4", "matmul_fp4")


def test_short_way_leaves_the_unusual_to_python():
    """On the CPU: -1 for host tensors, missing outputs, other objects and other argument counts."""
    x, w = torch.zeros(4, 64, dtype=torch.bfloat16), torch.ones(64)
    q, s = torch.zeros(4, 64, dtype=torch.int8), torch.zeros(4, 1)
    full = (x, w, None, 1e-6, None, None, None, q, s, None, None, None, None)
    assert _marshal.rmsnorm_quant(*full) == -1
    assert _marshal.rmsnorm_quant(*full[:7], None, s, *full[9:]) == -1
    assert _marshal.rmsnorm_quant(None, *full[1:]) == -1
    assert _marshal.rmsnorm_quant("x", *full[1:]) == -1
    for name, n in zip(NAMES, (13, 8, 8, 4, 8)):
        f = getattr(_marshal, name)
        assert f(*[None] * n) == -1 and f(*[None] * (n - 1)) == -1 and f() == -1 and f(*[3.5] * n) == -1
    with pytest.raises(TypeError):
        _marshal.bind(1, 2)
    with pytest.raises(ValueError):
        _marshal.bind(0, 0, 0, 0, 0, 0)


def _calls():
    """One call of each function with every output given; returns {name: outputs}."""
    g = torch.Generator(device="cuda").manual_seed(11)
    rows, k, n = 37, 256, 96
    x, r, gy = (torch.randn(rows, k, generator=g, device="cuda").bfloat16() for _ in range(3))
    w = torch.nn.Parameter(torch.rand(k, generator=g, device="cuda"))
    b = torch.randn(n, k, generator=g, device="cuda").bfloat16()
    e = lambda *s, dtype=torch.uint8: torch.zeros(s, dtype=dtype, device="cuda")  # noqa: E731
    one = torch.tensor([0.01], device="cuda")
    out = {}
    h, y, rstd = torch.zeros_like(x), torch.zeros_like(x), e(rows, dtype=torch.float32)
    q, s, _ = sdq.rmsnorm_quant(x, w.detach(), r, 1e-5, 64, codes="e4m3", scales="e8m0",
                                q=e(rows, k, dtype=torch.float8_e4m3fn), s=e(rows, 4), h=h, y=y, rstd=rstd)
    out["norm"] = (q, s, h, y, rstd)
    q4, s4, _ = sdq.rmsnorm_quant(x, w.detach(), codes="e2m1", scales="e4m3", q=e(rows, k // 2),
                                  s=e(*sdq.fp4_scale_shape(rows, k, "e4m3")).view(torch.float8_e4m3fn), global_scale=one)
    out["norm4"] = (q4, s4)
    gx, gw = torch.zeros_like(x), e(k, dtype=torch.float32)
    sdq.rmsnorm_backward(gy, h, w.detach(), rstd, r, grad_x=gx, grad_weight=gw)
    out["backward"] = (gx, gw)
    a = sdq.quantize_fp4(x, "e8m0", "both", q=e(rows, k // 2), s=e(*sdq.fp4_scale_shape(rows, k)), q_t=e(k, 32),
                         s_t=e(*sdq.fp4_scale_shape(k, 64)))
    c = sdq.quantize_fp4(x, axis="columns", q_t=e(k, 32), s_t=e(*sdq.fp4_scale_shape(k, 64)))
    out["quantize"], out["columns"] = a, c
    out["dequantize"] = (sdq.dequantize_fp4(q4, s4, one, out=torch.zeros_like(x)),)
    bq, bs = sdq.quantize_fp4(b, q=e(n, k // 2), s=e(*sdq.fp4_scale_shape(n, k)))
    out["matmul"] = (sdq.matmul_fp4(a[0], a[1], bq, bs, out=e(rows, n, dtype=torch.float32)),)
    torch.cuda.synchronize()
    return out


@pytest.mark.gpu
def test_both_ways_make_the_same_call(monkeypatch):
    made = []

    def counted(name):
        f = getattr(_marshal, name)

        def call(*args):
            made.append((name, f(*args)))
            return made[-1][1]
        return call

    for name in NAMES:
        monkeypatch.setattr(lowbit._marshal, name, counted(name))
    short = _calls()
    assert len(made) == 8 and all(status == 0 for _, status in made), made
    monkeypatch.undo()
    for name in NAMES:
        monkeypatch.setattr(lowbit._marshal, name, lambda *args: -1)
    long = _calls()
    for name in short:
        for a, b in zip(short[name], long[name]):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), name


@pytest.mark.gpu
def test_both_ways_refuse_alike(monkeypatch):
    x = torch.zeros(4, 72, dtype=torch.bfloat16, device="cuda")[:, :64]          # rows on 16 bytes: fine
    bad = torch.zeros(4, 68, dtype=torch.bfloat16, device="cuda")[:, :64]        # rows that are not
    w, q, s = torch.ones(64, device="cuda"), torch.zeros(4, 64, dtype=torch.int8, device="cuda"), torch.zeros(4, 1, device="cuda")
    for way in range(2):
        sdq.rmsnorm_quant(x, w, q=q, s=s)
        with pytest.raises(sdq.SdqError) as e:
            sdq.rmsnorm_quant(bad, w, q=q, s=s)
        assert e.value.status == sdq.Status.ERR_ALIGN
        for kw in (dict(codes="e4m3"), dict(scales="e8m0"), dict(group_size=48), dict(h=x), dict(rstd=w)):
            with pytest.raises(ValueError):
                sdq.rmsnorm_quant(x, w, **dict(dict(q=q, s=s), **kw))
        for name in NAMES:
            monkeypatch.setattr(lowbit._marshal, name, lambda *args: -1)


@pytest.mark.gpu
def test_first_calls_inside_a_capture():
    """A process whose very first calls are captured: nothing is set up that a capture forbids."""
    code = """
import torch
import swiglu_backward_int8_b200 as sdq
x = torch.randn(40, 256, device="cuda").bfloat16()
w = torch.ones(256, device="cuda")
big = torch.randint(0, 256, (1700, 128), dtype=torch.uint8, device="cuda")
big_s = torch.full(sdq.fp4_scale_shape(1700, 256), 127, dtype=torch.uint8, device="cuda")
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    q, s, h = sdq.rmsnorm_quant(x, w, x.clone(), codes="e2m1")
    y = sdq.matmul_fp4(q, s, q, s)
    z = sdq.matmul_fp4(big, big_s, big, big_s)
    v = sdq.dequantize_fp4(q, s)
    t = sdq.quantize_fp4(x, axis="both")
    gx, gw = sdq.rmsnorm_backward(x, h, w, torch.ones(40, device="cuda"))
g.replay()
torch.cuda.synchronize()
assert sdq.sdq_device_status() == 0
want = v.double() @ v.double().t()
assert ((y.double() - want).abs() <= 2.0 ** -7 * want.abs() + 1e-3).all()
b = sdq.dequantize_fp4(big, big_s).double()
want = b @ b.t()
assert ((z.double() - want).abs() <= 2.0 ** -7 * want.abs() + 1e-2).all()
print("ok")
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip().endswith("ok"), r.stdout + r.stderr


def _apart(rows, cols, dtype, gap):
    """A [rows, cols] view whose rows lie `gap` elements apart."""
    buf = torch.empty((rows - 1) * gap + cols, dtype=dtype, device="cuda")
    return buf.as_strided((rows, cols), (gap, 1))


@pytest.mark.gpu
def test_offsets_past_32_bits():
    """Rows more than 2^32 bytes apart, in every operand that has a stride."""
    rows, k, gap = 3, 64, (1 << 31) + 64
    x = torch.randn(rows, k, device="cuda").bfloat16()
    w = torch.ones(k, device="cuda")
    far = _apart(rows, k, torch.bfloat16, gap)
    far.copy_(x)
    q8 = _apart(rows, k, torch.int8, gap)
    rstd = torch.empty(rows, device="cuda")
    a = sdq.rmsnorm_quant(far, w, q=q8, rstd=rstd)
    b = sdq.rmsnorm_quant(x, w)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    ga, gb = sdq.rmsnorm_backward(far, far, w, rstd, grad_x=far), sdq.rmsnorm_backward(x, x, w, rstd)
    assert torch.equal(ga[0], gb[0]) and torch.equal(ga[1], gb[1])
    far.copy_(x)
    del q8
    torch.cuda.empty_cache()
    q4, q4t = _apart(rows, k // 2, torch.uint8, gap), _apart(k, 16, torch.uint8, 1 << 27)
    _, s, _, st = sdq.quantize_fp4(far, axis="both", q=q4, q_t=q4t)
    c, cs, ct, cts = sdq.quantize_fp4(x, axis="both")
    assert torch.equal(q4, c) and torch.equal(q4t, ct)
    near = sdq.dequantize_fp4(c, cs)
    assert torch.equal(sdq.dequantize_fp4(q4, s, out=far), near)
    out = far[:, :rows]
    assert torch.equal(sdq.matmul_fp4(q4, s, q4, s, out=out), sdq.matmul_fp4(c, cs, c, cs))


@pytest.mark.gpu
def test_calls_on_a_stream_of_their_own_wait_for_its_work():
    """Inputs written just before on the same side stream, outputs read just after."""
    stream = torch.cuda.Stream()
    want = None
    for side in (False, True, True):
        with torch.cuda.stream(stream if side else torch.cuda.current_stream()):
            x = torch.full((300, 512), 1.0, device="cuda")
            for _ in range(20):
                x = x * 1.01 + 0.1
            q, s = sdq.quantize_fp4(x.bfloat16())
            y = sdq.matmul_fp4(q, s, q, s, out_dtype=torch.float32) * 2
        torch.cuda.synchronize()
        want = y if want is None else want
        assert torch.equal(y, want)
