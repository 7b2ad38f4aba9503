"""The operators around the projections run together, as a quantized MLP uses
them: norm, 4-bit product, SwiGLU, quantizer, product; a linear layer's forward
and both its gradients; and the same under a CUDA graph, on other streams and
side by side."""
from __future__ import annotations

import pytest
import torch

import swiglu_backward_int8_b200 as sdq

pytestmark = pytest.mark.gpu


def _weights(gen, n, k, scales):
    w = (torch.randn(n, k, generator=gen, device="cuda") * k ** -0.5).bfloat16()
    g = (w.float().abs().max() / 2688).reshape(1) if scales == "e4m3" else None
    return (*sdq.quantize_fp4(w, scales, global_scale=g), g)


def _mlp(x, res, wn, gate_up, down, scales, g):
    q, s, h = sdq.rmsnorm_quant(x, wn, res, codes="e2m1", scales=scales, global_scale=g)
    gu = sdq.matmul_fp4(q, s, gate_up[0], gate_up[1], a_global=g, b_global=gate_up[2])
    inter = gu.shape[1] // 2
    act, _ = sdq.swiglu_q8_1(gu[:, :inter], gu[:, inter:])
    qa, sa = sdq.quantize_fp4(act, scales, global_scale=g)
    return h, q, s, gu, act, sdq.matmul_fp4(qa, sa, down[0], down[1], a_global=g, b_global=down[2])


def _values(q, s, g):
    """Exact: a code times its scale has at most six bits, so bf16 holds it; the scale per tensor comes after."""
    return sdq.dequantize_fp4(q, s).double() * (1 if g is None else g.double())


@pytest.mark.parametrize("scales", ["e8m0", "e4m3"])
@pytest.mark.parametrize("rows", [1, 37, 300])
def test_mlp_forward(scales, rows):
    gen = torch.Generator(device="cuda").manual_seed(rows)
    k, inter = 512, 704
    x, res = (torch.randn(rows, k, generator=gen, device="cuda").bfloat16() for _ in range(2))
    wn = torch.rand(k, generator=gen, device="cuda") + 0.5
    gate_up, down = _weights(gen, 2 * inter, k, scales), _weights(gen, k, inter, scales)
    g = torch.tensor([2.0 ** -8], device="cuda") if scales == "e4m3" else None
    h, q, s, gu, act, y = _mlp(x, res, wn, gate_up, down, scales, g)
    assert torch.equal(h, (x.float() + res.float()).bfloat16())
    # each step from the one before it, in 64 bits: a 4-bit code is off by a quarter
    # of its group's largest value at most ([4, 6] has a step of 2, and E4M3
    # scales add 2^-4), the products by 2^-8 and k / 16 2^-23 of the magnitudes,
    # silu by 2^-8
    hd = h.double()
    want = hd / (hd.square().mean(1, keepdim=True) + 1e-6).sqrt() * wn.double()
    n = {"e8m0": 32, "e4m3": 16}[scales]
    top = want.abs().reshape(rows, -1, n).amax(2).repeat_interleave(n, 1)
    assert ((_values(q, s, g) - want).abs() <= 0.26 * top).all()
    a, b = _values(q, s, g), _values(*gate_up)
    w, m = a @ b.t(), a.abs() @ b.abs().t()
    assert ((gu.double() - w).abs() <= 2.0 ** -8 * w.abs() + (k / 16 + 2) * 2.0 ** -23 * m).all()
    gd, ud = gu[:, :inter].double(), gu[:, inter:].double()
    w = gd * torch.sigmoid(gd) * ud
    assert ((act.double() - w).abs() <= 2.0 ** -7 * w.abs() + 1e-30).all()
    qa, sa = sdq.quantize_fp4(act, scales, global_scale=g)
    a, b = _values(qa, sa, g), _values(*down)
    w, m = a @ b.t(), a.abs() @ b.abs().t()
    assert ((y.double() - w).abs() <= 2.0 ** -8 * w.abs() + (inter / 16 + 2) * 2.0 ** -23 * m).all()


@pytest.mark.parametrize("scales", ["e8m0", "e4m3"])
@pytest.mark.parametrize("rows", [5, 200])
def test_linear_forward_and_gradients(scales, rows):
    """y = x W^T, its data and its weight gradient, each a product of 4-bit operands; the gradients against
    autograd through the values that the operands stand for."""
    gen = torch.Generator(device="cuda").manual_seed(rows)
    k, n = 320, 288
    x = torch.randn(rows, k, generator=gen, device="cuda").bfloat16()
    w = (torch.randn(n, k, generator=gen, device="cuda") * 0.1).bfloat16()
    gy = torch.randn(rows, n, generator=gen, device="cuda").bfloat16()
    qx, sx, qxt, sxt = sdq.quantize_fp4(x, scales, "both")
    qw, sw, qwt, swt = sdq.quantize_fp4(w, scales, "both")
    qg, sg, qgt, sgt = sdq.quantize_fp4(gy, scales, "both")
    y = sdq.matmul_fp4(qx, sx, qw, sw, out_dtype=torch.float32)
    gx = sdq.matmul_fp4(qg, sg, qwt, swt, out_dtype=torch.float32)
    gw = sdq.matmul_fp4(qgt, sgt, qxt, sxt, out_dtype=torch.float32)
    d = lambda q, s: sdq.dequantize_fp4(q, s).double()  # noqa: E731
    for got, a, b in ((y, d(qx, sx), d(qw, sw)), (gx, d(qg, sg), d(qwt, swt)), (gw, d(qgt, sgt), d(qxt, sxt))):
        tol = (a.shape[1] / 16 + 2) * 2.0 ** -23 * (a.abs() @ b.abs().t())
        assert ((got.double() - a @ b.t()).abs() <= tol).all()
    # the transposed codes are those of the transposed tensor, the missing rows zeros
    pad = torch.zeros(-(-rows // 32) * 32, k, dtype=torch.bfloat16, device="cuda")
    pad[:rows] = x
    q2, s2 = sdq.quantize_fp4(pad.t().contiguous(), scales)
    assert torch.equal(q2, qxt) and torch.equal(d(q2, s2), d(qxt, sxt))
    xa, wa = d(qx, sx).requires_grad_(), d(qw, sw).requires_grad_()
    (xa @ wa.t() * gy.double()).sum().backward()
    # what remains is the quantization of gy and of the other operand: a quarter of a group's largest value each
    rel = lambda a, b: float((a.double() - b).norm() / b.norm())  # noqa: E731
    assert rel(gx, xa.grad) < 0.26 and rel(gw[:n], wa.grad) < 0.52


def _chain_state(seed, rows, scales="e8m0"):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    k, inter = 256, 384
    x, res = (torch.randn(rows, k, generator=gen, device="cuda").bfloat16() for _ in range(2))
    wn = torch.rand(k, generator=gen, device="cuda") + 0.5
    g = torch.tensor([2.0 ** -8], device="cuda") if scales == "e4m3" else None
    return x, res, wn, _weights(gen, 2 * inter, k, scales), _weights(gen, k, inter, scales), scales, g


@pytest.mark.parametrize("rows", [3, 200])
def test_graph_replays_on_new_inputs(rows):
    st = _chain_state(1, rows)
    other = _chain_state(2, rows)
    want = [t.clone() for t in _mlp(*other[:2], *st[2:])]
    gy = torch.randn(rows, 256, device="cuda").bfloat16()
    rstd = torch.ones(rows, device="cuda")
    want_b = [t.clone() for t in sdq.rmsnorm_backward(gy, other[0], st[2], rstd)]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = _mlp(*st)
        outs_b = sdq.rmsnorm_backward(gy, st[0], st[2], rstd)
    for _ in range(3):
        st[0].copy_(other[0])
        st[1].copy_(other[1])
        for t in (*outs, *outs_b):
            t.view(torch.uint8).zero_()
        graph.replay()
        torch.cuda.synchronize()
        # (scale tiles: rows past the last are not written)
        for i, (a, b) in enumerate(zip((*outs, *outs_b), (*want, *want_b))):
            assert i == 2 or torch.equal(a, b), i
    assert sdq.sdq_device_status() == 0


def test_back_to_back_and_on_other_streams():
    """Calls queued one behind the other (each kernel may start while the one before it ends) and on two streams at
    once give what calls with a synchronize between them give."""
    states = [_chain_state(s, r, sc) for s, (r, sc) in enumerate([(1, "e8m0"), (150, "e4m3"), (40, "e8m0"), (300, "e8m0")])]
    want = []
    for st in states:
        outs = _mlp(*st)
        torch.cuda.synchronize()
        want.append(outs)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        got = []
        for i, st in enumerate(states):
            with torch.cuda.stream(streams[i % 2]):
                got.append(_mlp(*st))
        for st in states:
            got.append(_mlp(*st))
        torch.cuda.synchronize()
        for outs, ref in zip(got, want + want):
            for i, (a, b) in enumerate(zip(outs, ref)):
                assert i == 2 or torch.equal(a, b), i
    assert sdq.sdq_device_status() == 0
