"""The norm, its backward, the 4-bit quantizer and the product at the ends of their ranges: tensors of zeros with
the scale per tensor that zeros give, rows and scales whose squares and products leave fp32's range."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import swiglu_backward_int8_b200 as sdq
from tests import lowbit_ref as R

pytestmark = pytest.mark.gpu


def _bytes(t):
    return t.view(torch.uint8).cpu().numpy()


@pytest.mark.parametrize("rows,channels", [(1, 32), (40, 64), (130, 288)])
def test_tensor_of_zeros_with_its_own_scale_per_tensor(rows, channels):
    """amax / 2688 of zeros is 0: scales of 1 and codes of 0, which keep their sign, along both axes and after a norm."""
    x = torch.zeros(rows, channels, dtype=torch.bfloat16, device="cuda")
    x[:, 1::2] = -0.0
    g = (x.float().abs().amax() / 2688).reshape(1)
    assert float(g) == 0
    pad = -(-rows // 32) * 32
    s, st = (torch.full(sdq.fp4_scale_shape(r, k, "e4m3"), 0xA5, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
             for r, k in ((rows, channels), (channels, pad)))
    q, _, qt, _ = sdq.quantize_fp4(x, "e4m3", "both", s=s, s_t=st, global_scale=g)
    assert (R.unpack(_bytes(q)) == np.where(np.arange(channels) % 2, 8, 0)).all()
    assert (R.unpack(_bytes(qt))[:, :rows] == np.where(np.arange(channels) % 2, 8, 0)[:, None]).all()
    assert (R.unpack(_bytes(qt))[:, rows:] == 0).all()
    assert (_bytes(s).reshape(-1)[R.tile_index(rows, channels // 16)] == 0x38).all()
    assert (_bytes(st).reshape(-1)[R.tile_index(channels, pad // 16)] == 0x38).all()
    assert (sdq.dequantize_fp4(q, s, g) == 0).all() and (sdq.dequantize_fp4(qt, st, g) == 0).all()
    q, s, _ = sdq.rmsnorm_quant(x, torch.ones(channels, device="cuda"), codes="e2m1", scales="e4m3", global_scale=g)
    assert (R.unpack(_bytes(q)) & 7 == 0).all()
    assert (_bytes(s).reshape(-1)[R.tile_index(rows, channels // 16)] == 0x38).all()
    y = sdq.matmul_fp4(q, s, q, s, a_global=g, b_global=g)
    assert (y == 0).all()


@pytest.mark.parametrize("g", [1e-45, 1e-38, 0.37, 1e30, 3e38])
def test_groups_of_zeros_among_others(g):
    """Rows of zeros next to others, with scales per tensor from the smallest to the largest."""
    x = torch.randn(70, 96, device="cuda").bfloat16()
    x[5], x[33:64], x[:, 32:64] = 0, 0, 0
    q, s, qt, st = sdq.quantize_fp4(x, "e4m3", "both", global_scale=torch.tensor([g], device="cuda"))
    zero = x == 0
    for c, t, z in ((q, s, zero), (qt, st, torch.nn.functional.pad(zero.t(), (0, 26), value=True))):
        c, z = R.unpack(_bytes(c)), z.cpu().numpy()
        assert (c[z] & 7 == 0).all()
        none = z.reshape(z.shape[0], -1, 16).all(2)
        assert none.any() and (_bytes(t).reshape(-1)[R.tile_index(*none.shape)][none] == 0x38).all()


@pytest.mark.parametrize("rows,channels", [(6, 256), (2000, 64), (700, 6160), (3, 16400)])
@pytest.mark.parametrize("size,grad", [(3e-20, 1.0), (1e-25, 1e-3), (1e18, 1e-6), (3e17, 1e-9)])
def test_backward_of_tiny_and_huge_rows(rows, channels, size, grad):
    """rstd^2 or rstd^3 would leave fp32's range here (or its normal numbers); grad_x does not.  Every product that the
    formula names stays normal, so the errors are those of ordinary rows: half a bf16 step and, with 4 vectors of a
    thread at most (every 1024th of a longer row), (4 + 24) 2^-24 of the magnitudes."""
    gen = torch.Generator(device="cuda").manual_seed(rows)
    h = (torch.randn(rows, channels, generator=gen, device="cuda") * size).bfloat16()
    gy = (torch.randn(rows, channels, generator=gen, device="cuda") * grad).bfloat16()
    w = torch.rand(channels, generator=gen, device="cuda") + 0.5
    rstd = torch.rsqrt(h.double().square().mean(1)).float()
    gx, gw, mag, magw = R.norm_backward(gy, h, w, rstd, None)
    got, gotw = sdq.rmsnorm_backward(gy, h, w, rstd)
    assert float(gx.abs().max()) < 1e38 and got.isfinite().all()
    # (results below 2^-126 are rounded to bf16's subnormal spacing, 2^-133)
    assert ((got.double() - gx).abs() <= 2.0 ** -8 * gx.abs() + 28 * 2.0 ** -24 * mag + 2.0 ** -134).all()
    assert ((gotw.double() - gw).abs() <= (-(-rows // 32) + 96) * 2.0 ** -24 * magw).all()


@pytest.mark.parametrize("ga,gb", [(1e-25, 1e-18), (1e-12, 1e-30), (2e-38, 0.5), (3e20, 5e19), (1e30, 1e-33), (1e-20, 0.0)])
@pytest.mark.parametrize("m,n,k", [(20, 40, 256), (20, 40, 4096), (1700, 1600, 256)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_product_of_scales_per_tensor_past_the_range(ga, gb, m, n, k, dtype):
    """The two scales' product leaves fp32's normal range, the output does not (or is 0).  The sums as in test_fp4_gpu;
    two more products, 2^-24 each; half a bf16 step."""
    gen = torch.Generator(device="cuda").manual_seed(m + k)
    size = 1e-3 if ga > 1e15 and gb > 1e15 else 30.0
    a, b = ((torch.randn(r, k, generator=gen, device="cuda") * size).bfloat16() for r in (m, n))
    (a, a_s), (b, b_s) = sdq.quantize_fp4(a, "e4m3"), sdq.quantize_fp4(b, "e4m3")
    av, bv = sdq.dequantize_fp4(a, a_s).double(), sdq.dequantize_fp4(b, b_s).double()     # (at most seven bits: exact)
    g = [torch.tensor([v], device="cuda") for v in (ga, gb)]
    got = sdq.matmul_fp4(a, a_s, b, b_s, a_global=g[0], b_global=g[1], out_dtype=dtype).double()
    alpha = float(g[0].double() * g[1].double())
    want, mag = (av @ bv.t()) * alpha, (av.abs() @ bv.abs().t()) * alpha
    assert float(mag.max()) < 1e38
    tol = (k / 16 + 2) * 2.0 ** -23 * mag + 2.0 ** -23 * want.abs()
    if dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * want.abs() + 2.0 ** -134
    assert ((got - want).abs() <= tol + 2.0 ** -149).all(), float(((got - want).abs() / tol.clamp(min=1e-300)).max())


def test_norm_of_a_weight_that_the_kernel_before_writes():
    """The weight's memory changes in each call before the norm; both kernels may overlap up to the norm's wait."""
    gen = torch.Generator(device="cuda").manual_seed(4)
    x, gy = (torch.randn(900, 4096, generator=gen, device="cuda").bfloat16() for _ in range(2))
    base = torch.randn(1, 4096, generator=gen, device="cuda")
    codes = [sdq.quantize_fp4((base * f).bfloat16()) for f in (1, -2)]
    weights = [sdq.dequantize_fp4(*c) for c in codes]
    rstd = torch.empty(900, device="cuda")
    want = [(sdq.rmsnorm_quant(x, w[0], rstd=rstd)[0], *sdq.rmsnorm_backward(gy, x, w[0], rstd)) for w in weights]
    w = torch.empty_like(weights[0])
    for _ in range(10):
        got = []
        for i in range(20):
            sdq.dequantize_fp4(*codes[i & 1], out=w)
            q = sdq.rmsnorm_quant(x, w[0])[0]
            sdq.dequantize_fp4(*codes[1 - (i & 1)], out=w)
            sdq.dequantize_fp4(*codes[i & 1], out=w)
            got.append((q, *sdq.rmsnorm_backward(gy, x, w[0], rstd)))
        torch.cuda.synchronize()
        for i, outs in enumerate(got):
            assert all(torch.equal(a, b) for a, b in zip(outs, want[i & 1])), i


def test_residual_sum_of_any_bits():
    """h = bf16(x + residual) for every kind of number: subnormals, both zeros, infinities, sums that overflow, ties."""
    gen = torch.Generator(device="cuda").manual_seed(8)
    rows, channels = 300, 1024
    x, r = (torch.randint(-32768, 32768, (rows, channels), generator=gen, device="cuda", dtype=torch.int16).view(torch.bfloat16)
            for _ in range(2))
    r[:100] = (x[:100].float() * (torch.randint(-4, 5, (100, channels), generator=gen, device="cuda") * 0.00390625)).bfloat16()
    r[100:150] = -x[100:150]
    small = torch.randint(0, 512, (2, 50, channels), generator=gen, device="cuda", dtype=torch.int16)     # below 2^-124
    x[150:200], r[150:200] = small[0].view(torch.bfloat16), -small[1].view(torch.bfloat16)
    for n in (rows, 3):
        _, _, h = sdq.rmsnorm_quant(x[-n:], torch.ones(channels, device="cuda"), r[-n:])
        want = (x[-n:].float() + r[-n:].float()).bfloat16()
        assert torch.equal(h.isnan(), want.isnan())
        assert torch.equal(h[~want.isnan()].view(torch.int16), want[~want.isnan()].view(torch.int16))


def _sums(m, n, k, scales, bytes_a, bytes_b, seed):
    """The product of random codes with scale bytes of two ranges, and its 64-bit form."""
    rng = np.random.default_rng(seed)
    out = []
    for rows, (lo, hi) in ((m, bytes_a), (n, bytes_b)):
        codes = rng.integers(0, 16, (rows, k))
        sb = rng.integers(lo, hi + 1, (rows, k // R.GROUP[scales]))
        t = torch.from_numpy(R.tiles(sb)).cuda()
        out.append((torch.from_numpy(R.pack(codes)).cuda(), t.view(torch.float8_e4m3fn) if scales == "e4m3" else t,
                    torch.from_numpy(R.values(codes, sb, scales)).cuda()))
    (a, a_s, av), (b, b_s, bv) = out
    return sdq.matmul_fp4(a, a_s, b, b_s, out_dtype=torch.float32).double(), av @ bv.t(), av.abs() @ bv.abs().t()


@pytest.mark.parametrize("m,n,k", [(7, 70, 320), (70, 300, 6240), (1700, 1600, 288)])
@pytest.mark.parametrize("scales,bytes_a,bytes_b", [("e8m0", (0, 6), (248, 254)), ("e8m0", (248, 254), (0, 6)), ("e8m0", (0, 4), (127, 130)),
                                                    ("e8m0", (180, 184), (170, 174)), ("e4m3", (0, 7), (0, 7)),
                                                    ("e4m3", (0, 9), (120, 126)), ("e4m3", (120, 126), (120, 126))])
def test_product_of_the_largest_and_smallest_scales(scales, bytes_a, bytes_b, m, n, k):
    """Scales from the ends of their formats, alone and against the other end: sums that fp32 holds are right.  The
    tolerance of test_fp4_gpu, and half of fp32's smallest step for each term where terms are subnormal."""
    got, want, mag = _sums(m, n, k, scales, bytes_a, bytes_b, m + k)
    assert float(mag.max()) < 3e38                         # (what the inputs are chosen for)
    assert ((got - want).abs() <= (k / 16 + 2) * 2.0 ** -23 * mag + k * 2.0 ** -150).all()
