"""Forms of the norm, its backward and the 4-bit product that a call's sizes choose, each at sizes past the others'
limits: products whose steps along k are shared by 2, 4 and 8 CTAs, backward calls past the few-rows kernel with
vectors that end anywhere in a row, and norms written over their inputs.

Tolerances, u = 2^-24.  The product's: test_fp4_gpu (a split adds the ranks' sums, 7 at most, and takes as many
steps out of each: k / 16 numbers and fewer than 2^-23 k / 16 in all).

Backward.  A row's dot: a thread adds four pairs a vector in each lane of a pair, then the two lanes, then its
vectors (four at most, or every 1024th of a longer row), then 10 levels of shuffles; the product before them is
rounded once: off by (4 + 1 + v + 10 + 1) u of the magnitudes, v the vectors a thread adds.  Its factor takes three
more roundings, n, gy w, the difference and the sum one each, and the result half a bf16 step:
|error| <= 2^-8 |grad_x| + (v + 24) u mag.

grad_weight.  n and the product are rounded once each.  Many rows: a thread adds ceil(rows / (parts rows_cta)) numbers
(148 parts at least, where there are as many rows), then up to 64 rows of a CTA, then ceil(592 / 32) partial sums,
then five levels.  Few rows: every 32nd row at the least, two levels, 32 warps.  Both: (ceil(rows / 32) + 96) u of
the magnitudes.
"""
from __future__ import annotations

import pytest
import torch

import swiglu_backward_int8_b200 as sdq
from tests import gpu_util as U
from tests import lowbit_ref as R
from tests.test_fp4_gpu import _product_check
from tests.test_norm_gpu import U24, _rows

pytestmark = pytest.mark.gpu


# (m, n, k): by the CTAs that share the steps on 148 multiprocessors, and the columns a CTA.  Some have several blocks
# of B or rows of tiles; ranks have 4 to 64 of the columns, some none.
SPLIT = [(128, 4096, 7168), (100, 3000, 6176),                                                       # 2, more than 32 columns
         (48, 300, 7168), (64, 4096, 7168), (100, 257, 6176), (128, 130, 7168), (300, 513, 7168), (70, 40, 12320),   # 4
         (90, 130, 24608), (128, 900, 30016),                                                       # 8
         (9, 7168, 4096), (20, 5632, 4096),                                                         # 2, up to 32 columns
         (5, 100, 800), (1, 4096, 7168),                                                            # 4
         (9, 200, 3360), (20, 140, 2080), (9, 200, 4096), (30, 129, 8192), (16, 129, 4128),         # 8
         (17, 100, 1344), (32, 260, 1056), (61, 7168, 4096)]                                        # 1


@pytest.mark.parametrize("scales", ["e8m0", "e4m3"])
@pytest.mark.parametrize("m,n,k", SPLIT)
def test_product_with_its_steps_shared(scales, m, n, k):
    _product_check(m, n, k, scales, torch.bfloat16, m + n + k)
    _product_check(m, n, k, scales, torch.float32, m * 3 + n + k)


@pytest.mark.parametrize("scales", ["e8m0", "e4m3"])
@pytest.mark.parametrize("m,n,k", [(60, 70, 6240), (20, 70, 2112)])
def test_product_with_its_steps_shared_nan_and_scales(scales, m, n, k):
    g = (0.0123, 3.7) if scales == "e4m3" else (None, None)
    _product_check(m, n, k, scales, torch.float32, 7, *g, nan_row=m - 2)


# ---- backward -----------------------------------------------------------------------

def _backward(rows, channels, dtype, with_gh, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    h, gy = _rows(gen, rows, channels, 1.5), _rows(gen, rows, channels, 0.3)
    gh = _rows(gen, rows, channels, 0.2) if with_gh else None
    w = (torch.randn(channels, generator=gen, device="cuda") + 1).to(dtype)
    rstd = torch.rsqrt(h.double().square().mean(1) + 1e-6).float()
    ws = U.Guarded((sdq.sdq_rmsnorm_backward_workspace_bytes(rows, channels),), torch.uint8, 0xA5)
    xb, wb = U.Guarded((rows, channels), torch.bfloat16, -1.0), U.Guarded((channels,), torch.float32, -1.0)
    got, gotw = sdq.rmsnorm_backward(gy, h, w, rstd, gh, grad_x=xb.t, grad_weight=wb.t, workspace=ws.t)
    torch.cuda.synchronize()
    assert ws.guards_intact() and xb.guards_intact() and wb.guards_intact()
    gx, gw, mag, magw = R.norm_backward(gy, h, w, rstd, gh)          # 64 bits, on the GPU
    v = 4 if channels <= 16384 else -(-channels // 8192)
    err = (got.double() - gx).abs()
    tol = 2.0 ** -8 * gx.abs() + (v + 24) * U24 * mag
    assert (err <= tol).all(), f"grad_x {(err / tol).max()}"
    err = (gotw.double() - gw).abs()
    assert (err <= (-(-rows // 32) + 96) * U24 * magw).all(), f"grad_weight {(err / magw).max() / U24}"
    return got.clone(), gotw.clone()


# past the few-rows kernel (2^22 values, 600 rows and 8 more a vector of 8 channels): two vectors a thread in several
# rows and in one, four with ragged ends, one with ragged lanes, rows read twice
BACKWARD = [(4000, 1408), (1900, 2400), (2700, 1552), (900, 6144), (800, 6160), (700, 8208), (400, 12304), (300, 16384),
            (1300, 48), (1500, 112), (1400, 128), (2100, 144), (300, 16400)]


@pytest.mark.parametrize("with_gh", [False, True])
@pytest.mark.parametrize("rows,channels", BACKWARD)
def test_backward_of_many_rows(rows, channels, with_gh):
    _backward(rows, channels, torch.bfloat16 if with_gh else torch.float32, with_gh, rows + channels)


@pytest.mark.parametrize("rows,channels", [(4000, 1408), (700, 6160), (900, 4096), (1500, 112), (300, 16400), (517, 7168)])
def test_backward_repeats_bit_for_bit(rows, channels):
    first = _backward(rows, channels, torch.bfloat16, True, 3)
    for _ in range(4):
        again = _backward(rows, channels, torch.bfloat16, True, 3)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


# ---- the norm -------------------------------------------------------------------------

@pytest.mark.parametrize("codes,scales,group", [("int8", "fp32", 0), ("e4m3", "fp32", 128), ("e2m1", "e4m3", 16)])
@pytest.mark.parametrize("rows,channels", [(5, 1408), (700, 1408), (2000, 64), (1203, 2400), (3, 16416), (170, 16416)])
def test_norm_over_its_inputs(codes, scales, group, rows, channels):
    """h written over x and over residual gives the bits of a call with an h of its own."""
    gen = torch.Generator(device="cuda").manual_seed(rows + channels)
    x, r = _rows(gen, rows, channels, 1.0, pad=16), _rows(gen, rows, channels, 1.0, pad=16)
    w = torch.rand(channels, generator=gen, device="cuda") - 0.5

    def call(over):
        a, b = (torch.empty_strided(t.shape, t.stride(), dtype=t.dtype, device="cuda").copy_(t) for t in (x, r))
        y, rstd = torch.empty(rows, channels, dtype=torch.bfloat16, device="cuda"), torch.empty(rows, device="cuda")
        q = torch.zeros(rows, channels // (2 if codes == "e2m1" else 1), device="cuda",
                        dtype={"int8": torch.int8, "e4m3": torch.float8_e4m3fn, "e2m1": torch.uint8}[codes])
        s = torch.zeros(sdq.fp4_scale_shape(rows, channels, scales), device="cuda", dtype=torch.uint8).view(torch.float8_e4m3fn) \
            if codes == "e2m1" else torch.zeros(rows, -(-channels // (group or channels)), device="cuda")
        h = {"x": a, "residual": b, None: torch.empty(rows, channels, dtype=torch.bfloat16, device="cuda")}[over]
        sdq.rmsnorm_quant(a, w, b, 1e-6, group, codes=codes, scales=scales, q=q, s=s, h=h, y=y, rstd=rstd)
        return h, q, s, y, rstd

    want = call(None)
    assert torch.equal(want[0], (x.float() + r.float()).bfloat16())
    for over in ("x", "residual"):
        for a, b in zip(call(over), want):
            assert torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8)), over


@pytest.mark.parametrize("rows,channels", [(16384, 7168), (4099, 1408), (37, 4096), (170, 16416)])
def test_norm_repeats_bit_for_bit(rows, channels):
    gen = torch.Generator(device="cuda").manual_seed(rows)
    x, r = _rows(gen, rows, channels, 0.7), _rows(gen, rows, channels, 1.5)
    w = (1 + 0.2 * torch.randn(channels, generator=gen, device="cuda")).bfloat16()
    first = [t.clone() for t in sdq.rmsnorm_quant(x, w, r, codes="e4m3")]
    for _ in range(8):
        for a, b in zip(sdq.rmsnorm_quant(x, w, r, codes="e4m3"), first):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("rows,channels", [(3, 7168), (1, 48), (700, 1408), (4000, 96), (900, 16384), (2, 16400), (3, 1 << 17)])
def test_norm_within_the_bound_of_its_order_of_sums(rows, channels):
    """A thread adds the squares of 16 channels, eight in each lane of a pair, then the two lanes, then its vectors (one,
    or every 1024th of a row past 16384 channels), then ten levels of shuffles: (18 + v) u of the sum.  1 / channels,
    the mean and eps round once each, half of all that reaches rstd; the root's approximation with a Newton step adds
    1.5 u (and the square of 2^-22), the two products of y one each, a group's scale one more."""
    gen = torch.Generator(device="cuda").manual_seed(rows + channels)
    x = _rows(gen, rows, channels, 1.3)
    w = torch.randn(channels, generator=gen, device="cuda")
    rstd = torch.empty(rows, device="cuda")
    _, s, _ = sdq.rmsnorm_quant(x, w, group_size=32, rstd=rstd)
    d = x.double()
    want = 1 / (d.square().mean(1) + 1e-6).sqrt()
    v = 1 if channels <= 16384 else -(-channels // 16384)
    bound = (21 + v) / 2 + 1.6
    assert ((rstd.double() / want - 1).abs() <= bound * U24).all(), float((rstd.double() / want - 1).abs().max() / U24)
    y = torch.nn.functional.pad(d * want[:, None] * w.double(), (0, -channels % 32))
    top = y.abs().reshape(rows, -1, 32).amax(2) / 127
    assert ((s.double() / top - 1).abs() <= (bound + 3.1) * U24).all(), float((s.double() / top - 1).abs().max() / U24)
