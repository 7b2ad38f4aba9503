"""The 4-bit quantizer and the product of 4-bit operands on the GPU against the
plain forms.

The quantizer's codes and scales are compared for equality: power-of-two scales
leave no rounding but the code's, and with E4M3 scales every quotient is the
correctly rounded fp32 one on both sides.

The product.  Every term (two codes, two scales) is exact in fp32.  The
accumulator adds k / 16 sums of 16 terms, each addition off by at most 2^-23 of the
magnitudes added so far (whether it rounds or cuts): |error| <= (k / 16 + 2) 2^-23
sum |a b|, plus 2^-8 of the result where that is bf16.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

import swiglu_backward_int8_b200 as sdq
from tests import gpu_util as U
from tests import lowbit_ref as R

pytestmark = pytest.mark.gpu
_DT = {"e8m0": torch.float8_e8m0fnu, "e4m3": torch.float8_e4m3fn}


def _x(seed, rows, channels, sigma=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(rows, channels, generator=g, device="cuda") * sigma
    x = torch.where(torch.rand(rows, channels, generator=g, device="cuda") < 0.01, x * 30, x)
    return x.bfloat16()


def _quantize(x, scales, axis, g=None):
    """The call on guarded, prefilled outputs; returns {"rows": (codes, tiles), "columns": ...} as numpy."""
    rows, channels = x.shape
    padded = -(-rows // 32) * 32
    out, kw = {}, {}
    for name, r, k, sfx in (("rows", rows, channels, ""), ("columns", channels, padded, "_t")):
        if axis in (name, "both"):
            q = U.Guarded((r, k // 2), torch.uint8, 0x5A)
            s = U.Guarded(sdq.fp4_scale_shape(r, k, scales), torch.uint8, 0xA5)
            kw["q" + sfx], kw["s" + sfx] = q.t, s.t.view(_DT[scales])
            out[name] = (q, s)
    sdq.quantize_fp4(x, scales, axis, global_scale=g, **kw)
    torch.cuda.synchronize()
    for q, s in out.values():
        assert q.guards_intact() and s.guards_intact()
    return {n: (q.t.cpu().numpy(), s.t.cpu().numpy()) for n, (q, s) in out.items()}


def _check(x, scales, axis, g=None, where=""):
    got = _quantize(x, scales, axis, g)
    xf = x.float().cpu().numpy()
    gf = 1.0 if g is None else float(g.cpu())
    for name, (q, s) in got.items():
        v = xf
        if name == "columns":
            v = np.zeros((-(-xf.shape[0] // 32) * 32, xf.shape[1]), np.float32)
            v[:xf.shape[0]] = xf
            v = np.ascontiguousarray(v.T)
        codes, sb = R.quantize_fp4(v, scales, gf)
        flat = s.reshape(-1)
        groups = sb.shape[1]
        full = R.tile_index(v.shape[0], -(-groups // 4) * 4)
        assert np.array_equal(flat[full[:, :groups]], sb), f"{where} {name}: scales"
        assert (flat[full[:, groups:]] == 0).all(), f"{where} {name}: padding groups"
        rest = np.ones(flat.size, bool)
        rest[full] = False
        assert (flat[rest] == 0xA5).all(), f"{where} {name}: rows past the last were written"
        assert np.array_equal(R.unpack(q), codes), f"{where} {name}: {(R.unpack(q) != codes).sum()} codes"


@pytest.mark.parametrize("scales", ["e8m0", "e4m3"])
@pytest.mark.parametrize("rows,channels", [(1, 32), (3, 64), (31, 96), (32, 160), (33, 256), (127, 288), (129, 32), (130, 1056),
                                           (300, 544), (19, 7168)])
def test_quantize_both_axes(scales, rows, channels):
    x = _x(rows + channels, rows, channels)
    _check(x, scales, "both", None, f"{rows}x{channels}")
    g = torch.tensor([float((x.float().abs().max() / 2688).bfloat16())], device="cuda") if scales == "e4m3" else None
    _check(x, scales, "rows", g, f"{rows}x{channels}")
    _check(x, scales, "columns", g, f"{rows}x{channels}")


def test_quantize_any_global_scale():
    x = _x(4, 200, 512)
    for g in (0.00731, 1.9e-3, 3.3, 1e-30, 1e30):
        _check(x, "e4m3", "both", torch.tensor([g], device="cuda"), f"g = {g}")


def test_quantize_values_and_global_scales_far_apart():
    """Group maxima over the global scale that overflow or vanish: the scale saturates at 448 or is 2^-9."""
    for top in (1e-38, 1e-27, 1e-19, 1e-17, 1e15, 1e17, 1e19, 1e25, 3e38):
        x = torch.cat([(_x(5, 40, 64).float().clamp(-30, 30) / 32 * top * f) for f in (1, 1e-3, 0.04)]).bfloat16()
        for g in (1e-37, 1e-25, 1e-18, 1.2e-18, 1e-15, 1.0, 1e15, 1.1e18, 1e20, 1e37):
            _check(x, "e4m3", "both", torch.tensor([g], device="cuda"), f"values to {top}, g = {g}")


@pytest.mark.parametrize("scales", ["e8m0", "e4m3"])
def test_quantize_ties_and_range_ends(scales):
    """Every tie of the codes at several scales, the largest and the smallest bf16 numbers, zeros of both signs."""
    ties = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 0.125, 5.75])
    rows = [ties * s for s in (1.0, 2.0 ** -120, 2.0 ** 120, 1.5, 7.0, -1.0, 2.0 ** -130, 0.0, -0.0)]
    rows += [np.full(16, 3.3895e38), np.full(16, 2.0 ** -133), np.linspace(0, 2.0 ** -126, 16)]
    x = torch.tensor(np.array([np.concatenate([r, -r[::-1]]) for r in rows]), dtype=torch.float64).float().bfloat16().cuda()
    _check(x, scales, "both", None, "ties")
    if scales == "e4m3":
        for g in (1.0 / 448, 0.25, 3.0):
            _check(x, scales, "rows", torch.tensor([g], device="cuda"), f"ties, g = {g}")


@pytest.mark.parametrize("scales", ["e8m0", "e4m3"])
def test_quantize_non_finite_groups_read_back_as_nan(scales):
    x = _x(9, 70, 128)
    x[3, 5], x[40, 100], x[69, 0] = float("nan"), float("inf"), float("-inf")
    _check(x, scales, "both")
    q, s = sdq.quantize_fp4(x, scales)
    back = sdq.dequantize_fp4(q, s).isnan().cpu()
    n = R.GROUP[scales]
    want = torch.zeros(70, 128, dtype=torch.bool)
    for r, c in ((3, 5), (40, 100), (69, 0)):
        want[r, c // n * n:c // n * n + n] = True
    assert torch.equal(back, want)


def test_quantize_strided():
    wide = _x(10, 50, 200)
    x = wide[:, 32:192]
    a, b = sdq.quantize_fp4(x, axis="both"), sdq.quantize_fp4(x.contiguous(), axis="both")
    assert all(torch.equal(u.view(torch.uint8)[..., :1], v.view(torch.uint8)[..., :1]) for u, v in zip(a[::2], b[::2]))
    q, qt = (torch.full(n, 0x77, dtype=torch.uint8, device="cuda") for n in ((50, 112), (160, 48)))
    sdq.quantize_fp4(x, axis="both", q=q[:, :80], q_t=qt[:, :32])
    assert torch.equal(q[:, :80], a[0]) and torch.equal(qt[:, :32], a[2])
    assert (q[:, 80:] == 0x77).all() and (qt[:, 32:] == 0x77).all()


@pytest.mark.parametrize("scales,n", [("e8m0", 32), ("e4m3", 16)])
def test_quantize_non_finite_values_in_every_place_of_a_group(scales, n):
    """Along both axes a group reads back as NaN where it holds a NaN or an infinity of either sign, nowhere else."""
    gen = torch.Generator(device="cuda").manual_seed(11)
    x = torch.randn(256, 224, generator=gen, device="cuda").bfloat16()
    bits = x.view(torch.int16)
    for i, b in enumerate((0x7FC0, -0x40, 0x7F80, -0x80, 0x7F81, -1)):       # NaN, infinity, NaN of other bits
        k = torch.arange(i, 224, 41 + i, device="cuda")
        bits[(k * 7 + 29 * i) % 256, k] = b
    bad = ~x.isfinite()
    q, s, qt, st = sdq.quantize_fp4(x, scales, "both")
    want = bad.view(256, -1, n).any(2).repeat_interleave(n, 1)
    assert torch.equal(sdq.dequantize_fp4(q, s).isnan(), want)
    want = bad.t().reshape(224, -1, n).any(2).repeat_interleave(n, 1)
    assert torch.equal(sdq.dequantize_fp4(qt, st).isnan(), want)
    for axis, pair in (("rows", (q, s)), ("columns", (qt, st))):
        got = sdq.quantize_fp4(x, scales, axis)
        assert torch.equal(sdq.dequantize_fp4(*got).isnan(), sdq.dequantize_fp4(*pair).isnan())


@pytest.mark.parametrize("scales", ["e8m0", "e4m3"])
@pytest.mark.parametrize("rows,k", [(1, 32), (129, 96), (200, 2080)])
def test_dequantize_every_code_and_scale(scales, rows, k):
    rng = np.random.default_rng(rows)
    q = rng.integers(0, 256, (rows, k // 2)).astype(np.uint8)
    sb = rng.integers(0, 256, (rows, k // R.GROUP[scales]))
    g = torch.tensor([0.037], device="cuda") if scales == "e4m3" else None
    out = U.Guarded((rows, k), torch.bfloat16, -1.0)
    sdq.dequantize_fp4(torch.from_numpy(q).cuda(), torch.from_numpy(R.tiles(sb)).cuda().view(_DT[scales]), g, out=out.t)
    torch.cuda.synchronize()
    assert out.guards_intact()
    unit = R.scale_values(sb, scales).astype(np.float32)
    if g is not None:
        unit = unit * np.float32(0.037)
    with np.errstate(all="ignore"):
        want = torch.from_numpy(R.e2m1_value(R.unpack(q)).astype(np.float32) * np.repeat(unit, R.GROUP[scales], 1)).bfloat16()
    got = out.t.cpu()
    assert torch.equal(torch.nan_to_num(got.float(), 7), torch.nan_to_num(want.float(), 7))
    assert torch.equal(got.isnan(), want.isnan())


def test_quantize_empty_and_refusals():
    x = torch.zeros(0, 64, dtype=torch.bfloat16, device="cuda")
    q, s, qt, st = sdq.quantize_fp4(x, axis="both")
    assert q.shape == (0, 32) and s.shape == (0, 1, 512) and qt.shape == (64, 0) and st.numel() == 0
    assert sdq.dequantize_fp4(q, s).shape == (0, 64)
    x = torch.zeros(4, 64, dtype=torch.bfloat16, device="cuda")
    q, s = sdq.quantize_fp4(x)
    one = torch.ones(1, device="cuda")
    for kw in (dict(scales="fp32"), dict(axis="both ways"), dict(q_t=q), dict(axis="columns", q=q), dict(s=s[:, :, :256]),
               dict(s=s, scales="e4m3"), dict(global_scale=one), dict(scales="e4m3", global_scale=one.double()),
               dict(scales="e4m3", global_scale=one.cpu()), dict(q=q[:3]), dict(q=q.int())):
        with pytest.raises(ValueError):
            sdq.quantize_fp4(x, **kw)
    for bad in (x[:, :48], x.half(), x[0]):
        with pytest.raises(ValueError):
            sdq.quantize_fp4(bad)
    for call in (lambda: sdq.dequantize_fp4(q[:, :24], s), lambda: sdq.dequantize_fp4(q, s, one),
                 lambda: sdq.dequantize_fp4(q, s, out=x.half()), lambda: sdq.matmul_fp4(q, s, q[:, :16], s),
                 lambda: sdq.matmul_fp4(q, s, q, s.view(torch.uint8).view(torch.float8_e4m3fn)),
                 lambda: sdq.matmul_fp4(q, s, q, s, out=x), lambda: sdq.matmul_fp4(q, s, q, s, out_dtype=torch.half),
                 lambda: sdq.matmul_fp4(q, s, q, s, a_global=one),
                 lambda: sdq.matmul_fp4(q, s, q, s, out=torch.zeros(4, 4, device="cuda"), out_dtype=torch.bfloat16)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(sdq.SdqError):                              # code rows that do not start on 16 bytes
        sdq.dequantize_fp4(torch.zeros(4, 40, dtype=torch.uint8, device="cuda")[:, :32], s)


# ---- the product ----------------------------------------------------------------

def _operand(rng, rows, k, scales, spread=3, nan_row=None):
    """Random codes and scales: (codes uint8, tiles on the GPU with junk in the rows past the last, values fp64)."""
    codes = rng.integers(0, 16, (rows, k))
    groups = k // R.GROUP[scales]
    base = 127 if scales == "e8m0" else 0x38
    step = 1 if scales == "e8m0" else 8
    sb = base + rng.integers(-spread * step, spread * step + 1, (rows, groups))
    if nan_row is not None:
        sb[nan_row, groups // 2] = 255 if scales == "e8m0" else 0x7F
    t = R.tiles(sb, fill=0xFF)                       # rows past the last: NaN scales, not used
    t.reshape(-1)[R.tile_index(rows, -(-groups // 4) * 4)[:, groups:]] = 0
    return (torch.from_numpy(R.pack(codes)).cuda(), torch.from_numpy(t).cuda().view(_DT[scales]),
            torch.from_numpy(R.values(codes, sb, scales)))


def _product_check(m, n, k, scales, dtype, seed, ga=None, gb=None, **kw):
    rng = np.random.default_rng(seed)
    a, a_s, av = _operand(rng, m, k, scales, **kw)
    b, b_s, bv = _operand(rng, n, k, scales)
    out = U.Guarded((m, n), dtype, -77.0)
    tg = lambda v: None if v is None else torch.tensor([v], device="cuda")  # noqa: E731
    got = sdq.matmul_fp4(a, a_s, b, b_s, a_global=tg(ga), b_global=tg(gb), out=out.t)
    torch.cuda.synchronize()
    assert sdq.sdq_device_status() == 0
    assert out.guards_intact()
    alpha = float(np.float32(ga or 1) * np.float32(gb or 1))
    want, mag = (av @ bv.t()) * alpha, (av.abs() @ bv.abs().t()) * abs(alpha)
    got = got.cpu().double()
    tol = (k / 16 + 2) * 2.0 ** -23 * mag + (2.0 ** -8 * want.abs() if dtype == torch.bfloat16 else 0)
    bad = ~((got - want).abs() <= tol) & ~(got.isnan() & want.isnan())
    assert not bad.any(), f"{m}x{n}x{k} {scales} {dtype}: {int(bad.sum())} off, first {bad.nonzero()[0].tolist()}, " \
        f"largest {((got - want).abs() / tol.clamp(min=1e-30)).nan_to_num().max():.3g} of the tolerance"


SIZES = [(1, 1, 32), (1, 130, 64), (2, 257, 96), (5, 7, 288), (16, 384, 512), (17, 100, 800), (33, 129, 256), (64, 640, 1056),
         (65, 128, 2080), (127, 300, 160), (128, 256, 1024), (129, 1, 32), (130, 7, 320), (200, 129, 544), (257, 255, 256),
         (300, 513, 768), (515, 260, 4128), (1, 2048, 7168), (40, 1000, 5152)]


@pytest.mark.parametrize("scales", ["e8m0", "e4m3"])
@pytest.mark.parametrize("m,n,k", SIZES)
def test_product(scales, m, n, k):
    _product_check(m, n, k, scales, torch.bfloat16, m + n + k)
    _product_check(m, n, k, scales, torch.float32, m * 3 + n + k)


def test_product_scales_per_tensor():
    for m in (3, 200):
        _product_check(m, 77, 256, "e4m3", torch.float32, 1, 0.0123, 3.7)
        _product_check(m, 77, 256, "e4m3", torch.bfloat16, 2, None, 1e-3)


@pytest.mark.parametrize("scales", ["e8m0", "e4m3"])
@pytest.mark.parametrize("m,n,k", [(9, 70, 320), (200, 300, 512)])
def test_product_whole_numbers_are_exact(scales, m, n, k):
    """Scales of 1 and integer codes: every partial sum is a whole number below 2^24."""
    rng = np.random.default_rng(k)
    ints = np.array([0, 2, 4, 5, 6, 7, 8, 10, 12, 13, 14, 15])
    ca, cb = ints[rng.integers(0, 12, (m, k))], ints[rng.integers(0, 12, (n, k))]
    one = 127 if scales == "e8m0" else 0x38
    groups = k // R.GROUP[scales]
    t = lambda r: torch.from_numpy(R.tiles(np.full((r, groups), one))).cuda().view(_DT[scales])  # noqa: E731
    got = sdq.matmul_fp4(torch.from_numpy(R.pack(ca)).cuda(), t(m), torch.from_numpy(R.pack(cb)).cuda(), t(n),
                         out_dtype=torch.float32)
    assert np.array_equal(got.cpu().numpy(), R.e2m1_value(ca) @ R.e2m1_value(cb).T)


@pytest.mark.parametrize("m", [20, 150])
def test_product_nan_stays_in_its_row(m):
    _product_check(m, 140, 288, "e8m0", torch.bfloat16, 5, nan_row=m - 3)
    _product_check(m, 140, 288, "e4m3", torch.bfloat16, 5, nan_row=m - 3)


@pytest.mark.parametrize("m", [6, 140])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_product_strided(m, dtype):
    """Padded code rows, and an output whose rows start on no particular boundary."""
    rng = np.random.default_rng(m)
    n, k = 150, 352
    a, a_s, _ = _operand(rng, m, k, "e8m0")
    b, b_s, _ = _operand(rng, n, k, "e8m0")
    want = sdq.matmul_fp4(a, a_s, b, b_s, out_dtype=dtype)
    wide_a, wide_b = (torch.full((r, 208), 0x77, dtype=torch.uint8, device="cuda") for r in (m, n))
    wide_a[:, 16:192], wide_b[:, 16:192] = a, b
    out = torch.full((m, n + 7), 9.0, dtype=dtype, device="cuda")
    sdq.matmul_fp4(wide_a[:, 16:192], a_s, wide_b[:, 16:192], b_s, out=out[:, 3:n + 3])
    assert torch.equal(out[:, 3:n + 3], want)
    assert (out[:, :3] == 9).all() and (out[:, n + 3:] == 9).all()


def test_product_empty():
    q = torch.zeros(4, 32, dtype=torch.uint8, device="cuda")
    s = torch.zeros(sdq.fp4_scale_shape(4, 64), dtype=torch.uint8, device="cuda")
    e, es = q[:0], torch.zeros(0, 1, 512, dtype=torch.uint8, device="cuda")
    assert sdq.matmul_fp4(e, es, q, s).shape == (0, 4) and sdq.matmul_fp4(q, s, e, es).shape == (4, 0)


def test_product_large():
    """Several waves of tiles, against a 64-bit product on the GPU."""
    g = torch.Generator(device="cuda").manual_seed(2)
    for scales, (m, n, k) in (("e8m0", (3000, 4100, 1056)), ("e4m3", (2500, 5000, 544))):
        x = torch.randn(m, k, generator=g, device="cuda").bfloat16()
        w = torch.randn(n, k, generator=g, device="cuda").bfloat16()
        (a, a_s), (b, b_s) = sdq.quantize_fp4(x, scales), sdq.quantize_fp4(w, scales)
        av, bv = sdq.dequantize_fp4(a, a_s).double(), sdq.dequantize_fp4(b, b_s).double()
        got = sdq.matmul_fp4(a, a_s, b, b_s).double()
        want, mag = av @ bv.t(), av.abs() @ bv.abs().t()
        # the values read back are bf16: exact for E8M0 scales and for E4M3 ones (four and three bits)
        assert ((got - want).abs() <= (k / 16 + 2) * 2.0 ** -23 * mag + 2.0 ** -8 * want.abs()).all()


# ---- the product with more tiles than the device takes at once ---------------------
#
# (the form that two multiprocessors share: 256 x 256 outputs, a persistent grid)

def _gpu_operand(rng, rows, k, scales, **kw):
    q, s, v = _operand(rng, rows, k, scales, **kw)
    return q, s, v.cuda()


@pytest.mark.parametrize("scales", ["e8m0", "e4m3"])
@pytest.mark.parametrize("m,n,k", [(1665, 1537, 32), (1537, 1665, 96), (1700, 1800, 288), (2561, 1280, 544), (130, 20000, 160),
                                   (20000, 130, 2080), (1664, 1664, 1312)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_product_of_many_tiles(scales, m, n, k, dtype):
    rng = np.random.default_rng(m + k)
    a, a_s, av = _gpu_operand(rng, m, k, scales, nan_row=m - 2)
    b, b_s, bv = _gpu_operand(rng, n, k, scales)
    ga, gb = (torch.tensor([0.37], device="cuda"), None) if scales == "e4m3" else (None, None)
    out = U.Guarded((m, n), dtype, -77.0)
    sdq.matmul_fp4(a, a_s, b, b_s, a_global=ga, b_global=gb, out=out.t)
    torch.cuda.synchronize()
    assert sdq.sdq_device_status() == 0 and out.guards_intact()
    alpha = 1.0 if ga is None else float(ga.double())
    want, mag = (av @ bv.t()) * alpha, (av.abs() @ bv.abs().t()) * alpha
    got = out.t.double()
    tol = (k / 16 + 2) * 2.0 ** -23 * mag + (2.0 ** -8 * want.abs() if dtype == torch.bfloat16 else 0)
    assert ((got - want).abs() <= tol)[torch.arange(m) != m - 2].all()
    assert got[m - 2].isnan().all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n", [1672, 1665])
def test_product_of_many_tiles_strided_and_exact(dtype, n):
    """Whole numbers (exact in fp32, and in bf16 up to 256), rows of the output that start on 16 bytes and that do not."""
    rng = np.random.default_rng(n)
    m, k = 1700, 64
    ints = np.array([0, 2, 4, 10, 12])                     # 0, 1, 2, -1, -2: sums within 64 * 4 = 256
    ca, cb = ints[rng.integers(0, 5, (m, k))], ints[rng.integers(0, 5, (n, k))]
    t = lambda r: torch.from_numpy(R.tiles(np.full((r, 2), 127))).cuda().view(_DT["e8m0"])  # noqa: E731
    out = torch.full((m, n + 8), 9.0, dtype=dtype, device="cuda")
    view = out[:, 8:] if n == 1672 else out[:, 3:n + 3]
    sdq.matmul_fp4(torch.from_numpy(R.pack(ca)).cuda(), t(m), torch.from_numpy(R.pack(cb)).cuda(), t(n), out=view)
    want = torch.from_numpy(R.e2m1_value(ca) @ R.e2m1_value(cb).T).cuda()
    assert torch.equal(view.double(), want)
    rest = torch.ones_like(out, dtype=torch.bool)
    rest[:, 8:] = n != 1672
    if n != 1672:
        rest[:, 3:n + 3] = False
    assert (out[rest] == 9).all()
