"""The quantizing RMS norm and its backward on the GPU against the 64-bit forms.

Tolerances.  y = h * rstd * weight in fp32: the sum of squares adds at most
`seq` numbers one after another in a thread, then 10 levels of shuffles, so it
is off by (seq + 10) 2^-24 of itself at most (all terms are positive), the mean,
eps, root and reciprocal by 4 roundings, half of which reach rstd, and two
products follow: y is off by D = ((seq + 14) / 2 + 4) 2^-24 of itself.
A scale is off by D + 2^-24, its group's largest value being off by D; a code
times its scale by half a step of the code, plus D and 3 2^-24 of the value
(the reciprocal, the product).  A power-of-two scale is equal, unless amax / Qmax
is within D of a power of two.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

import swiglu_backward_int8_b200 as sdq
from tests import gpu_util as U
from tests import lowbit_ref as R

pytestmark = pytest.mark.gpu
U24 = 2.0 ** -24


def _rows(gen, rows, channels, sigma, pad=0):
    t = (torch.randn(rows, channels + pad, generator=gen, device="cuda") * sigma).bfloat16()
    return t[:, :channels]


def _seq(channels):
    """Numbers a thread adds one after another: 8 a vector, up to 4 vectors, or the whole strip of a long row."""
    return 32 if channels <= 32768 else 8 * -(-channels // 8192)


def _half_step(a, codes):
    """Half the spacing of the codes at magnitude a (in units of the scale)."""
    if codes == "int8":
        return np.full_like(a, 0.5)
    if codes == "e4m3":
        e = np.floor(np.log2(np.maximum(a * (1 + 2.0 ** -20), 2.0 ** -6)))
        return 2.0 ** (e - 4)
    return np.where(a < 2, 0.25, np.where(a < 4, 0.5, 1.0))


def _check_codes(y, q, s, codes, scales, group, g, delta, where):
    """q: code values; s: scale values, one a group; y: fp64 rows."""
    rows, channels = y.shape
    n = group or channels
    pad = -channels % n
    yg = np.pad(y, ((0, 0), (0, pad))).reshape(rows, -1, n)
    qg = np.pad(q, ((0, 0), (0, pad))).reshape(rows, -1, n)
    amax = np.abs(yg).max(2)
    t = amax / R.QMAX[codes] / (g if scales == "e4m3" else 1)
    if scales == "fp32":
        want = np.where(amax > 0, np.maximum(t, 2.0 ** -149), 1)
        off = np.abs(s - want) > (delta + U24) * want + 2.0 ** -149
        assert not off.any(), f"{where}: {off.sum()} scales off, by {np.abs(s / want - 1).max()}"
    elif scales == "e8m0":
        k = R.pow2_ceil_exp(np.where(amax > 0, t, 1.0))
        lo, hi = (R.pow2_ceil_exp(np.where(amax > 0, t * f, 1.0)) for f in (1 - delta, 1 + delta))
        assert ((np.ldexp(1.0, lo) <= s) & (s <= np.ldexp(1.0, hi))).all(), f"{where}: scales"
        assert (s == np.ldexp(1.0, k)).mean() > 0.99
    else:
        lo, hi = (np.where(amax > 0, np.maximum(R.E4M3[R.e4m3_byte(t * f)], 2.0 ** -9), 1.0)
                  for f in (1 - delta - 2 * U24, 1 + delta + 2 * U24))
        assert ((lo <= s) & (s <= hi)).all(), f"{where}: scales"
    unit = (s * (g if scales == "e4m3" else 1))[..., None]
    a = np.abs(yg) / unit
    tol = _half_step(a, codes) * unit + (delta + 3 * U24) * np.abs(yg)
    sat = np.maximum(np.abs(yg) - R.QMAX[codes] * unit, 0)     # only E4M3 scales can fall short of amax / 6
    err = np.abs(qg * unit - yg)
    assert (err <= tol + sat).all(), f"{where}: codes off by {(err - tol - sat).max()} at {np.argmax(err - tol - sat)}"
    if scales != "e4m3":
        assert (sat <= (delta + 2 * U24) * np.abs(yg)).all()


def _run(x, w, residual, codes, scales, group, g=None, eps=1e-6, inplace=False, want_y=True):
    """One call on guarded outputs; every output checked against the 64-bit form."""
    rows, channels = x.shape
    e2m1 = codes == "e2m1"
    qd = {"int8": torch.int8, "e4m3": torch.uint8, "e2m1": torch.uint8}[codes]
    qb = U.Guarded((rows, channels // 2 if e2m1 else channels), qd, 0x55)
    groups = -(-channels // (group or channels))
    if e2m1:
        sb = U.Guarded(sdq.fp4_scale_shape(rows, channels, scales), torch.uint8, 0xA5)
    else:
        sb = U.Guarded((rows, groups), torch.float32 if scales == "fp32" else torch.uint8,
                       float("nan") if scales == "fp32" else 0xA5)
    yb, rb = U.Guarded((rows, channels), torch.bfloat16, -1.0), U.Guarded((rows,), torch.float32, -1.0)
    xc, wc = x.cpu(), w.cpu()
    rc = None if residual is None else residual.cpu()
    h = None if residual is None else (residual if inplace else torch.empty_like(x))
    qt = qb.t.view(torch.float8_e4m3fn) if codes == "e4m3" else qb.t
    st = sb.t if not (e2m1 and scales == "e4m3") else sb.t.view(torch.float8_e4m3fn)
    q2, s2, h2 = sdq.rmsnorm_quant(x, w, residual, eps, group, codes=codes, scales=scales, q=qt, s=st, h=h,
                                   y=yb.t if want_y else None, rstd=rb.t, global_scale=g)
    torch.cuda.synchronize()
    assert q2.data_ptr() == qt.data_ptr() and s2.data_ptr() == st.data_ptr()
    assert all(b.guards_intact() for b in (qb, sb, yb, rb))
    where = f"{rows}x{channels} {codes}/{scales} group {group}"
    want_h, y, rstd = R.norm(xc, rc, wc, eps)
    assert torch.equal(h2.cpu(), want_h), f"{where}: h"
    delta = ((_seq(channels) + 14) / 2 + 4) * U24
    r = rb.t.cpu().double()
    assert ((r - rstd).abs() <= delta * rstd).all(), f"{where}: rstd"
    y = y.numpy()
    if want_y:
        yy = yb.t.cpu().double().numpy()
        assert (np.abs(yy - y) <= (2.0 ** -8 + delta) * np.abs(y) + 2.0 ** -134).all(), f"{where}: y"
    qn = qb.t.cpu().numpy()
    if e2m1:
        qv = R.e2m1_value(R.unpack(qn))
        flat = sb.t.cpu().numpy().reshape(-1)
        idx = R.tile_index(rows, groups)
        sv = R.scale_values(flat[idx], scales)
        rest = np.ones(flat.size, bool)
        rest[R.tile_index(rows, -(-groups // 4) * 4)] = False
        assert (flat[rest] == 0xA5).all(), f"{where}: rows past the last were written"
        pad = R.tile_index(rows, -(-groups // 4) * 4)[:, groups:]
        assert (flat[pad] == 0).all(), f"{where}: padding groups are zero"
    else:
        qv = qn.astype(np.float64) if codes == "int8" else R.E4M3[qn]
        sn = sb.t.cpu().numpy()
        sv = sn.astype(np.float64) if scales == "fp32" else R.scale_values(sn, "e8m0")
    _check_codes(y, qv, sv, codes, scales, group, 1.0 if g is None else float(g.cpu()), delta, where)
    return qn, sb.t.cpu().numpy()


FORMATS = [("int8", "fp32", 128), ("int8", "e8m0", 64), ("int8", "fp32", 0), ("e4m3", "fp32", 256), ("e4m3", "e8m0", 32),
           ("e4m3", "e8m0", 0), ("e2m1", "e8m0", 32), ("e2m1", "e4m3", 16)]


@pytest.mark.parametrize("codes,scales,group", FORMATS)
@pytest.mark.parametrize("rows,channels", [(1, 32), (3, 96), (7, 288), (150, 64), (300, 1056), (5, 7168), (260, 4096)])
def test_norm_formats_and_sizes(codes, scales, group, rows, channels):
    gen = torch.Generator(device="cuda").manual_seed(rows * 7 + channels)
    x, r = _rows(gen, rows, channels, 0.7), _rows(gen, rows, channels, 2.0)
    w = torch.randn(channels, generator=gen, device="cuda") + 0.5
    g = torch.tensor([0.0137], device="cuda") if scales == "e4m3" else None
    _run(x, w.bfloat16(), r, codes, scales, group, g)
    _run(x, w, None, codes, scales, group, None, want_y=False)


@pytest.mark.parametrize("codes,scales,group", [("int8", "fp32", 128), ("e4m3", "e8m0", 256), ("int8", "fp32", 0)])
@pytest.mark.parametrize("rows,channels", [(2, 16), (9, 48), (170, 1040), (4, 8208), (2, 16400), (3, 32784), (2, 1 << 17)])
def test_norm_ragged_and_long_rows(codes, scales, group, rows, channels):
    """Channels that end inside a group, and rows longer than a CTA's registers hold."""
    gen = torch.Generator(device="cuda").manual_seed(rows + channels)
    _run(_rows(gen, rows, channels, 1.0), torch.rand(channels, generator=gen, device="cuda") - 0.5,
         _rows(gen, rows, channels, 1.0), codes, scales, group)


@pytest.mark.parametrize("rows", [4, 400])
def test_norm_long_rows_e2m1(rows):
    gen = torch.Generator(device="cuda").manual_seed(rows)
    for channels in (32800, 2080) if rows == 4 else (2080,):
        for scales, n in R.GROUP.items():
            _run(_rows(gen, rows, channels, 1.0), torch.ones(channels, device="cuda"), None, "e2m1", scales, n)


def test_norm_strided_and_in_place():
    gen = torch.Generator(device="cuda").manual_seed(5)
    x, r = _rows(gen, 33, 272, 1.0, pad=24), _rows(gen, 33, 272, 1.0, pad=8)
    w = torch.rand(272, generator=gen, device="cuda").bfloat16()
    beyond = torch.as_strided(r, (33, 8), (280, 1), 272).clone()
    _run(x, w, r, "int8", "fp32", 128, inplace=True)            # h written over residual's rows
    assert torch.equal(torch.as_strided(r, (33, 8), (280, 1), 272), beyond)
    q = torch.full((33, 320), 7, dtype=torch.int8, device="cuda")
    s = torch.full((33, 5), 7.0, device="cuda")
    a = sdq.rmsnorm_quant(x, w, q=q[:, :272], s=s[:, :3])
    b = sdq.rmsnorm_quant(x.contiguous(), w)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert (q[:, 272:] == 7).all() and (s[:, 3:] == 7).all()


@pytest.mark.parametrize("codes,scales,group", [("int8", "fp32", 32), ("e4m3", "e8m0", 32), ("e2m1", "e8m0", 32),
                                                ("e2m1", "e4m3", 16)])
def test_norm_zero_and_non_finite_rows(codes, scales, group):
    gen = torch.Generator(device="cuda").manual_seed(6)
    x = _rows(gen, 6, 128, 1.0)
    x[0] = 0
    x[1, 64:96] = 0
    x[2, 5] = float("nan")
    x[3, 70] = float("inf")
    w = torch.ones(128, device="cuda")
    q, s, _ = sdq.rmsnorm_quant(x, w, group_size=group, codes=codes, scales=scales)
    q, s = q.view(torch.uint8).cpu().numpy(), s.view(torch.uint8 if scales != "fp32" else torch.float32).cpu().numpy()
    if codes == "e2m1":
        s = R.scale_values(s.reshape(-1)[R.tile_index(6, 128 // group)], scales)
        q = np.repeat(q, 2, 1)
    elif scales == "e8m0":
        s = R.scale_values(s, "e8m0")
    n = 32 // group
    q &= {"int8": 0xFF, "e4m3": 0x7F, "e2m1": 0x77}[codes]         # a zero keeps its sign
    assert (s[0] == 1).all() and (q[0] == 0).all()
    assert (s[1, 2 * n:3 * n] == 1).all() and (q[1, 64:96] == 0).all() and (q[1, :64] != 0).any()
    assert np.isnan(s[2]).all() and (q[2] == 0).all()            # the mean is NaN: all of the row
    bad = 70 // group                                             # rstd = 0: one NaN, the rest zeros
    assert np.isnan(s[3, bad]) and (np.delete(s[3], bad) == 1).all() and (q[3] == 0).all()
    assert np.isfinite(s[4:]).all()


def test_norm_tiny_and_huge_weights():
    """Groups whose scale leaves the normal fp32 range, and the largest finite ones."""
    gen = torch.Generator(device="cuda").manual_seed(8)
    x = _rows(gen, 4, 256, 1.0)
    for top in (1e-44, 1e-41, 1e-38, 1e-36, 3e37):
        w = torch.full((256,), top, device="cuda")
        q, s, _ = sdq.rmsnorm_quant(x, w, group_size=32, codes="int8", scales="fp32")
        y = R.norm(x.cpu(), None, w.cpu().double(), 1e-6)[1].numpy().reshape(4, 8, 32)
        s = s.cpu().double().numpy()
        got = q.cpu().double().numpy().reshape(4, 8, 32) * s[..., None]
        # y itself is a multiple of 2^-149 here; a code is off by half a scale
        tol = 0.5 * s[..., None] + 2.0 ** -148 + 2.0 ** -18 * np.abs(y)
        assert (np.abs(got - y) <= tol).all(), top
        q8, s8, _ = sdq.rmsnorm_quant(x, w, group_size=32, codes="e2m1", scales="e8m0")
        v = R.values(R.unpack(q8.cpu().numpy()), s8.view(torch.uint8).cpu().numpy().reshape(-1)[R.tile_index(4, 8)], "e8m0")
        sv = R.scale_values(s8.view(torch.uint8).cpu().numpy().reshape(-1)[R.tile_index(4, 8)], "e8m0")
        tol = np.repeat(sv, 32, 1)
        assert (np.abs(v - y.reshape(4, 256)) <= tol + 2.0 ** -148).all(), top


def test_norm_rows_are_independent_of_their_number():
    """The first rows of a long call equal the same rows alone (another variant): the sums differ in order only."""
    gen = torch.Generator(device="cuda").manual_seed(9)
    x = _rows(gen, 1000, 1408, 1.0)
    w = torch.rand(1408, generator=gen, device="cuda")
    q, s, _ = sdq.rmsnorm_quant(x, w)
    q1, s1, _ = sdq.rmsnorm_quant(x[:3], w)
    delta = (2 * ((32 + 14) / 2 + 4) + 1) * U24
    assert ((s[:3] - s1).abs() <= delta * s1).all()
    assert ((q[:3].int() - q1.int()).abs() <= 1).all() and (q[:3] == q1).float().mean() > 0.999
    assert torch.equal(sdq.rmsnorm_quant(x, w)[0], q)


def test_norm_empty_and_refusals():
    x = torch.zeros(0, 64, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(64, device="cuda")
    q, s, h = sdq.rmsnorm_quant(x, w)
    assert q.shape == (0, 64) and s.shape == (0, 1) and h is x
    q, s, _ = sdq.rmsnorm_quant(x, w, codes="e2m1")
    assert q.shape == (0, 32) and s.shape == (0, 1, 512)
    x = torch.zeros(4, 64, dtype=torch.bfloat16, device="cuda")
    for kw in (dict(codes="int4"), dict(codes="int8", scales="e4m3"), dict(codes="e2m1", scales="fp32"),
               dict(group_size=16), dict(codes="e2m1", group_size=64), dict(h=x), dict(residual=x[:2]),
               dict(rstd=w), dict(q=torch.zeros(4, 64, dtype=torch.uint8, device="cuda"), codes="int8"),
               dict(global_scale=w[:1]), dict(residual=x, h=x.float()), dict(y=x.t())):
        with pytest.raises(ValueError):
            sdq.rmsnorm_quant(x, w, **kw)
    for bad in (x[:, :24], x.float(), x[:, ::2]):
        with pytest.raises(ValueError):
            sdq.rmsnorm_quant(bad, w[:bad.shape[1]])
    with pytest.raises(ValueError):
        sdq.rmsnorm_quant(x, w.half())
    with pytest.raises(sdq.SdqError):                             # rows that do not start on 16 bytes
        sdq.rmsnorm_quant(torch.zeros(4, 68, dtype=torch.bfloat16, device="cuda")[:, :64], w)


# ---- backward -------------------------------------------------------------------
#
# grad_x: the row's sum is off by (seq + 14) 2^-24 of the sum of its magnitudes,
# each product and sum by 2^-24 of what it adds, and the result by 2^-8 of itself:
# |error| <= 2^-8 |grad_x| + (seq + 24) 2^-24 mag, mag the magnitudes added.
# grad_weight: a CTA adds at most ceil(rows / parts) numbers in a row, then
# parts / 8 + 8 sums follow, each number with 3 roundings of its own.

def _seq_bwd(channels):
    return 32 if channels <= 16384 else 8 * -(-channels // 8192)


def _check_bwd(rows, channels, weight_dtype, with_gh, seed, pad=0, alias=None):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    h, gy = _rows(gen, rows, channels, 1.5, pad), _rows(gen, rows, channels, 0.3, pad)
    gh = _rows(gen, rows, channels, 0.2, pad) if with_gh else None
    w = (torch.randn(channels, generator=gen, device="cuda") + 1).to(weight_dtype)
    rstd = torch.rsqrt(h.double().square().mean(1) + 1e-6).float()
    gx, gw, mag, magw = R.norm_backward(gy.cpu(), h.cpu(), w.cpu(), rstd.cpu(), None if gh is None else gh.cpu())
    out = {None: None, "grad_y": gy, "h": h, "grad_h": gh}[alias]
    ws = U.Guarded((sdq.sdq_rmsnorm_backward_workspace_bytes(rows, channels),), torch.uint8, 0xA5)
    wb = U.Guarded((channels,), torch.float32, -1.0)
    got, gotw = sdq.rmsnorm_backward(gy, h, w, rstd, gh, grad_x=out, grad_weight=wb.t, workspace=ws.t)
    torch.cuda.synchronize()
    assert ws.guards_intact() and wb.guards_intact()
    err = (got.cpu().double() - gx).abs()
    tol = 2.0 ** -8 * gx.abs() + (_seq_bwd(channels) + 24) * U24 * mag
    assert (err <= tol).all(), f"grad_x {(err / tol).max()}"
    adds = -(-rows // 148) + 592 / 8 + 8 + 3
    err = (gotw.cpu().double() - gw).abs()
    assert (err <= adds * U24 * magw).all(), f"grad_weight {(err / magw).max() / U24}"
    return got, gotw


@pytest.mark.parametrize("rows,channels", [(1, 16), (2, 48), (5, 272), (33, 1040), (149, 2064), (700, 1408), (3, 4096),
                                           (600, 7168), (5, 12304), (2, 20000), (300, 16400), (1300, 64)])
@pytest.mark.parametrize("with_gh", [False, True])
def test_norm_backward(rows, channels, with_gh):
    _check_bwd(rows, channels, torch.bfloat16 if with_gh else torch.float32, with_gh, rows + channels)


@pytest.mark.parametrize("codes,scales,group", [("int8", "fp32", 128), ("e4m3", "fp32", 0), ("e2m1", "e8m0", 32)])
@pytest.mark.parametrize("rows,channels", [(2601, 1408), (1199, 2400), (1502, 2816), (1203, 3584)])
def test_norm_rows_of_odd_warps(codes, scales, group, rows, channels):
    """Three, five, six and seven warps a row, several rounds of them, the last not whole."""
    gen = torch.Generator(device="cuda").manual_seed(rows + channels)
    _run(_rows(gen, rows, channels, 1.0), torch.rand(channels, generator=gen, device="cuda") - 0.5,
         _rows(gen, rows, channels, 1.0), codes, scales, group)


@pytest.mark.parametrize("rows,channels", [(3001, 1408), (5003, 1536), (1303, 2400), (1502, 2816), (1201, 3584),
                                           (700, 6144), (650, 6160)])
def test_norm_backward_rows_of_odd_warps(rows, channels):
    _check_bwd(rows, channels, torch.bfloat16, True, rows + channels)


@pytest.mark.parametrize("rows,channels", [(2003, 2048), (1131, 528), (607, 16), (830, 2832), (1100, 3600), (31, 96)])
def test_norm_backward_of_few_rows_in_wide_ctas(rows, channels):
    _check_bwd(rows, channels, torch.float32, True, rows + channels)


def test_norm_backward_strided_and_in_place():
    for alias in ("grad_y", "h", "grad_h"):
        _check_bwd(40, 528, torch.float32, True, 3, pad=16, alias=alias)
        _check_bwd(3, 16640, torch.float32, True, 4, pad=16, alias=alias)


@pytest.mark.parametrize("rows,channels", [(300, 1040), (500, 256), (200, 7168), (900, 3008)])
def test_norm_backward_of_few_rows_in_place(rows, channels):
    """grad_weight is summed from grad_y and h: it must not meet grad_x written over them."""
    for alias in ("grad_y", "h", "grad_h"):
        for seed in range(6):
            _check_bwd(rows, channels, torch.float32, True, seed, alias=alias)


def test_norm_backward_empty_and_repeatable():
    w = torch.ones(64, device="cuda")
    x = torch.zeros(0, 64, dtype=torch.bfloat16, device="cuda")
    gw = torch.full((64,), 7.0, device="cuda")
    gx, _ = sdq.rmsnorm_backward(x, x, w, torch.zeros(0, device="cuda"), grad_weight=gw)
    assert gx.shape == (0, 64) and (gw == 0).all()
    a, b = (_check_bwd(1000, 1408, torch.float32, True, 12) for _ in range(2))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_norm_backward_refusals():
    x = torch.zeros(4, 64, dtype=torch.bfloat16, device="cuda")
    w, r = torch.ones(64, device="cuda"), torch.ones(4, device="cuda")
    for a, kw in (((x, x[:3], w, r), {}), ((x, x, w[:32], r), {}), ((x, x, w, r[:3]), {}), ((x, x, w, r.double()), {}),
                  ((x[:, :24], x[:, :24], w[:24], r), {}), ((x, x, w, r, x.float()), {}),
                  ((x, x, w, r), dict(grad_weight=w.bfloat16())), ((x, x, w, r), dict(grad_x=x.t()))):
        with pytest.raises(ValueError):
            sdq.rmsnorm_backward(*a, **kw)
    with pytest.raises(sdq.SdqError) as e:
        sdq.rmsnorm_backward(x, x, w, r, workspace=torch.zeros(64, dtype=torch.uint8, device="cuda"))
    assert e.value.status == sdq.Status.ERR_WORKSPACE


def test_backward_is_the_derivative_of_the_forward():
    """Differences of the forward (its bf16 y, through 64-bit sums) against the backward's gradients."""
    gen = torch.Generator(device="cuda").manual_seed(21)
    rows, channels, eps = 16, 256, 1e-3
    x = _rows(gen, rows, channels, 1.0)
    w = torch.rand(channels, generator=gen, device="cuda") + 0.5
    gy = _rows(gen, rows, channels, 1.0)
    rstd = torch.empty(rows, device="cuda")
    sdq.rmsnorm_quant(x, w, eps=eps, rstd=rstd)
    gx, gw = sdq.rmsnorm_backward(gy, x, w, rstd)

    def loss(x, w):
        y = torch.empty(rows, channels, dtype=torch.bfloat16, device="cuda")
        sdq.rmsnorm_quant(x, w, eps=eps, y=y)
        return (y.double() * gy.double()).sum()

    # weights move by d: y is linear in them.  Each y is rounded to 2^-8 of itself at
    # either end, independently: the difference is off by 2^-8 * sqrt(2 sum (y gy)^2)
    # at one standard deviation at most; six are allowed.
    d = torch.randn(channels, generator=gen, device="cuda") * 0.25
    y = x.double() * rstd.double()[:, None] * w.double()
    noise = 6 * 2.0 ** -8 * float((2 * (y * gy.double()).square().sum()).sqrt())
    assert abs(float(loss(x, w + d) - loss(x, w - d)) / 2 - float((gw.double() * d.double()).sum())) <= noise
    # x moves along e by bf16 steps: second-order terms are below (|e| / |x|)^2 of the loss's scale
    e = (torch.randn(rows, channels, generator=gen, device="cuda") * 0.02).bfloat16()
    xp, xm = (x.float() + e.float()).bfloat16(), (x.float() - e.float()).bfloat16()
    step = (xp.double() - xm.double()) / 2
    curve = 8 * (0.02 ** 2) * float((y * gy.double()).abs().sum()) * 0.02
    assert abs(float(loss(xp, w) - loss(xm, w)) / 2 - float((gx.double() * step).sum())) <= noise + curve
