"""The norm, the 4-bit quantizer and the 4-bit product: argument checks of the C
entries and the Python functions, on the CPU (nothing is launched), and the
plain forms that the GPU tests compare with."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import swiglu_backward_int8_b200 as sdq
from tests import lowbit_ref as R

A = 1 << 20   # an aligned fake address: validation never dereferences
OK, NULL, GROUP, SHAPE, ALIGN, WORKSPACE, FORMAT, STRIDE = 0, 1, 2, 3, 4, 7, 9, 10
MX, NV = sdq.FMT_E2M1 | sdq.FMT_E8M0, sdq.FMT_E2M1 | sdq.FMT_SCALE_E4M3


def _norm(**kw):
    a = dict(x=A, ld_x=256, residual=A, ld_residual=256, weight=A, h=A, ld_h=256, q=A, ld_q=256, s=A, ld_s=2, y=None,
             ld_y=0, rstd=None, global_scale=None, rows=5, channels=256, group_size=128, format=0)
    a.update(kw)
    return tuple(a.values())


@pytest.mark.parametrize("kw,status", [
    ({}, OK),
    (dict(format=sdq.FMT_E4M3 | sdq.FMT_E8M0 | sdq.FMT_WEIGHT_F32, s=A + 1), OK),
    (dict(format=MX, group_size=32, ld_q=128, ld_s=0), OK),
    (dict(format=NV, group_size=16, ld_q=128, ld_s=0, global_scale=A), OK),
    (dict(group_size=0, ld_s=1), OK),
    (dict(residual=None, h=None), OK),
    (dict(y=A, ld_y=264, rstd=A + 4), OK),
    (dict(rows=0, x=None, q=None), OK),
    (dict(channels=16, ld_s=1), OK),
    (dict(format=128), FORMAT),
    (dict(format=sdq.FMT_OUT_F32), FORMAT),
    (dict(format=sdq.FMT_E2M1), FORMAT),                        # which scales?
    (dict(format=MX | sdq.FMT_SCALE_E4M3), FORMAT),
    (dict(format=MX | sdq.FMT_E4M3), FORMAT),
    (dict(format=sdq.FMT_SCALE_E4M3), FORMAT),                  # E4M3 scales go with E2M1 codes
    (dict(format=MX, group_size=16), GROUP),
    (dict(format=NV, group_size=32), GROUP),
    (dict(group_size=16), GROUP),
    (dict(group_size=512), GROUP),
    (dict(group_size=-1), GROUP),
    (dict(rows=-1), SHAPE),
    (dict(rows=1 << 31), SHAPE),
    (dict(channels=0), SHAPE),
    (dict(channels=24), SHAPE),
    (dict(channels=(1 << 20) + 16), SHAPE),
    (dict(format=MX, group_size=32, channels=48), SHAPE),
    (dict(x=None), NULL),
    (dict(weight=None), NULL),
    (dict(s=None), NULL),
    (dict(h=None), NULL),                                       # a residual without h
    (dict(ld_x=255), STRIDE),
    (dict(ld_h=128), STRIDE),
    (dict(ld_q=255), STRIDE),
    (dict(ld_s=1), STRIDE),
    (dict(y=A, ld_y=8), STRIDE),
    (dict(ld_residual=(1 << 36) + 8), STRIDE),
    (dict(ld_x=260), ALIGN),
    (dict(x=A + 8), ALIGN),
    (dict(ld_q=264), ALIGN),
    (dict(weight=A + 4), ALIGN),
    (dict(s=A + 2), ALIGN),
    (dict(rstd=A + 1), ALIGN),
    (dict(format=MX, group_size=32, ld_q=128, s=A + 8), ALIGN),
])
def test_validate_norm(kw, status):
    assert sdq.sdq_validate_rmsnorm_quant(*_norm(**kw)) == status
    if status:   # the entry itself answers the same, without a GPU
        with pytest.raises(sdq.SdqError) as e:
            sdq.sdq_rmsnorm_quant(*_norm(**kw), 1e-6, None)
        assert e.value.status == status


def _bwd(**kw):
    a = dict(gy=A, ld_gy=256, h=A, ld_h=256, weight=A, rstd=A, gh=A, ld_gh=256, gx=A, ld_gx=256, gw=A, rows=5,
             channels=256, format=0, workspace=A, workspace_bytes=5 * 1024)
    a.update(kw)
    return tuple(a.values())


@pytest.mark.parametrize("kw,status", [
    ({}, OK),
    (dict(gh=None, ld_gh=0, format=sdq.FMT_WEIGHT_F32), OK),
    (dict(rows=0, gy=None, workspace=None, workspace_bytes=4 * 256), OK),
    (dict(rows=10 ** 6, workspace_bytes=592 * 1024), OK),
    (dict(format=sdq.FMT_E4M3), FORMAT),
    (dict(rows=-1), SHAPE),
    (dict(channels=8), SHAPE),
    (dict(gw=None), NULL),
    (dict(gw=None, rows=0), NULL),
    (dict(rstd=None), NULL),
    (dict(workspace=None), NULL),
    (dict(workspace_bytes=5 * 1024 - 1), WORKSPACE),
    (dict(workspace=A + 4), WORKSPACE),
    (dict(ld_gx=248), STRIDE),
    (dict(ld_gh=100), STRIDE),
    (dict(ld_gy=257), ALIGN),
    (dict(gx=A + 2), ALIGN),
    (dict(gw=A + 2), ALIGN),
])
def test_validate_norm_backward(kw, status):
    assert sdq.sdq_validate_rmsnorm_backward(*_bwd(**kw)) == status


def test_backward_workspace_bytes():
    f = sdq.sdq_rmsnorm_backward_workspace_bytes
    assert f(1, 16) == 64 and f(100, 4096) == 100 * 4096 * 4
    assert f(10 ** 6, 4096) == f(592, 4096) == 592 * 4096 * 4      # bounded, whatever the rows
    assert f(5, 24) == f(-1, 64) == f(5, 0) == 0


def _quant(**kw):
    a = dict(x=A, ld_x=96, q=A, ld_q=48, s=A, q_t=A, ld_q_t=16, s_t=A, g=None, rows=5, channels=96,
             format=sdq.FMT_E8M0)
    a.update(kw)
    return tuple(a.values())


@pytest.mark.parametrize("kw,status", [
    ({}, OK),
    (dict(q=None, s=None), OK),
    (dict(q_t=None, s_t=None, ld_q_t=0), OK),
    (dict(format=sdq.FMT_SCALE_E4M3, g=A), OK),
    (dict(rows=0, x=None), OK),
    (dict(format=0), FORMAT),
    (dict(format=sdq.FMT_E8M0 | sdq.FMT_SCALE_E4M3), FORMAT),
    (dict(format=MX), FORMAT),
    (dict(channels=80), SHAPE),
    (dict(channels=0), SHAPE),
    (dict(rows=-1), SHAPE),
    (dict(x=None), NULL),
    (dict(q=None, q_t=None), NULL),
    (dict(s=None), NULL),
    (dict(s_t=None), NULL),
    (dict(ld_x=95), STRIDE),
    (dict(ld_q=32), STRIDE),
    (dict(rows=33, ld_q_t=16), STRIDE),                          # 33 rows: 64 codes a channel
    (dict(rows=33, ld_q_t=32), OK),
    (dict(ld_q=56), ALIGN),
    (dict(q_t=A + 8), ALIGN),
    (dict(s=A + 4), ALIGN),
    (dict(ld_x=100), ALIGN),
    (dict(g=A + 1), ALIGN),
])
def test_validate_quantize(kw, status):
    assert sdq.sdq_validate_quantize_fp4(*_quant(**kw)) == status


def _dequant(**kw):
    a = dict(q=A, ld_q=48, s=A, g=None, out=A, ld_out=96, rows=5, channels=96, format=sdq.FMT_E8M0)
    a.update(kw)
    return tuple(a.values())


@pytest.mark.parametrize("kw,status", [
    ({}, OK), (dict(rows=0, q=None), OK), (dict(format=7), FORMAT), (dict(channels=16), SHAPE), (dict(s=None), NULL),
    (dict(ld_out=88), STRIDE), (dict(out=A + 8), ALIGN), (dict(ld_q=50), ALIGN), (dict(ld_out=100), ALIGN),
])
def test_validate_dequantize(kw, status):
    assert sdq.sdq_validate_dequantize_fp4(*_dequant(**kw)) == status


def _matmul(**kw):
    a = dict(a=A, ld_a=48, a_s=A, a_g=None, b=A, ld_b=48, b_s=A, b_g=None, out=A, ld_out=7, m=5, n=7, k=96,
             format=sdq.FMT_E8M0)
    a.update(kw)
    return tuple(a.values())


@pytest.mark.parametrize("kw,status", [
    ({}, OK),
    (dict(format=sdq.FMT_SCALE_E4M3 | sdq.FMT_OUT_F32, a_g=A, b_g=A), OK),
    (dict(out=A + 2), OK),                                       # bf16 out: its own alignment is enough
    (dict(m=0, a=None), OK),
    (dict(n=0, b=None), OK),
    (dict(format=sdq.FMT_OUT_F32), FORMAT),
    (dict(format=sdq.FMT_E8M0 | sdq.FMT_WEIGHT_F32), FORMAT),
    (dict(k=40), SHAPE),
    (dict(k=0), SHAPE),
    (dict(m=-1), SHAPE),
    (dict(n=1 << 31), SHAPE),
    (dict(m=1 << 30, n=1 << 30), SHAPE),
    (dict(b_s=None), NULL),
    (dict(out=None), NULL),
    (dict(ld_a=32), STRIDE),
    (dict(ld_out=6), STRIDE),
    (dict(ld_b=56), ALIGN),
    (dict(a_s=A + 8), ALIGN),
    (dict(out=A + 2, format=sdq.FMT_E8M0 | sdq.FMT_OUT_F32), ALIGN),
    (dict(b_g=A + 2), ALIGN),
])
def test_validate_matmul(kw, status):
    assert sdq.sdq_validate_matmul_fp4(*_matmul(**kw)) == status


def test_scale_shapes():
    assert sdq.fp4_scale_shape(1, 32) == (1, 1, 512)
    assert sdq.fp4_scale_shape(129, 160, "e8m0") == (2, 2, 512)
    assert sdq.fp4_scale_shape(129, 160, "e4m3") == (2, 3, 512)
    assert sdq.sdq_fp4_scale_bytes(129, 160, sdq.FMT_SCALE_E4M3) == 2 * 3 * 512
    assert sdq.sdq_fp4_scale_bytes(129, 160, 0) == 0 and sdq.sdq_fp4_scale_bytes(1, 33, sdq.FMT_E8M0) == 0
    for bad in ((1, 33, "e8m0"), (1, 0, "e8m0"), (-1, 32, "e8m0"), (1, 32, "fp32")):
        with pytest.raises(ValueError):
            sdq.fp4_scale_shape(*bad)


def test_python_refuses_host_tensors():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    w = torch.ones(64)
    q, s = torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(1, 1, 512, dtype=torch.uint8)
    for call in (lambda: sdq.rmsnorm_quant(x, w), lambda: sdq.rmsnorm_backward(x, x, w, torch.ones(4)),
                 lambda: sdq.quantize_fp4(x), lambda: sdq.dequantize_fp4(q, s), lambda: sdq.matmul_fp4(q, s, q, s)):
        with pytest.raises(ValueError, match="CUDA"):
            call()


# ---- the plain forms ----------------------------------------------------------

def test_e2m1_and_e4m3_rounding_by_hand():
    v = np.array([0.25, 0.2500001, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 5.0001, 7.0, -0.25, -2.5, -0.0])
    assert R.e2m1_value(R.e2m1_code(v)).tolist() == [0, 0.5, 1, 1, 2, 2, 4, 4, 6, 6, 0, -2, 0]
    v = np.array([0, 2.0 ** -10, 2.0 ** -10 * 1.01, 1.0625, 1.1875, 448, 464, 1e9])
    assert R.E4M3[R.e4m3_byte(v)].tolist() == [0, 0, 2.0 ** -9, 1.0, 1.25, 448, 448, 448]


def test_tiles_and_packing_round_trip():
    rng = np.random.default_rng(1)
    c = rng.integers(0, 16, (3, 64))
    assert np.array_equal(R.unpack(R.pack(c)), c) and R.pack(c)[0, 0] == c[0, 0] + 16 * c[0, 1]
    sb = rng.integers(0, 255, (200, 6))
    t = R.tiles(sb)
    assert t.shape == (2, 2, 512) and np.array_equal(t.reshape(-1)[R.tile_index(200, 6)], sb)
    assert t[1, 1, (150 % 32) * 16 + 0 * 4 + 1] == sb[150, 5]     # row 150 is 22 of the second tile's first 32


def test_norm_gradient_formula_against_autograd_and_differences():
    g = torch.Generator().manual_seed(3)
    x = torch.randn(5, 48, generator=g, dtype=torch.float64, requires_grad=True)
    w = torch.randn(48, generator=g, dtype=torch.float64, requires_grad=True)
    gy, gh = torch.randn(2, 5, 48, generator=g, dtype=torch.float64)
    eps = 1e-3

    def loss(x, w):
        return (x * torch.rsqrt(x.square().mean(1, keepdim=True) + eps) * w * gy + x * gh).sum()

    loss(x, w).backward()
    rstd = torch.rsqrt(x.detach().square().mean(1) + eps)
    gx, gw, _, _ = R.norm_backward(gy, x.detach(), w.detach(), rstd, gh)
    assert torch.allclose(gx, x.grad, rtol=1e-12, atol=1e-12) and torch.allclose(gw, w.grad, rtol=1e-12, atol=1e-12)
    with torch.no_grad():
        for i, j in ((0, 0), (3, 17), (4, 47)):
            d = torch.zeros_like(x)
            d[i, j] = 1e-5
            assert abs((loss(x + d, w) - loss(x - d, w)) / 2e-5 - gx[i, j]) < 1e-7     # O(step^2) = 1e-10 and cancellation 1e-16 / 1e-5
