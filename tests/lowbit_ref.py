"""Plain 64-bit forms of the operators around the projections (RMS norm into
codes, its backward, 4-bit quantizer and product), on the CPU, and the
tolerances of the comparisons with them."""
from __future__ import annotations

import numpy as np
import torch

E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
QMAX = {"int8": 127.0, "e4m3": 448.0, "e2m1": 6.0}
GROUP = {"e8m0": 32, "e4m3": 16}


def e4m3_values() -> np.ndarray:
    """The value of each of the 256 E4M3 bytes."""
    b = np.arange(256)
    e, m = (b >> 3) & 15, b & 7
    v = np.where(e == 0, m * 2.0 ** -9, (1 + m / 8) * 2.0 ** (e - 7.0))
    v[b & 0x7F == 0x7F] = np.nan
    return np.where(b & 0x80, -v, v)


E4M3 = e4m3_values()


def scale_values(b: np.ndarray, scales: str) -> np.ndarray:
    b = np.asarray(b)
    if scales == "e4m3":
        return E4M3[b]
    return np.where(b == 255, np.nan, np.ldexp(1.0, b.astype(np.int64) - 127))


def e4m3_byte(v: np.ndarray) -> np.ndarray:
    """Nearest E4M3 byte of v >= 0, ties to the even mantissa, saturated."""
    grid = E4M3[:0x7F]
    hi = np.searchsorted(grid, v).clip(0, 0x7E)
    lo = (hi - 1).clip(0)
    dl, dh = v - grid[lo], grid[hi] - v
    return np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)


def e2m1_code(v: np.ndarray) -> np.ndarray:
    """Nearest E2M1 code, ties to the even code, saturated; the sign kept."""
    mids = (E2M1[1:] + E2M1[:-1]) / 2
    a = np.abs(v)
    lo, hi = np.searchsorted(mids, a, side="left"), np.searchsorted(mids, a, side="right")
    return np.where(lo % 2 == 0, lo, hi) | np.where(np.signbit(v), 8, 0)


def e2m1_value(c: np.ndarray) -> np.ndarray:
    return np.where(c & 8, -1.0, 1.0) * E2M1[c & 7]


def pow2_ceil_exp(t: np.ndarray) -> np.ndarray:
    """The smallest k in [-127, 127] with 2^k >= t > 0."""
    m, e = np.frexp(t)
    return np.where(m == 0.5, e - 1, e).clip(-127, 127)


def quantize_fp4(x: np.ndarray, scales: str, g: float = 1.0):
    """(codes, scale bytes) of the rows of x (fp32 values), from the formulas:
    the scale's quotient and the codes' are fp32 quotients, correctly rounded."""
    x = np.asarray(x, np.float32)
    rows, k = x.shape
    n = GROUP[scales]
    v = x.reshape(rows, -1, n)
    bad = ~np.isfinite(v).all(2)
    v = np.where(bad[..., None], np.float32(0), v)
    amax = np.abs(v).max(2)
    with np.errstate(all="ignore"):
        if scales == "e8m0":
            e = pow2_ceil_exp(np.where(amax > 0, amax / np.float32(6), np.float32(1)))
            sb = e + 127
            unit = np.ldexp(1.0, e)
        else:
            s = amax / (np.float32(6) * np.float32(g))
            sb = np.maximum(e4m3_byte(s.astype(np.float64)), 1)
            sb = np.where(amax > 0, sb, 0x38)
            unit = (E4M3[sb].astype(np.float32) * np.float32(g)).astype(np.float64)
        q = (v / unit[..., None].astype(np.float32)) if scales == "e4m3" else v.astype(np.float64) / unit[..., None]
    codes = np.where(bad[..., None], 0, e2m1_code(q.astype(np.float64)))
    sb = np.where(bad, 255 if scales == "e8m0" else 0x7F, sb)
    return codes.reshape(rows, k), sb


def pack(codes: np.ndarray) -> np.ndarray:
    return (codes[:, 0::2] | (codes[:, 1::2] << 4)).astype(np.uint8)


def unpack(packed: np.ndarray) -> np.ndarray:
    out = np.empty((packed.shape[0], 2 * packed.shape[1]), np.int64)
    out[:, 0::2], out[:, 1::2] = packed & 15, packed >> 4
    return out


def tile_index(rows: int, groups: int):
    """Flat offsets of the scales [rows, groups] in their tiles."""
    r, j = np.arange(rows)[:, None], np.arange(groups)[None, :]
    return (r // 128 * (-(-groups // 4)) + j // 4) * 512 + r % 32 * 16 + r % 128 // 32 * 4 + j % 4


def tiles(sb: np.ndarray, fill: int = 0) -> np.ndarray:
    rows, groups = sb.shape
    out = np.full((-(-rows // 128), -(-groups // 4), 512), fill, np.uint8)
    out.reshape(-1)[tile_index(rows, groups)] = sb
    return out


def values(codes: np.ndarray, sb: np.ndarray, scales: str, g: float = 1.0) -> np.ndarray:
    """The numbers behind codes [rows, k] and scale bytes [rows, groups]."""
    unit = scale_values(sb, scales) * (g if scales == "e4m3" else 1.0)
    return e2m1_value(codes) * np.repeat(unit, GROUP[scales], axis=1)


def norm(x: torch.Tensor, residual, weight: torch.Tensor, eps: float):
    """(h bf16, y fp64, rstd fp64): h as the definition rounds it."""
    h = x if residual is None else (x.float() + residual.float()).bfloat16()
    d = h.double()
    rstd = 1 / torch.sqrt(d.square().mean(1) + eps)
    return h, d * rstd[:, None] * weight.double(), rstd


def norm_backward(gy, h, weight, rstd, gh):
    """(grad_x, grad_weight, sum of the magnitudes in each), fp64."""
    gy, n, w = gy.double(), h.double() * rstd.double()[:, None], weight.double()
    g, r = gy * w, rstd.double()[:, None]
    c = (g * n).mean(1, keepdim=True)
    gx, mag = r * (g - n * c), r * (g.abs() + n.abs() * (g * n).abs().mean(1, keepdim=True))
    if gh is not None:
        gx, mag = gx + gh.double(), mag + gh.double().abs()
    return gx, (gy * n).sum(0), mag, (gy * n).abs().sum(0)
