"""The operators around the projections of a quantized MLP, next to the fused
SwiGLU op: RMS norm into 8- or 4-bit codes and its backward, the microscaled
4-bit quantizer, and the product of two 4-bit operands.  Formulas, layouts and
limits: include/sdq.h.

4-bit operands are a pair of tensors: codes, uint8 [rows, k / 2] (two E2M1 codes
to a byte), and scale tiles of shape ``fp4_scale_shape(rows, k, scales)``:
``scales="e8m0"`` (powers of two for 32 values; dtype float8_e8m0fnu or uint8) or
``scales="e4m3"`` (E4M3 for 16 values; float8_e4m3fn), the latter times an
optional scale per tensor, a float32 tensor of one element on the device.

Every call runs on the current stream of its tensors' device.  Tensors are 2-D
and row-major; rows may be padded.  ValueError for arguments that do not fit
together, SdqError for a status of the library.
"""
from __future__ import annotations

from typing import Optional, Tuple

import torch

from . import _extension
from ._check import _rows
from ._lib import (FMT_E2M1, FMT_E4M3, FMT_E8M0, FMT_OUT_F32, FMT_SCALE_E4M3, FMT_WEIGHT_F32,
                   SdqError, entry_addresses, sdq_dequantize_fp4, sdq_matmul_fp4, sdq_quantize_fp4, sdq_rmsnorm_backward,
                   sdq_rmsnorm_backward_workspace_bytes, sdq_rmsnorm_quant)

# Each function below first offers its arguments to its namesake in csrc/marshal.cpp,
# which makes the ordinary call (every output given, on the current device) and
# answers with its status, or with -1: then the checks and allocations here run.
_marshal = _extension.load(entry_addresses())

_BF16 = (torch.bfloat16,)
_F32 = (torch.float32,)
_U8 = (torch.uint8,)
_WEIGHT = (torch.bfloat16, torch.float32)
_CODES = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn, "e2m1": torch.uint8}
_CODES_OF = {torch.int8: "int8", torch.float8_e4m3fn: "e4m3", torch.uint8: "e2m1"}
_SCALES = {"fp32": torch.float32, "e8m0": torch.float8_e8m0fnu, "e4m3": torch.float8_e4m3fn}
_SCALES_OF = {torch.float32: "fp32", torch.float8_e8m0fnu: "e8m0", torch.uint8: "e8m0",
              torch.float8_e4m3fn: "e4m3"}
_FP4_GROUP = {"e8m0": 32, "e4m3": 16}
_FP4_FORMAT = {"e8m0": FMT_E8M0, "e4m3": FMT_SCALE_E4M3}


def _made(status: int, entry: str) -> bool:
    """Whether the short way made the call."""
    if status > 0:
        raise SdqError(status, entry)
    return status == 0


def fp4_scale_shape(rows: int, k: int, scales: str = "e8m0") -> Tuple[int, int, int]:
    """Shape of the scale tiles of [rows, k] 4-bit codes: (ceil(rows / 128),
    ceil(groups / 4), 512), with groups of 32 ("e8m0") or 16 ("e4m3") values."""
    if scales not in _FP4_GROUP:
        raise ValueError(f"4-bit codes have \"e8m0\" or \"e4m3\" scales, not {scales!r}")
    if rows < 0 or k < 32 or k % 32:
        raise ValueError(f"k={k} must be a positive multiple of 32 and rows={rows} not negative")
    groups = k // _FP4_GROUP[scales]
    return -(-rows // 128), -(-groups // 4), 512


def _scales_of(s: Optional[torch.Tensor], given: Optional[str], default: str) -> str:
    found = given if s is None or given is not None else _SCALES_OF.get(s.dtype)
    found = default if found is None and s is None else found
    if found not in _SCALES:
        raise ValueError(f"cannot tell the scale format{'' if s is None else f' from dtype {s.dtype}'}; pass scales=...")
    if s is not None and _SCALES_OF.get(s.dtype) != found:
        raise ValueError(f"{found} scales do not go into {s.dtype}")
    return found


def _tiles(name: str, s: torch.Tensor, rows: int, k: int, scales: str, device) -> int:
    """Check scale tiles; returns their address."""
    shape = (-(-rows // 128), -(-(k // _FP4_GROUP[scales]) // 4), 512)
    if s.shape != shape or _SCALES_OF.get(s.dtype) != scales or s.get_device() != device.index or not s.is_contiguous():
        raise ValueError(f"{name}: expected contiguous {scales} scale tiles {shape} on {device}, got {s.dtype} "
                         f"{tuple(s.shape)} on {s.device}")
    return s.data_ptr()


def _codes(name: str, q: torch.Tensor, rows: int, k: int, device) -> int:
    return _rows(name, q, (rows, k // 2), _U8, True, device)


def _length(k: int) -> None:
    if k < 32 or k % 32:
        raise ValueError(f"k={k} must be a positive multiple of 32")


def _one(name: str, g: Optional[torch.Tensor], scales: str, device) -> Optional[int]:
    """The address of a scale per tensor, or None."""
    if g is None:
        return None
    if scales != "e4m3":
        raise ValueError(f"{name} goes with \"e4m3\" scales")
    if g.numel() != 1 or g.dtype != torch.float32 or g.get_device() != device.index:
        raise ValueError(f"{name} must be one float32 on {device}")
    return g.data_ptr()


def _vector(name: str, v: torch.Tensor, n: int, dtypes, device) -> int:
    if v.shape != (n,) or v.dtype not in dtypes or v.get_device() != device.index or not v.is_contiguous():
        raise ValueError(f"{name}: expected contiguous {' or '.join(map(str, dtypes))} [{n}] on {device}, got {v.dtype} "
                         f"{tuple(v.shape)} on {v.device}")
    return v.data_ptr()


def _two_d(name: str, t: torch.Tensor) -> Tuple[int, int]:
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    return t.shape


def _call(entry, device, *args) -> None:
    """The entry point on the device's current stream."""
    with torch.cuda.device(device):
        entry(*args, torch.cuda.current_stream(device).cuda_stream)


def rmsnorm_quant(x: torch.Tensor, weight: torch.Tensor, residual: Optional[torch.Tensor] = None,
                  eps: float = 1e-6, group_size: Optional[int] = None, *, codes: Optional[str] = None,
                  scales: Optional[str] = None, q: Optional[torch.Tensor] = None,
                  s: Optional[torch.Tensor] = None, h: Optional[torch.Tensor] = None,
                  y: Optional[torch.Tensor] = None, rstd: Optional[torch.Tensor] = None,
                  global_scale: Optional[torch.Tensor] = None
                  ) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """h = bf16(x + residual), its RMS norm times weight, and the codes and
    scales of that: returns (q, s, h), allocating what is not given (h is x
    without a residual).

    x, residual: bf16 [rows, channels]; weight: bf16 or fp32 [channels].
    ``codes`` "int8" (the default), "e4m3" or "e2m1" and ``scales`` "fp32" (the
    default), "e8m0" or, for "e2m1" only, "e4m3" follow the dtypes of q and s
    where those are given.  ``group_size``: channels a scale: 32, 64, 128 (the
    default), 256 or 0 (one scale a row); 4-bit codes have 32 ("e8m0") or 16
    ("e4m3").  8-bit codes: q [rows, channels], s [rows, ceil(channels /
    group_size)]; "e2m1": q uint8 [rows, channels / 2], s scale tiles.
    ``h`` may be x or residual itself.  Optional outputs: ``y`` (bf16, the
    normed rows) and ``rstd`` (fp32 [rows], for ``rmsnorm_backward``).
    ``global_scale``: the scale per tensor of "e2m1" codes with "e4m3" scales."""
    if _made(_marshal.rmsnorm_quant(x, weight, residual, eps, group_size, codes, scales, q, s, h, y, rstd, global_scale),
             "sdq_rmsnorm_quant"):
        return q, s, (x if residual is None else h)
    rows, channels = _two_d("x", x)
    dev = x.device
    codes = codes or ("int8" if q is None else _CODES_OF.get(q.dtype))
    if codes not in _CODES or (q is not None and q.dtype != _CODES[codes]):
        raise ValueError(f"codes {codes!r} do not go with q of {None if q is None else q.dtype}")
    e2m1 = codes == "e2m1"
    scales = _scales_of(s, scales, "e8m0" if e2m1 else "fp32")
    if (scales in _FP4_GROUP if e2m1 else scales != "e4m3") is False:
        raise ValueError(f"{codes} codes do not go with {scales} scales")
    if group_size is None:
        group_size = _FP4_GROUP[scales] if e2m1 else 128
    if e2m1 and group_size != _FP4_GROUP[scales] or not e2m1 and group_size not in (0, 32, 64, 128, 256):
        raise ValueError(f"group_size {group_size} does not go with {codes} codes and {scales} scales")
    if channels < 1 or channels % (32 if e2m1 else 16):
        raise ValueError(f"{channels} channels: a positive multiple of {32 if e2m1 else 16} is needed")
    fmt = {"int8": 0, "e4m3": FMT_E4M3, "e2m1": FMT_E2M1}[codes] | \
        {"fp32": 0, "e8m0": FMT_E8M0, "e4m3": FMT_SCALE_E4M3}[scales] | \
        (FMT_WEIGHT_F32 if weight.dtype == torch.float32 else 0)
    ld_x = _rows("x", x, (rows, channels), _BF16, True, dev)
    wp = _vector("weight", weight, channels, _WEIGHT, dev)
    rp, ld_r, hp, ld_h = None, 0, None, 0
    if residual is not None:
        rp, ld_r = residual.data_ptr(), _rows("residual", residual, (rows, channels), _BF16, True, dev)
        if h is None:
            h = torch.empty((rows, channels), dtype=torch.bfloat16, device=dev)
        hp, ld_h = h.data_ptr(), _rows("h", h, (rows, channels), _BF16, True, dev)
    elif h is not None:
        raise ValueError("h is written only with a residual")
    else:
        h = x
    if e2m1:
        if q is None:
            q = torch.empty((rows, channels // 2), dtype=torch.uint8, device=dev)
        if s is None:
            s = torch.empty(fp4_scale_shape(rows, channels, scales), dtype=_SCALES[scales], device=dev)
        ld_q, ld_s = _codes("q", q, rows, channels, dev), 0
        _tiles("s", s, rows, channels, scales, dev)
    else:
        groups = -(-channels // (group_size or channels))
        if q is None:
            q = torch.empty((rows, channels), dtype=_CODES[codes], device=dev)
        if s is None:
            s = torch.empty((rows, groups), dtype=_SCALES[scales], device=dev)
        ld_q = _rows("q", q, (rows, channels), (_CODES[codes],), True, dev)
        ld_s = _rows("s", s, (rows, groups), (s.dtype,), True, dev)
    yp, ld_y = None, 0
    if y is not None:
        yp, ld_y = y.data_ptr(), _rows("y", y, (rows, channels), _BF16, True, dev)
    _call(sdq_rmsnorm_quant, dev, x.data_ptr(), ld_x, rp, ld_r, wp, hp, ld_h, q.data_ptr(), ld_q, s.data_ptr(), ld_s,
          yp, ld_y, None if rstd is None else _vector("rstd", rstd, rows, _F32, dev),
          _one("global_scale", global_scale, scales, dev), rows, channels, group_size, fmt, eps)
    return q, s, h


def rmsnorm_backward(grad_y: torch.Tensor, h: torch.Tensor, weight: torch.Tensor, rstd: torch.Tensor,
                     grad_h: Optional[torch.Tensor] = None, *, grad_x: Optional[torch.Tensor] = None,
                     grad_weight: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None
                     ) -> Tuple[torch.Tensor, torch.Tensor]:
    """The norm's gradients: (grad_x bf16 [rows, channels], grad_weight fp32
    [channels]).  grad_x is the gradient of x and of residual alike; ``grad_h``
    (bf16, optional) is the gradient that reaches h past the norm and is added
    to it.  h and rstd are what ``rmsnorm_quant`` returned and wrote.  grad_x may be
    grad_y, h or grad_h itself.  ``workspace``: uint8, at least
    ``sdq_rmsnorm_backward_workspace_bytes(rows, channels)`` bytes (allocated where
    not given); calls that overlap need one each."""
    if _made(_marshal.rmsnorm_backward(grad_y, h, weight, rstd, grad_h, grad_x, grad_weight, workspace),
             "sdq_rmsnorm_backward"):
        return grad_x, grad_weight
    rows, channels = _two_d("grad_y", grad_y)
    dev = grad_y.device
    need = sdq_rmsnorm_backward_workspace_bytes(rows, channels)
    if need == 0:
        raise ValueError(f"{channels} channels: a positive multiple of 16 is needed")
    ld_gy = _rows("grad_y", grad_y, (rows, channels), _BF16, True, dev)
    ld_h = _rows("h", h, (rows, channels), _BF16, True, dev)
    wp = _vector("weight", weight, channels, _WEIGHT, dev)
    sp = _vector("rstd", rstd, rows, _F32, dev)
    ghp, ld_gh = None, 0
    if grad_h is not None:
        ghp, ld_gh = grad_h.data_ptr(), _rows("grad_h", grad_h, (rows, channels), _BF16, True, dev)
    if grad_x is None:
        grad_x = torch.empty((rows, channels), dtype=torch.bfloat16, device=dev)
    if grad_weight is None:
        grad_weight = torch.empty((channels,), dtype=torch.float32, device=dev)
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    elif workspace.device != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace must be contiguous on {dev}")
    _call(sdq_rmsnorm_backward, dev, grad_y.data_ptr(), ld_gy, h.data_ptr(), ld_h, wp, sp, ghp, ld_gh,
          grad_x.data_ptr(), _rows("grad_x", grad_x, (rows, channels), _BF16, True, dev),
          _vector("grad_weight", grad_weight, channels, _F32, dev), rows, channels,
          FMT_WEIGHT_F32 if weight.dtype == torch.float32 else 0, workspace.data_ptr(),
          workspace.numel() * workspace.element_size())
    return grad_x, grad_weight


def quantize_fp4(x: torch.Tensor, scales: Optional[str] = None, axis: str = "rows", *,
                 q: Optional[torch.Tensor] = None, s: Optional[torch.Tensor] = None,
                 q_t: Optional[torch.Tensor] = None, s_t: Optional[torch.Tensor] = None,
                 global_scale: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, ...]:
    """4-bit codes and scale tiles of x (bf16 [rows, channels], channels a
    multiple of 32): along the rows, (q, s), with ``axis="rows"``; along the
    columns, transposed, (q_t, s_t), with "columns"; (q, s, q_t, s_t) with "both",
    reading x once.  q_t is [channels, R / 2] with R the rows rounded up to a
    multiple of 32; the missing ones count as zeros.  What is not given is
    allocated; ``scales`` ("e8m0", the default, or "e4m3") follows the given
    tiles."""
    if _made(_marshal.quantize_fp4(x, scales, axis, q, s, q_t, s_t, global_scale), "sdq_quantize_fp4"):
        return (q, s) if axis == "rows" else (q_t, s_t) if axis == "columns" else (q, s, q_t, s_t)
    rows, channels = _two_d("x", x)
    dev = x.device
    if axis not in ("rows", "columns", "both"):
        raise ValueError(f"axis is \"rows\", \"columns\" or \"both\", not {axis!r}")
    scales = _scales_of(s if s is not None else s_t, scales, "e8m0")
    fp4_scale_shape(rows, channels, scales)   # channels a multiple of 32, 4-bit scales
    ld_x = _rows("x", x, (rows, channels), _BF16, True, dev)
    padded = -(-rows // 32) * 32
    out: list = []
    args: list = []
    for on, what, r, k, codes, tiles in ((axis != "columns", "", rows, channels, q, s),
                                         (axis != "rows", "_t", channels, padded, q_t, s_t)):
        if not on:
            if codes is not None or tiles is not None:
                raise ValueError(f"q{what} and s{what} are not written with axis={axis!r}")
            args += [None, 0, None]
            continue
        if codes is None:
            codes = torch.empty((r, k // 2), dtype=torch.uint8, device=dev)
        if tiles is None:   # (no rows: no columns either, and no tiles)
            tiles = torch.empty(fp4_scale_shape(r, k, scales) if k else (-(-r // 128), 0, 512),
                                dtype=_SCALES[scales], device=dev)
        out += [codes, tiles]
        if k:
            args += [codes.data_ptr(), _codes("q" + what, codes, r, k, dev), _tiles("s" + what, tiles, r, k, scales, dev)]
        else:
            args += [None, 0, None]
    _call(sdq_quantize_fp4, dev, x.data_ptr(), ld_x, *args, _one("global_scale", global_scale, scales, dev), rows,
          channels, _FP4_FORMAT[scales])
    return tuple(out)


def dequantize_fp4(q: torch.Tensor, s: torch.Tensor, global_scale: Optional[torch.Tensor] = None, *,
                   out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The values of 4-bit codes and scale tiles, bf16 [rows, k]."""
    if _made(_marshal.dequantize_fp4(q, s, global_scale, out), "sdq_dequantize_fp4"):
        return out
    rows, k = _two_d("q", q)
    k *= 2
    dev = q.device
    scales = _scales_of(s, None, "e8m0")
    _length(k)
    ld_q, sp = _codes("q", q, rows, k, dev), _tiles("s", s, rows, k, scales, dev)
    if out is None:
        out = torch.empty((rows, k), dtype=torch.bfloat16, device=dev)
    _call(sdq_dequantize_fp4, dev, q.data_ptr(), ld_q, sp, _one("global_scale", global_scale, scales, dev),
          out.data_ptr(), _rows("out", out, (rows, k), _BF16, True, dev), rows, k, _FP4_FORMAT[scales])
    return out


def matmul_fp4(a: torch.Tensor, a_s: torch.Tensor, b: torch.Tensor, b_s: torch.Tensor, *,
               a_global: Optional[torch.Tensor] = None, b_global: Optional[torch.Tensor] = None,
               out: Optional[torch.Tensor] = None, out_dtype: Optional[torch.dtype] = None) -> torch.Tensor:
    """The product of two 4-bit operands, out[i, j] = sum_k a[i, k] b[j, k],
    summed in fp32: a [m, k] and b [n, k] as codes and scale tiles of one format,
    out [m, n] bf16 (the default) or float32."""
    if _made(_marshal.matmul_fp4(a, a_s, b, b_s, a_global, b_global, out, out_dtype), "sdq_matmul_fp4"):
        return out
    m, ka = _two_d("a", a)
    n, kb = _two_d("b", b)
    if ka != kb:
        raise ValueError(f"a has rows of {2 * ka} codes and b of {2 * kb}")
    k, dev = 2 * ka, a.device
    scales = _scales_of(a_s, None, "e8m0")
    _length(k)
    ld_a, ld_b = _codes("a", a, m, k, dev), _codes("b", b, n, k, dev)
    ap, bp = _tiles("a_s", a_s, m, k, scales, dev), _tiles("b_s", b_s, n, k, scales, dev)
    if out is None:
        out = torch.empty((m, n), dtype=out_dtype or torch.bfloat16, device=dev)
    elif out_dtype is not None and out.dtype != out_dtype:
        raise ValueError(f"out is {out.dtype}, not {out_dtype}")
    ld_out = _rows("out", out, (m, n), _WEIGHT, True, dev)
    _call(sdq_matmul_fp4, dev, a.data_ptr(), ld_a, ap, _one("a_global", a_global, scales, dev), b.data_ptr(), ld_b, bp,
          _one("b_global", b_global, scales, dev), out.data_ptr(), ld_out, m, n, k,
          _FP4_FORMAT[scales] | (FMT_OUT_F32 if out.dtype == torch.float32 else 0))
    return out
