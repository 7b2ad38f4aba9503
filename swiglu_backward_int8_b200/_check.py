"""Argument checks that the entry points share."""
from __future__ import annotations

import torch


def _rows(name: str, t: torch.Tensor, shape, dtypes, want_cuda: bool, device) -> int:
    """Check a 2-D row-major operand (rows may be padded: stride(0) >= its
    row); returns its leading dimension in elements."""
    if t.dim() != 2 or tuple(t.shape) != tuple(shape) or t.dtype not in dtypes:
        raise ValueError(f"{name}: expected {' or '.join(map(str, dtypes))} {tuple(shape)}, "
                         f"got {t.dtype} {tuple(t.shape)}")
    if t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError(f"{name} must have unit stride along its rows")
    if t.shape[0] > 1 and t.stride(0) < t.shape[1]:
        raise ValueError(f"{name}: rows overlap (stride {t.stride(0)} < row length {t.shape[1]})")
    if not want_cuda and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous for the host-buffer entry points")
    if want_cuda and (not t.is_cuda or t.device != device):
        raise ValueError(f"{name} must be a CUDA tensor on {device}")
    if not want_cuda and t.is_cuda:
        raise ValueError(f"{name} must be a host tensor")
    return int(t.stride(0)) if t.shape[0] > 1 else int(t.shape[1])
