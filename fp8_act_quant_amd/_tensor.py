"""Argument checks shared by the routed-expert and 8-bit integer operators."""
from __future__ import annotations

import torch

from ._lib import FP8Q_OUT_BF16, FP8Q_OUT_F32

CODE = {torch.float32: FP8Q_OUT_F32, torch.bfloat16: FP8Q_OUT_BF16}


def need(t, name: str, dtype, shape=None, align: int = 4, device=None) -> None:
    """t is a contiguous GPU tensor of dtype (or one of them), shape and alignment."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if t.dtype not in dtype if isinstance(dtype, tuple) else t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.data_ptr() % align:
        raise ValueError(f"{name} must be {align}-byte aligned")


def launch(fn: str, call, t: torch.Tensor, *args) -> None:
    """Calls the library on t's device and torch's current stream there."""
    from ._lib import check
    if torch.cuda.current_device() == t.device.index:
        status = call(*args, torch.cuda.current_stream().cuda_stream)
    else:
        with torch.cuda.device(t.device):
            status = call(*args, torch.cuda.current_stream().cuda_stream)
    check(fn, status)
