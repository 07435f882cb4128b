"""Argument checks and the call itself, shared by the routed-expert and 8-bit operators.

Small calls (a decode step's) are bounded by the host: the checks read only tensor attributes
(about 0.05 us each), and the current stream comes as the raw handle (0.1 us; a
torch.cuda.Stream object costs 2.8 us), so that a call takes about 8 us, most of it the launch and
torch's allocation of the outputs."""
from __future__ import annotations

import torch

from ._lib import FP8Q_OUT_BF16, FP8Q_OUT_F32, check

CODE = {torch.float32: FP8Q_OUT_F32, torch.bfloat16: FP8Q_OUT_BF16}
FLOATS = (torch.float32, torch.bfloat16)

_raw_stream = torch._C._cuda_getCurrentRawStream
_current_device = torch._C._cuda_getDevice


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


def need_float(t, name: str, dtype=FLOATS, shape=None, device=None) -> None:
    """need() for a float32 or bfloat16 tensor, aligned to its elements."""
    need(t, name, dtype, shape, 1, device)
    if t.data_ptr() % t.element_size():
        raise ValueError(f"{name} must be {t.element_size()}-byte aligned")


def launch(fn: str, call, t: torch.Tensor, *args) -> None:
    """Calls the library on t's device and torch's current stream there."""
    index = t.get_device()
    if _current_device() == index:
        status = call(*args, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            status = call(*args, _raw_stream(index))
    if status:
        check(fn, status)
