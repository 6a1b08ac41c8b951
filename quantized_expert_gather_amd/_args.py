"""Argument checks that the operators beside the expert layer share."""

from __future__ import annotations

import contextlib

import torch

#: torch dtype -> MOE_Q4_DTYPE_*
DTYPES = {torch.bfloat16: 0, torch.float32: 1, torch.float16: 2}

_same_device = contextlib.nullcontext()


def matrix(t, dtypes, name: str):
    """A device matrix with contiguous rows: (pointer, row stride in elements)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor (got {t.device})")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} has dtype {t.dtype}, expected one of {tuple(dtypes)}")
    if t.dim() != 2:
        raise ValueError(f"{name} must have two dimensions (got {t.dim()})")
    rows, cols = t.shape
    ld, step = t.stride()
    if step != 1 and cols > 1:
        raise ValueError(f"{name} must have contiguous rows")
    if rows <= 1 or ld < cols:
        if rows > 1:
            raise ValueError(f"{name} has overlapping rows")
        ld = cols
    return t.data_ptr(), ld


def array(t, dtype, shape, name: str, device) -> int:
    """Pointer of a contiguous device tensor of this type, shape and device."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.dtype != dtype and not (isinstance(dtype, tuple) and t.dtype in dtype):
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def on_device(device):
    """The tensors' device made the current one, if it is not."""
    return _same_device if device.index == torch.cuda.current_device() else torch.cuda.device(device)


def stream_of(stream, device):
    """(HIP stream handle, torch stream or None): the caller's stream, or the
    device's current one."""
    if stream is None:
        return torch.cuda.current_stream(device).cuda_stream, None
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream, stream
    handle = int(stream)
    return handle, torch.cuda.ExternalStream(handle, device=device)


def used_on(side, *tensors) -> None:
    """Tensors that were allocated here and are used on another stream keep
    their memory until that stream has passed the work enqueued so far."""
    if side is not None:
        for t in tensors:
            if t is not None:
                t.record_stream(side)
