"""Argument checks and the call that the operators beside the expert layer
share.  A checked call costs a few microseconds of host time, most of it the
launch, so checks read attributes once and build messages only on failure."""

from __future__ import annotations

import torch

#: torch dtype -> MOE_Q4_DTYPE_*
DTYPES = {torch.bfloat16: 0, torch.float32: 1, torch.float16: 2}


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
    if ld < cols:
        if rows > 1:
            raise ValueError(f"{name} has overlapping rows")
        ld = cols
    return t.data_ptr(), ld if rows > 1 else cols


def array(t, dtype, shape, name: str, device) -> int:
    """Pointer of a contiguous device tensor of this type (one of these types), shape and device."""
    if isinstance(t, torch.Tensor) and t.shape == shape and t.device == device and t.is_contiguous() and \
            (t.dtype is dtype or (type(dtype) is tuple and t.dtype in dtype)):
        return t.data_ptr()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")


def new(shape, strides, dtype, device):
    """An uninitialised contiguous tensor (with its strides given, torch takes a shorter way)."""
    return torch.empty_strided(shape, strides, dtype=dtype, device=device)


def on_stream(stream, tensor):
    """Context of a call on a stream of the caller's (a torch stream or a HIP
    handle): what the call allocates belongs to that stream too, so neither
    earlier work on the current stream nor later work there shares its memory."""
    device = tensor.device
    if not isinstance(stream, torch.cuda.Stream):
        handle = int(stream)
        stream = torch.cuda.ExternalStream(handle, device=device) if handle else torch.cuda.default_stream(device)
    elif stream.device != device:
        raise ValueError(f"stream is on {stream.device}, the tensors on {device}")
    return torch.cuda.stream(stream)


def current_handle(device) -> int:
    """HIP handle of the device's current stream."""
    return torch._C._cuda_getCurrentRawStream(device.index)


def call(fn, args, device, handle) -> int:
    """Runs fn(*args, handle) with the tensors' device current; returns its status."""
    if torch._C._cuda_getDevice() == device.index:
        return fn(*args, handle)
    with torch.cuda.device(device):
        return fn(*args, handle)
