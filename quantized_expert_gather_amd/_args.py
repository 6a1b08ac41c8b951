"""Argument checks and the call that the operators beside the expert layer
share.  A checked call costs a few microseconds of host time, most of it the
launch, so checks read attributes once and build messages only on failure."""

from __future__ import annotations

import torch

#: torch dtype -> MOE_Q4_DTYPE_*
DTYPES = {torch.bfloat16: 0, torch.float32: 1, torch.float16: 2}

_raw_stream = torch._C._cuda_getCurrentRawStream if hasattr(torch._C, "_cuda_getCurrentRawStream") else None


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


def stream_handle(stream, device) -> int:
    """HIP stream handle of a call: the caller's stream, or the device's current one."""
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(device.index)
        return torch.cuda.current_stream(device).cuda_stream
    return stream.cuda_stream if isinstance(stream, torch.cuda.Stream) else int(stream)


def call(fn, args, device, stream, made) -> int:
    """Runs fn(*args, stream) with the tensors' device current; returns its status.

    Tensors that were allocated here (``made``; None entries skipped) and are
    used on another stream than the current one keep their memory until that
    stream has passed the work enqueued so far.
    """
    handle = stream_handle(stream, device)
    if torch._C._cuda_getDevice() == device.index:
        st = fn(*args, handle)
    else:
        with torch.cuda.device(device):
            st = fn(*args, handle)
    if stream is not None:
        side = stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(handle, device=device)
        for t in made:
            if t is not None:
                t.record_stream(side)
    return st
