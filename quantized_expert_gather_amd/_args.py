"""Argument checks and the call that the operators beside the expert layer
share.  A checked call costs a few microseconds of host time, most of it the
launch, so checks read attributes once and build messages only on failure."""

from __future__ import annotations

import torch
from torch.autograd import forward_ad

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


def plane(t, dtypes, name: str):
    """As :func:`matrix`, with the shape: (pointer, row stride, shape).  The usual
    matrix, contiguous and as it should be, is asked least."""
    if isinstance(t, torch.Tensor) and t.is_cuda and t.dtype in dtypes and t.dim() == 2 and t.is_contiguous():
        shape = t.shape
        return t.data_ptr(), shape[1], shape
    p, ld = matrix(t, dtypes, name)
    return p, ld, t.shape


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


def scratch(t, device):
    """(pointer, bytes) of a given workspace."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("workspace must be a torch.Tensor")
    n = t.numel()
    return array(t, torch.uint8, (n,), "workspace", device), n


def new(shape, strides, dtype, device):
    """An uninitialised contiguous tensor (with its strides given, torch takes a shorter way)."""
    return torch.empty_strided(shape, strides, dtype=dtype, device=device)


def no_tangent(where, *tensors):
    """Refuses dual tensors of forward-mode differentiation, whose tangents a
    result would lose."""
    if forward_ad._current_level >= 0:
        for t in tensors:
            if isinstance(t, torch.Tensor) and forward_ad.unpack_dual(t).tangent is not None:
                raise RuntimeError(f"{where} has no forward-mode derivative, but an input has a tangent")


def written(*given):
    """Marks the output tensors that a caller gave (not None) as changed in place,
    as torch's own operations do: a backward pass that saved one then raises."""
    for t in given:
        if t is not None:
            torch.autograd.graph.increment_version(t)


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
