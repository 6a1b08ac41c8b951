"""Gated feed-forward block of dense weights, with its gradient (``moe_glu``,
``moe_glu_backward``)."""

from __future__ import annotations

import torch

import quantized_expert_gather_amd as _q

from ._args import DTYPES, array, call, current_handle, new, no_tangent, on_stream, plane, scratch, written
from .router import _not_captured

_X = (torch.bfloat16, torch.float16)


def moe_glu_workspace_bytes(T: int, H: int, I: int) -> int:
    return int(_q.lib().moe_glu_workspace_bytes(T, H, I))


def moe_glu_backward_workspace_bytes(T: int, H: int, I: int, saved: bool = True) -> int:
    return int(_q.lib().moe_glu_backward_workspace_bytes(T, H, I, 1 if saved else 0))


def _wants(t) -> bool:
    return isinstance(t, torch.Tensor) and t.requires_grad


def _operands(x, wg, wu):
    """Checked x and weights: (pointers and strides of a call, T, H, I)."""
    xt = x.dtype if isinstance(x, torch.Tensor) else None
    xp, ldx, (T, H) = plane(x, _X, "x")
    gp, ldw, shape = plane(wg, (xt,), "wg")
    up, ldu, given = plane(wu, (xt,), "wu")
    if shape[1] != H or given != shape or wg.device != x.device or wu.device != x.device:
        raise ValueError(f"wg and wu must be [I, {H}] on {x.device}")
    if ldw != ldu:
        raise ValueError("wg and wu must have the same row stride")
    return (DTYPES[xt], xp, ldx, gp, up, ldw), T, H, shape[0]


def _result(out, shape, dtype, name, device):
    """(tensor, pointer, row stride) of a result, made here where none is given."""
    if out is None:
        out = new(shape, (shape[1], 1), dtype, device)
        return out, out.data_ptr(), shape[1]
    p, ld, given = plane(out, (dtype,), name)
    if given != shape or out.device != device:
        raise ValueError(f"{name} must be {list(shape)} on {device}")
    return out, p, ld


def _scratch(workspace, need, device):
    """(tensor kept alive, pointer, bytes) of a call's workspace."""
    if workspace is not None:
        return workspace, *scratch(workspace, device)
    if not need:
        return None, 0, 0
    workspace = new((need,), (1,), torch.uint8, device)
    return workspace, workspace.data_ptr(), need


def _forward(x, wg, wu, out, saved, workspace, keep=False):
    """(h, the projections: `saved`, or made here with `keep`)."""
    head, T, H, I = _operands(x, wg, wu)
    dev = x.device
    given_outputs = out, saved
    if keep:
        saved = new((2, T, I), (T * I, I, 1), torch.float32, dev)
    out, hp, ldh = _result(out, (T, I), x.dtype, "out", dev)
    sp = 0 if saved is None else array(saved, torch.float32, (2, T, I), "saved", dev)
    lib = _q.lib()
    workspace, wsp, wsn = _scratch(workspace, lib.moe_glu_workspace_bytes(T, H, I), dev)
    st = call(lib.moe_glu_forward, (*head, T, H, I, hp, ldh, sp, wsp, wsn), dev, current_handle(dev))
    if st:
        raise _q.MoeQ4Error(st, "moe_glu_forward")
    written(*given_outputs)
    return out, saved


class _GluFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, wg, wu, recompute, workspace):
        h, saved = _forward(x, wg, wu, None, None, workspace, not recompute)
        ctx.save_for_backward(x, wg, wu, saved)
        return h

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dh):
        _not_captured("moe_glu_backward")
        x, wg, wu, saved = ctx.saved_tensors
        need_x, need_w = ctx.needs_input_grad[0], ctx.needs_input_grad[1] or ctx.needs_input_grad[2]
        dx, dwg, dwu = _backward(x, wg, wu, dh.contiguous(), saved, None, None, None, None, need_x, need_w)
        return dx, dwg, dwu, None, None


def moe_glu(x, wg, wu, out=None, saved=None, recompute: bool = False, workspace=None, stream=None) -> torch.Tensor:
    """``silu(x @ wg.T) * (x @ wu.T)`` (see include/moe_q4.h for the contract).

    x bf16 or fp16 [T, H], wg and wu [I, H] of the same type (contiguous rows;
    row strides multiples of 8, the same for both weights, which may be the
    halves of one matrix); H and I multiples of 8.  Returns h [T, I].

    h carries a gradient to x, wg and wu where one of these requires one; an
    output tensor, which cannot, is refused then.  The two projections are
    kept for it in fp32 (8 bytes for each of h's elements), or computed again
    with ``recompute``.  A step recorded into a graph passes a tensor ``saved``
    (fp32 [2, T, I]) that the call fills and calls :func:`moe_glu_backward`
    itself (backward() refuses there).  ``stream`` (a torch stream or a HIP
    handle) is as ``with torch.cuda.stream(stream)`` around the call.
    """
    if stream is not None and isinstance(x, torch.Tensor):
        with on_stream(stream, x):
            return moe_glu(x, wg, wu, out, saved, recompute, workspace)
    no_tangent("moe_glu", x, wg, wu)
    if torch.is_grad_enabled() and (_wants(x) or _wants(wg) or _wants(wu)):
        if out is not None or saved is not None:
            raise RuntimeError("moe_glu: given output tensors carry no gradient, but an input requires one")
        return _GluFunction.apply(x, wg, wu, recompute, workspace)
    return _forward(x, wg, wu, out, saved, workspace)[0]


def _backward(x, wg, wu, dh, saved, dx, dwg, dwu, workspace, need_x, need_w):
    head, T, H, I = _operands(x, wg, wu)
    dev = x.device
    given_outputs = dx, dwg, dwu
    ep, lde, given = plane(dh, (x.dtype,), "dh")
    if given != (T, I) or dh.device != dev:
        raise ValueError(f"dh must be [{T}, {I}] on {dev}")
    sp = 0 if saved is None else array(saved, torch.float32, (2, T, I), "saved", dev)
    dp = ldd = gp = up = 0
    if need_x:
        dx, dp, ldd = _result(dx, (T, H), x.dtype, "dx", dev)
    if need_w:
        dwg = new((I, H), (H, 1), x.dtype, dev) if dwg is None else dwg
        dwu = new((I, H), (H, 1), x.dtype, dev) if dwu is None else dwu
        gp = array(dwg, x.dtype, (I, H), "dwg", dev)
        up = array(dwu, x.dtype, (I, H), "dwu", dev)
    lib = _q.lib()
    need = lib.moe_glu_backward_workspace_bytes(T, H, I, 0 if saved is None else 1)
    workspace, wsp, wsn = _scratch(workspace, need, dev)
    st = call(lib.moe_glu_backward, (*head, ep, lde, sp, T, H, I, dp, ldd, gp, up, wsp, wsn), dev, current_handle(dev))
    if st:
        raise _q.MoeQ4Error(st, "moe_glu_backward")
    written(*given_outputs)
    return dx, dwg, dwu


def moe_glu_backward(x, wg, wu, dh, saved=None, dx=None, dwg=None, dwu=None, workspace=None, stream=None):
    """Gradient of :func:`moe_glu`: from dh [T, I] (x's type) and the ``saved``
    projections of the forward (computed again where None), returns (dx, dwg,
    dwu) in x's type."""
    if stream is not None and isinstance(x, torch.Tensor):
        with on_stream(stream, x):
            return moe_glu_backward(x, wg, wu, dh, saved, dx, dwg, dwu, workspace)
    return _backward(x, wg, wu, dh, saved, dx, dwg, dwu, workspace, True, True)
