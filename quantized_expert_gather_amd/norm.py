"""Root-mean-square norm with the residual's addition and 8-bit output, its
gradient, and the quantization into 8 bits (``moe_rms_norm``,
``moe_rms_norm_fp8``, ``moe_rms_norm_backward``, ``moe_quantize_fp8``)."""

from __future__ import annotations

import torch

import quantized_expert_gather_amd as _q

from ._args import DTYPES, array, call, current_handle, new, no_tangent, on_stream, plane, scratch, written
from .router import _not_captured

F8 = torch.float8_e4m3fn
_F8S = (F8,)
_TYPES = tuple(DTYPES)


def _weight(weight, H, device):
    """(pointer, MOE_Q4_DTYPE_*) of a norm's weight, or (0, 0)."""
    if weight is None:
        return 0, 0
    return array(weight, _TYPES, (H,), "weight", device), DTYPES[weight.dtype]


def _like(t, shape, out, dtypes, name):
    """(tensor, pointer, row stride) of a matrix of t's shape and device, made here where none is given."""
    if out is None:
        out = new(shape, (shape[1], 1), dtypes[0], t.device)
        return out, out.data_ptr(), shape[1]
    p, ld, given = plane(out, dtypes, name)
    if given != shape or out.device != t.device:
        raise ValueError(f"{name} must be {list(shape)} on {t.device}")
    return out, p, ld


def _norm(x, weight, residual, eps, total, y, want_y, codes, scales, want_codes, where):
    given_outputs = total, y, codes, scales
    xp, ldx, shape = plane(x, _TYPES, "x")
    T, H = shape
    dev = x.device
    xt = x.dtype
    wp, wd = _weight(weight, H, dev)
    rp = ldr = rd = tp = ldt = 0
    if residual is not None:
        rt = residual.dtype if isinstance(residual, torch.Tensor) else None
        rp, ldr, given = plane(residual, (xt, torch.float32), "residual")
        if given != shape or residual.device != dev:
            raise ValueError("residual must have the shape and device of x")
        rd = DTYPES[rt]
        total, tp, ldt = _like(x, shape, total, (rt,), "total")
    elif total is not None:
        raise ValueError("total without a residual")
    yp = yd = ldy = cp = ldc = sp = 0
    if want_y:
        y, yp, ldy = _like(x, shape, y, want_y, "out")
        yd = DTYPES[y.dtype]
    if want_codes:
        codes, cp, ldc = _like(x, shape, codes, _F8S, "codes")
        G = (H + 127) // 128
        if scales is None:
            scales = new((T, G), (G, 1), torch.float32, dev)
            sp = scales.data_ptr()
        else:
            sp = array(scales, torch.float32, (T, G), "scales", dev)
    st = call(_q.lib().moe_rms_norm, (xp, DTYPES[xt], ldx, rp, rd, ldr, wp, wd, T, H, eps, tp, ldt, yp, yd, ldy, cp, ldc, sp), dev,
              current_handle(dev))
    if st:
        raise _q.MoeQ4Error(st, where)
    written(*given_outputs)
    return y, total, codes, scales


def _wants(t) -> bool:
    return isinstance(t, torch.Tensor) and t.requires_grad


def _out_types(x, out, out_dtype):
    if not isinstance(x, torch.Tensor):
        raise TypeError("x must be a torch.Tensor")
    if out is not None:
        if not isinstance(out, torch.Tensor):
            raise TypeError("out must be a torch.Tensor")
        if out_dtype not in (None, out.dtype):
            raise ValueError("out is not of out_dtype")
        return _TYPES
    od = x.dtype if out_dtype is None else out_dtype
    if od not in DTYPES:
        raise TypeError(f"out_dtype {od} is not one of {tuple(DTYPES)}")
    return (od,)


class _NormFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, residual, eps, out_dtype):
        y, total, _, _ = _norm(x, weight, residual, eps, None, None, _out_types(x, None, out_dtype), None, None, False,
                               "moe_rms_norm")
        ctx.set_materialize_grads(False)
        ctx.save_for_backward(x if residual is None else total, weight)
        ctx.how = (eps, x.dtype, residual is not None)
        return y if residual is None else (y, total)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy, dtotal=None):
        _not_captured("moe_rms_norm_backward")
        total, weight = ctx.saved_tensors
        eps, x_dtype, has_residual = ctx.how
        if dy is None:  # the sum alone was used
            dx, dw = dtotal, None
        else:
            dx, dw = _back(total, weight, dy.contiguous(), None if dtotal is None else dtotal.contiguous(), eps, None, None,
                           None, weight is not None and ctx.needs_input_grad[1])
        return None if dx is None else dx.to(x_dtype), dw, dx if has_residual else None, None, None


def moe_rms_norm(x, weight=None, residual=None, eps: float = 1e-6, total=None, out=None, out_dtype=None, stream=None):
    """Norm of ``x``, or of ``x + residual`` (see include/moe_q4.h).

    x [T, H] bf16, fp16 or fp32 with contiguous rows; residual [T, H] of x's
    type or fp32; weight [H] of any of the three, or None.  Returns y in
    ``out_dtype`` (x's type if not given), and with a residual (y, total):
    ``total`` is the sum in the residual's type; passing ``total=residual``
    adds in place.  Autograd sees given tensors as changed: a backward pass
    that needs what they held raises.

    y and total carry gradients to x, weight and residual where one of these
    requires one; given outputs, which cannot, are refused then.  A step
    recorded into a graph calls :func:`moe_rms_norm_backward` itself
    (backward() refuses there).  ``stream`` (a torch stream or a HIP handle) is
    as ``with torch.cuda.stream(stream)`` around the call.
    """
    if stream is not None and isinstance(x, torch.Tensor):
        with on_stream(stream, x):
            return moe_rms_norm(x, weight, residual, eps, total, out, out_dtype)
    no_tangent("moe_rms_norm", x, weight, residual)
    if torch.is_grad_enabled() and (_wants(x) or _wants(weight) or _wants(residual)):
        if total is not None or out is not None:
            raise RuntimeError("moe_rms_norm: given output tensors carry no gradient, but an input requires one")
        return _NormFunction.apply(x, weight, residual, eps, out_dtype)
    y, total, _, _ = _norm(x, weight, residual, eps, total, out, _out_types(x, out, out_dtype), None, None, False,
                           "moe_rms_norm")
    return y if residual is None else (y, total)


class _StreamFunction(torch.autograd.Function):
    """x + residual, which `add` computes beside the codes."""

    @staticmethod
    def forward(ctx, x, residual, add):
        ctx.x_dtype = x.dtype
        return add(x, residual)

    @staticmethod
    def backward(ctx, dtotal):
        if torch.cuda.is_current_stream_capturing():  # (as _not_captured)
            raise RuntimeError("backward() of a graph-captured step: moe_rms_norm_fp8's total has the gradient of x and residual itself")
        return dtotal.to(ctx.x_dtype), dtotal, None


def moe_rms_norm_fp8(x, weight=None, residual=None, eps: float = 1e-6, total=None, codes=None, scales=None, stream=None):
    """:func:`moe_rms_norm` with an output in 8 bits: returns (codes
    float8_e4m3fn [T, H], scales fp32 [T, ceil(H / 128)]) as
    :func:`moe_linear_fp8_forward` takes them, and with a residual (codes,
    scales, total).  codes and scales carry no gradient; total, the stream that
    goes on, carries its own to x and residual where one of these requires one
    (a given total, which cannot, is refused then)."""
    if stream is not None and isinstance(x, torch.Tensor):
        with on_stream(stream, x):
            return moe_rms_norm_fp8(x, weight, residual, eps, total, codes, scales)
    if residual is not None:
        no_tangent("moe_rms_norm_fp8", x, residual)
    if residual is not None and torch.is_grad_enabled() and (_wants(x) or _wants(residual)):
        if total is not None:
            raise RuntimeError("moe_rms_norm_fp8: a given total carries no gradient, but x or residual requires one")
        made = []

        def add(x, residual):
            _, t, c, s = _norm(x, weight, residual, eps, None, None, (), codes, scales, True, "moe_rms_norm_fp8")
            made.extend((c, s))
            return t

        total = _StreamFunction.apply(x, residual, add)
        return (*made, total)
    _, total, codes, scales = _norm(x, weight, residual, eps, total, None, (), codes, scales, True, "moe_rms_norm_fp8")
    return (codes, scales) if residual is None else (codes, scales, total)


def moe_rms_norm_backward_workspace_bytes(T: int, H: int) -> int:
    return int(_q.lib().moe_rms_norm_backward_workspace_bytes(T, H))


def _back(total, weight, dy, dtotal, eps, dx, dweight, workspace, want_dweight):
    given_outputs = dx, dweight
    rp, ldr, shape = plane(total, _TYPES, "total")
    T, H = shape
    dev = total.device
    wp, wd = _weight(weight, H, dev)
    yp, ldy, given = plane(dy, _TYPES, "dy")
    if given != shape or dy.device != dev:
        raise ValueError("dy must have the shape and device of total")
    tp = ldt = 0
    if dtotal is not None:
        tp, ldt, given = plane(dtotal, (total.dtype,), "dtotal")
        if given != shape or dtotal.device != dev:
            raise ValueError("dtotal must have the shape and device of total")
    dx, dp, ldd = _like(total, shape, dx, (total.dtype,), "dx")
    gp = wsp = wsn = 0
    if dweight is not None and not want_dweight:
        raise ValueError("dweight without a weight")
    if want_dweight:
        if dweight is None:
            dweight = new((H,), (1,), weight.dtype, dev)
            gp = dweight.data_ptr()
        else:
            gp = array(dweight, weight.dtype, (H,), "dweight", dev)
        if workspace is None:
            wsn = _q.lib().moe_rms_norm_backward_workspace_bytes(T, H)
            workspace = new((wsn,), (1,), torch.uint8, dev)
            wsp = workspace.data_ptr()
        else:
            wsp, wsn = scratch(workspace, dev)
    args = (rp, DTYPES[total.dtype], ldr, wp, wd, yp, DTYPES[dy.dtype], ldy, tp, ldt, T, H, eps, dp, ldd, gp, wsp, wsn)
    st = call(_q.lib().moe_rms_norm_backward, args, dev, current_handle(dev))
    if st:
        raise _q.MoeQ4Error(st, "moe_rms_norm_backward")
    written(*given_outputs)
    return dx, dweight


def moe_rms_norm_backward(total, weight, dy, dtotal=None, eps: float = 1e-6, dx=None, dweight=None, workspace=None,
                          stream=None):
    """Gradient of :func:`moe_rms_norm`: ``total`` is the sum that it returned (x
    where there was no residual), dy [T, H] the gradient of y, dtotal (total's
    type, or None) that of total.  Returns (dx in total's type, which is the
    gradient of x and of the residual, and dweight in weight's type, None
    where weight is None)."""
    if stream is not None and isinstance(total, torch.Tensor):
        with on_stream(stream, total):
            return moe_rms_norm_backward(total, weight, dy, dtotal, eps, dx, dweight, workspace)
    return _back(total, weight, dy, dtotal, eps, dx, dweight, workspace, weight is not None)


def moe_quantize_fp8(x, block_rows: int = 1, codes=None, scales=None, stream=None):
    """E4M3 codes and fp32 scales of ``x`` [T, K] (bf16, fp16 or fp32, contiguous
    rows) for blocks of 1 x 128 (activations) or, with ``block_rows=128``, of
    128 x 128 (weights), as :func:`moe_linear_fp8_forward` takes them: (codes
    float8_e4m3fn [T, K], scales [ceil(T / block_rows), ceil(K / 128)])."""
    if stream is not None and isinstance(x, torch.Tensor):
        with on_stream(stream, x):
            return moe_quantize_fp8(x, block_rows, codes, scales)
    xp, ldx, given = plane(x, _TYPES, "x")
    T, K = given
    dev = x.device
    given_outputs = codes, scales
    rows = int(block_rows)
    if rows not in (1, 128):
        raise ValueError(f"block_rows {block_rows} is neither 1 nor 128")
    codes, cp, ldc = _like(x, given, codes, _F8S, "codes")
    shape = ((T + rows - 1) // rows, (K + 127) // 128)
    if scales is None:
        scales = new(shape, (shape[1], 1), torch.float32, dev)
        sp = scales.data_ptr()
    else:
        sp = array(scales, torch.float32, shape, "scales", dev)
    st = call(_q.lib().moe_quantize_fp8, (xp, DTYPES[x.dtype], ldx, T, K, rows, cp, ldc, sp), dev, current_handle(dev))
    if st:
        raise _q.MoeQ4Error(st, "moe_quantize_fp8")
    written(*given_outputs)
    return codes, scales
