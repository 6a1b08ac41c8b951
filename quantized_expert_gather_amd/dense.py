"""Dense products with 4-bit weights (``moe_linear_codec_forward``)."""

from __future__ import annotations

import torch

import quantized_expert_gather_amd as _q

from ._args import DTYPES, array, call, current_handle, matrix, new, on_stream

_X = (torch.bfloat16, torch.float16)
_CODES = (torch.int32, getattr(torch, "uint32", torch.int32))
#: 4-bit codec (name or MOE_Q4_CODEC_*) -> MOE_Q4_CODEC_*, inputs per scale, scale type, whether it has biases
_SPECS = {}
for _name, (_code, _gs, _bits) in _q.CODECS.items():
    if _bits == 4:
        _affine = _name.startswith("affine")
        _SPECS[_name] = _SPECS[_code] = (_code, _gs, torch.bfloat16 if _affine else torch.uint8, _affine)


def moe_linear_codec_workspace_bytes(codec, L: int, N: int, K: int) -> int:
    return int(_q.lib().moe_linear_codec_workspace_bytes(_q._codec_id(codec), L, N, K))


def _linear_args(codec, x, w, s, b, bias, out, out_dtype, workspace):
    """Checked arguments of a call up to the stream, out, and the workspace made here."""
    spec = _SPECS.get(codec)
    if spec is None:
        raise ValueError(f"codec {codec!r} has no 4-bit dense product")
    code, gs, scale_type, affine = spec
    xp, ldx = matrix(x, _X, "x")
    L, K = x.shape
    dev = x.device
    if not isinstance(w, torch.Tensor) or w.dim() != 2:
        raise ValueError("w [N, K/8] expected")
    N = w.shape[0]
    if K % gs:
        raise _q.MoeQ4Error(_q.MOE_Q4_ERR_UNSUPPORTED, "moe_linear_codec_forward")
    if w.dtype in _CODES and w.shape[1] == K // 8 and w.device == dev and w.is_contiguous():
        wp = w.data_ptr()
    else:
        wp = array(w, _CODES, (N, K // 8), "w", dev)
    rows = (N, K // gs)
    sp = array(s, scale_type, rows, "s", dev)
    bp = array(b, torch.bfloat16, rows, "b", dev) if affine else 0
    ap = 0 if bias is None else array(bias, torch.float32, (N,), "bias", dev)
    if out is None:
        od = x.dtype if out_dtype is None else out_dtype
        if od not in DTYPES:
            raise TypeError(f"out_dtype {od} is not one of {tuple(DTYPES)}")
        out = new((L, N), (N, 1), od, dev)
        op, ldo = out.data_ptr(), N
    else:
        op, ldo = matrix(out, DTYPES, "out")
        od = out.dtype
        if out.shape != (L, N) or out.device != dev or out_dtype not in (None, od):
            raise ValueError(f"out must be [{L}, {N}] on {dev}, of out_dtype")
    need = _q.lib().moe_linear_codec_workspace_bytes(code, L, N, K) if workspace is None else 0
    scratch = None
    wsp = wsn = 0
    if workspace is not None:
        wsn = workspace.numel()
        wsp = array(workspace, torch.uint8, (wsn,), "workspace", dev)
    elif need:
        scratch = new((need,), (1,), torch.uint8, dev)
        wsp, wsn = scratch.data_ptr(), need
    args = (code, xp, DTYPES[x.dtype], ldx, wp, sp, bp, ap, L, N, K, op, DTYPES[od], ldo, wsp, wsn)
    return args, out, scratch


def moe_linear_codec_forward(codec, x, w, s, b=None, bias=None, out=None, out_dtype=None, workspace=None,
                             stream=None) -> torch.Tensor:
    """``x @ W.T + bias`` with 4-bit W (see include/moe_q4.h for the contract).

    ``codec`` is a 4-bit name of :data:`CODECS` or its MOE_Q4_CODEC_* value.
    x bf16 or fp16 [L, K] (contiguous rows; row stride a multiple of 8);
    w int32 (uint32 bits) [N, K/8]; s [N, K/group] bf16 (affine codecs) or
    uint8; b bf16 [N, K/group] (affine codecs only); bias fp32 [N].  Returns
    out [L, N] in ``out_dtype`` (bf16, fp16 or fp32; x's type if not given),
    with no gradient.  ``stream`` (a torch stream or a HIP handle) is as
    ``with torch.cuda.stream(stream)`` around the call.
    """
    if stream is not None and isinstance(x, torch.Tensor):
        with on_stream(stream, x):
            return moe_linear_codec_forward(codec, x, w, s, b, bias, out, out_dtype, workspace)
    args, out, _scratch = _linear_args(codec, x, w, s, b, bias, out, out_dtype, workspace)
    st = call(_q.lib().moe_linear_codec_forward, args, x.device, current_handle(x.device))
    if st:
        raise _q.MoeQ4Error(st, "moe_linear_codec_forward")
    return out


class PreparedLinear:
    """A :func:`moe_linear_codec_forward` whose arguments were checked and
    marshalled once; calling it only crosses the C ABI.  It runs on the stream
    given here (the one current here if none is), with the tensors' device
    current.  The tensors must stay alive and in place for as long as the
    object is used; two of them that may run at the same time need workspaces
    of their own (each makes its own if none is given)."""

    def __init__(self, codec, x, w, s, b=None, bias=None, out=None, out_dtype=None, workspace=None, stream=None):
        if stream is not None and isinstance(x, torch.Tensor):
            with on_stream(stream, x):
                args, out, scratch = _linear_args(codec, x, w, s, b, bias, out, out_dtype, workspace)
                handle = current_handle(x.device)
        else:
            args, out, scratch = _linear_args(codec, x, w, s, b, bias, out, out_dtype, workspace)
            handle = current_handle(x.device)
        self.out = out
        self._keep = (x, w, s, b, bias, workspace, scratch, stream)
        self._args = args
        self._handle = handle
        self._fn = _q.lib().moe_linear_codec_forward
        self._device = x.device

    def __call__(self) -> torch.Tensor:
        st = call(self._fn, self._args, self._device, self._handle)
        if st:
            raise _q.MoeQ4Error(st, "moe_linear_codec_forward")
        return self.out
