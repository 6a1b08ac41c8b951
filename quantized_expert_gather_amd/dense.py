"""Dense products with 4-bit weights (``moe_linear_codec_forward``)."""

from __future__ import annotations

import torch

import quantized_expert_gather_amd as _q

from ._args import DTYPES, array, matrix, on_device, stream_of, used_on

_X = (torch.bfloat16, torch.float16)
_CODES = (torch.int32, getattr(torch, "uint32", torch.int32))


def moe_linear_codec_workspace_bytes(codec, L: int, N: int, K: int) -> int:
    return int(_q.lib().moe_linear_codec_workspace_bytes(_q._codec_id(codec), L, N, K))


def _linear_args(codec, x, w, s, b, bias, out, out_dtype, workspace):
    """Checked arguments of a call up to the stream, and the tensors made here."""
    code = _q._codec_id(codec)
    spec = _q._LINEAR_CODECS.get(code)
    if spec is None:
        raise ValueError(f"codec {codec!r} has no 4-bit dense product")
    gs, affine = spec
    xp, ldx = matrix(x, _X, "x")
    L, K = x.shape
    dev = x.device
    if not isinstance(w, torch.Tensor) or w.dim() != 2:
        raise ValueError("w [N, K/8] expected")
    N = w.shape[0]
    if K % gs:
        raise _q.MoeQ4Error(_q.MOE_Q4_ERR_UNSUPPORTED, "moe_linear_codec_forward")
    scale_type = torch.bfloat16 if affine else torch.uint8
    wp = array(w, _CODES, (N, K // 8), "w", dev)
    sp = array(s, scale_type, (N, K // gs), "s", dev)
    bp = array(b, torch.bfloat16, (N, K // gs), "b", dev) if affine else 0
    ap = 0 if bias is None else array(bias, torch.float32, (N,), "bias", dev)
    made = None
    if out is None:
        od = x.dtype if out_dtype is None else out_dtype
        if od not in DTYPES:
            raise TypeError(f"out_dtype {od} is not one of {tuple(DTYPES)}")
        out = made = torch.empty((L, N), dtype=od, device=dev)
        op, ldo = out.data_ptr(), N
    else:
        op, ldo = matrix(out, DTYPES, "out")
        if out.shape != (L, N) or out.device != dev or out_dtype not in (None, out.dtype):
            raise ValueError(f"out must be [{L}, {N}] on {dev}, of out_dtype")
    need = _q.lib().moe_linear_codec_workspace_bytes(code, L, N, K)
    scratch = None
    wsp, wsn = 0, 0
    if workspace is not None:
        wsn = workspace.numel()
        wsp = array(workspace, torch.uint8, (wsn,), "workspace", dev)
    elif need:
        scratch = torch.empty(need, dtype=torch.uint8, device=dev)
        wsp, wsn = scratch.data_ptr(), need
    args = (code, xp, DTYPES[x.dtype], ldx, wp, sp, bp, ap, L, N, K, op, DTYPES[out.dtype], ldo, wsp, wsn)
    return args, out, made, scratch


def moe_linear_codec_forward(codec, x, w, s, b=None, bias=None, out=None, out_dtype=None, workspace=None,
                             stream=None) -> torch.Tensor:
    """``x @ W.T + bias`` with 4-bit W (see include/moe_q4.h for the contract).

    ``codec`` is a 4-bit name of :data:`CODECS` or its MOE_Q4_CODEC_* value.
    x bf16 or fp16 [L, K] (contiguous rows; row stride a multiple of 8);
    w int32 (uint32 bits) [N, K/8]; s [N, K/group] bf16 (affine codecs) or
    uint8; b bf16 [N, K/group] (affine codecs only); bias fp32 [N].  Returns
    out [L, N] in ``out_dtype`` (bf16, fp16 or fp32; x's type if not given).
    """
    args, out, made, scratch = _linear_args(codec, x, w, s, b, bias, out, out_dtype, workspace)
    handle, side = stream_of(stream, x.device)
    with on_device(x.device):
        _q._check(_q.lib().moe_linear_codec_forward(*args, handle), "moe_linear_codec_forward")
    if side is not None:
        used_on(side, made, scratch)
    return out


class PreparedLinear:
    """A :func:`moe_linear_codec_forward` whose arguments were checked and
    marshalled once; calling it only crosses the C ABI.  It runs on the stream
    given here (the one current here if none is), with the tensors' device
    current.  The tensors must stay alive and in place for as long as the
    object is used; two of them that may run at the same time need workspaces
    of their own (each makes its own if none is given)."""

    def __init__(self, codec, x, w, s, b=None, bias=None, out=None, out_dtype=None, workspace=None, stream=None):
        args, out, _, scratch = _linear_args(codec, x, w, s, b, bias, out, out_dtype, workspace)
        self.out = out
        self._keep = (x, w, s, b, bias, workspace, scratch, stream)
        self._args = (*args, stream_of(stream, x.device)[0])
        self._fn = _q.lib().moe_linear_codec_forward
        self._device = x.device

    def __call__(self) -> torch.Tensor:
        with on_device(self._device):
            st = self._fn(*self._args)
        if st:
            raise _q.MoeQ4Error(st, "moe_linear_codec_forward")
        return self.out
