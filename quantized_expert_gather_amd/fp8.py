"""Products in 8 bits with a scale for each block of 128 (``moe_linear_fp8_forward``)."""

from __future__ import annotations

import torch

import quantized_expert_gather_amd as _q

from ._args import DTYPES, array, call, current_handle, matrix, new, on_stream, plane, scratch, written

F8 = torch.float8_e4m3fn
_F8S = (F8,)


def moe_linear_fp8_workspace_bytes(L: int, N: int, K: int) -> int:
    return int(_q.lib().moe_linear_fp8_workspace_bytes(L, N, K))


def moe_linear_fp8_forward(x, sx, w, sw, bias=None, out=None, out_dtype=None, workspace=None, stream=None) -> torch.Tensor:
    """``(x * sx) @ (w * sw).T + bias`` of E4M3 codes (see include/moe_q4.h for the contract).

    x float8_e4m3fn [L, K] (contiguous rows; row stride a multiple of 16) with
    fp32 scales sx [L, ceil(K / 128)]; w float8_e4m3fn [N, K] with fp32 scales
    sw [ceil(N / 128), ceil(K / 128)]: as :func:`moe_rms_norm_fp8` and
    :func:`moe_quantize_fp8` make them; K a multiple of 16.  bias fp32 [N].
    Returns out [L, N] in ``out_dtype`` (bf16 if not given, fp16 or fp32), with
    no gradient.  ``stream`` (a torch stream or a HIP handle) is as ``with
    torch.cuda.stream(stream)`` around the call.
    """
    if stream is not None and isinstance(x, torch.Tensor):
        with on_stream(stream, x):
            return moe_linear_fp8_forward(x, sx, w, sw, bias, out, out_dtype, workspace)
    xp, ldx, shape = plane(x, _F8S, "x")
    L, K = shape
    dev = x.device
    if not isinstance(w, torch.Tensor) or w.dim() != 2:
        raise ValueError("w [N, K] expected")
    N = w.shape[0]
    G = (K + 127) // 128
    wp = array(w, F8, (N, K), "w", dev)
    sxp = array(sx, torch.float32, (L, G), "sx", dev)
    swp = array(sw, torch.float32, ((N + 127) // 128, G), "sw", dev)
    bp = 0 if bias is None else array(bias, torch.float32, (N,), "bias", dev)
    given_output = out
    if out is None:
        od = torch.bfloat16 if out_dtype is None else out_dtype
        if od not in DTYPES:
            raise TypeError(f"out_dtype {od} is not one of {tuple(DTYPES)}")
        out = new((L, N), (N, 1), od, dev)
        op, ldo = out.data_ptr(), N
    else:
        op, ldo = matrix(out, DTYPES, "out")
        od = out.dtype
        if out.shape != (L, N) or out.device != dev or out_dtype not in (None, od):
            raise ValueError(f"out must be [{L}, {N}] on {dev}, of out_dtype")
    lib = _q.lib()
    wsp = wsn = 0
    if workspace is not None:
        wsp, wsn = scratch(workspace, dev)
    else:
        wsn = lib.moe_linear_fp8_workspace_bytes(L, N, K)
        if wsn:
            workspace = new((wsn,), (1,), torch.uint8, dev)
            wsp = workspace.data_ptr()
    args = (xp, ldx, sxp, wp, swp, bp, L, N, K, op, DTYPES[od], ldo, wsp, wsn)
    st = call(lib.moe_linear_fp8_forward, args, dev, current_handle(dev))
    if st:
        raise _q.MoeQ4Error(st, "moe_linear_fp8_forward")
    written(given_output)
    return out
