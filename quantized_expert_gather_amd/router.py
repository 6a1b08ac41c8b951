"""The router's selection and the balance loss, with their gradients
(``moe_router_topk``, ``moe_balance_loss`` and their ``_backward``)."""

from __future__ import annotations

from typing import Tuple

import torch

import quantized_expert_gather_amd as _q

from ._args import DTYPES, array, call, current_handle, matrix, new, on_stream


def _score(score) -> int:
    code = _q.SCORES.get(score)
    if code is not None:
        return code
    if isinstance(score, str):
        raise ValueError(f"unknown score {score!r}, expected one of {tuple(_q.SCORES)}")
    return int(score)


def _not_captured(name):
    # torch's accumulation of a captured gradient into a leaf that an eager graph still holds ends the process
    if torch.cuda.is_current_stream_capturing():
        raise RuntimeError(f"backward() of a graph-captured step: call {name} itself")


def _gradient(logits, dlogits):
    """(tensor, pointer, row stride) of a gradient like `logits`."""
    if dlogits is None:
        E = logits.shape[1]
        d = new(logits.shape, (E, 1), logits.dtype, logits.device)
        return d, d.data_ptr(), E
    p, ldd = matrix(dlogits, (logits.dtype,), "dlogits")
    if dlogits.shape != logits.shape or dlogits.device != logits.device:
        raise ValueError("dlogits must have the shape and device of logits")
    return dlogits, p, ldd


def _topk(logits, k, select_bias, score, renormalize, scale, topk_ids=None, topk_weights=None):
    zp, ld = matrix(logits, DTYPES, "logits")
    T, E = logits.shape
    dev = logits.device
    k = int(k)
    if not 1 <= k <= E:
        raise _q.MoeQ4Error(_q.MOE_Q4_ERR_SHAPE, "moe_router_topk")
    bp = 0 if select_bias is None else array(select_bias, torch.float32, (E,), "select_bias", dev)
    if topk_ids is None:
        topk_ids = new((T, k), (k, 1), torch.int32, dev)
        ip = topk_ids.data_ptr()
    else:
        ip = array(topk_ids, torch.int32, (T, k), "topk_ids", dev)
    if topk_weights is None:
        topk_weights = new((T, k), (k, 1), torch.float32, dev)
        wp = topk_weights.data_ptr()
    else:
        wp = array(topk_weights, torch.float32, (T, k), "topk_weights", dev)
    args = (zp, DTYPES[logits.dtype], ld, bp, T, k, E, _score(score), 1 if renormalize else 0, scale, ip, wp)
    st = call(_q.lib().moe_router_topk, args, dev, current_handle(dev))
    if st:
        raise _q.MoeQ4Error(st, "moe_router_topk")
    return topk_ids, topk_weights


class _TopkFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, k, select_bias, score, renormalize, scale):
        ids, w = _topk(logits, k, select_bias, score, renormalize, scale)
        ctx.mark_non_differentiable(ids)
        ctx.save_for_backward(logits, ids)
        ctx.how = (score, renormalize, scale)
        return ids, w

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, _dids, dweights):
        _not_captured("moe_router_topk_backward")
        logits, ids = ctx.saved_tensors
        score, renormalize, scale = ctx.how
        dz = moe_router_topk_backward(logits, ids, dweights.float().contiguous(), score=score, renormalize=renormalize,
                                      scale=scale)
        return dz, None, None, None, None, None


def moe_router_topk(logits, k: int, select_bias=None, score="softmax", renormalize: bool = True, scale: float = 1.0,
                    topk_ids=None, topk_weights=None, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """The k experts of each token and their weights (see include/moe_q4.h).

    logits [T, E] bf16, fp16 or fp32 with contiguous rows; select_bias fp32
    [E], added to the scores for the choice only.  Returns (topk_ids int32 [T,
    k], topk_weights fp32 [T, k]) as :func:`moe_swiglu_q4_forward` takes them.

    The weights carry a gradient to logits where logits requires one; output
    tensors, which cannot, are refused then.  A step recorded into a graph
    calls :func:`moe_router_topk_backward` itself (backward() refuses there).
    ``stream`` (a torch stream or a HIP handle) is as ``with
    torch.cuda.stream(stream)`` around the call.
    """
    if stream is not None and isinstance(logits, torch.Tensor):
        with on_stream(stream, logits):
            return moe_router_topk(logits, k, select_bias, score, renormalize, scale, topk_ids, topk_weights)
    if isinstance(logits, torch.Tensor) and logits.requires_grad and torch.is_grad_enabled():
        if topk_ids is not None or topk_weights is not None:
            raise RuntimeError("moe_router_topk: given output tensors carry no gradient, but logits requires one")
        return _TopkFunction.apply(logits, k, select_bias, score, renormalize, scale)
    return _topk(logits, k, select_bias, score, renormalize, scale, topk_ids, topk_weights)


def moe_router_topk_backward(logits, topk_ids, dweights, score="softmax", renormalize: bool = True, scale: float = 1.0,
                             dlogits=None, stream=None) -> torch.Tensor:
    """Gradient of :func:`moe_router_topk`'s weights with respect to logits, the
    choice held fixed: dweights fp32 [T, k] -> dlogits [T, E] in logits' type."""
    if stream is not None and isinstance(logits, torch.Tensor):
        with on_stream(stream, logits):
            return moe_router_topk_backward(logits, topk_ids, dweights, score, renormalize, scale, dlogits)
    zp, ld = matrix(logits, DTYPES, "logits")
    T, E = logits.shape
    dev = logits.device
    if not isinstance(topk_ids, torch.Tensor) or topk_ids.dim() != 2:
        raise ValueError("topk_ids [T, k] expected")
    k = topk_ids.shape[1]
    ip = array(topk_ids, torch.int32, (T, k), "topk_ids", dev)
    gp = array(dweights, torch.float32, (T, k), "dweights", dev)
    d, dp, ldd = _gradient(logits, dlogits)
    args = (zp, DTYPES[logits.dtype], ld, ip, gp, T, k, E, _score(score), 1 if renormalize else 0, scale, dp, ldd)
    st = call(_q.lib().moe_router_topk_backward, args, dev, current_handle(dev))
    if st:
        raise _q.MoeQ4Error(st, "moe_router_topk_backward")
    return d


def moe_balance_loss_workspace_bytes(S: int, T: int, E: int) -> int:
    return int(_q.lib().moe_balance_loss_workspace_bytes(S, T, E))


def _tokens_of(logits, seqs):
    seqs = int(seqs)
    if seqs < 1 or logits.shape[0] % seqs:
        raise ValueError(f"{logits.shape[0]} tokens are not {seqs} sequences of equal length")
    return seqs, logits.shape[0] // seqs


def _mask_ptr(token_mask, rows, device):
    if token_mask is None:
        return 0
    if isinstance(token_mask, torch.Tensor):
        token_mask = token_mask.reshape(-1) if token_mask.is_contiguous() else token_mask
    return array(token_mask, (torch.bool, torch.uint8), (rows,), "token_mask", device)


def _balance(logits, topk_ids, coef, score, seqs, token_mask, workspace):
    zp, ld = matrix(logits, DTYPES, "logits")
    rows, E = logits.shape
    dev = logits.device
    S, T = _tokens_of(logits, seqs)
    if not isinstance(topk_ids, torch.Tensor) or topk_ids.dim() != 2:
        raise ValueError("topk_ids [tokens, k] expected")
    k = topk_ids.shape[1]
    ip = array(topk_ids, torch.int32, (rows, k), "topk_ids", dev)
    mp = _mask_ptr(token_mask, rows, dev)
    lib = _q.lib()
    loss, tokens = new((S,), (1,), torch.float32, dev), new((S,), (1,), torch.int32, dev)
    counts = new((S, E), (E, 1), torch.int32, dev)
    scratch = None
    if workspace is None:
        wsn = lib.moe_balance_loss_workspace_bytes(S, T, E)
        scratch = new((wsn,), (1,), torch.uint8, dev)
        wsp = scratch.data_ptr()
    else:
        wsn = workspace.numel()
        wsp = array(workspace, torch.uint8, (wsn,), "workspace", dev)
    args = (zp, DTYPES[logits.dtype], ld, ip, mp, S, T, k, E, _score(score), coef, loss.data_ptr(), counts.data_ptr(),
            tokens.data_ptr(), wsp, wsn)
    st = call(lib.moe_balance_loss, args, dev, current_handle(dev))
    if st:
        raise _q.MoeQ4Error(st, "moe_balance_loss")
    return loss, counts, tokens


class _BalanceFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, topk_ids, coef, score, seqs, token_mask, workspace):
        loss, counts, tokens = _balance(logits, topk_ids, coef, score, seqs, token_mask, workspace)
        ctx.mark_non_differentiable(counts, tokens)
        ctx.save_for_backward(logits, counts, tokens, token_mask)
        ctx.how = (topk_ids.shape[1], coef, score)
        return loss, counts, tokens

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dloss, _dcounts, _dtokens):
        _not_captured("moe_balance_loss_backward")
        logits, counts, tokens, token_mask = ctx.saved_tensors
        k, coef, score = ctx.how
        dz = moe_balance_loss_backward(logits, counts, tokens, dloss.float().contiguous(), k, coef=coef, score=score,
                                       token_mask=token_mask)
        return dz, None, None, None, None, None, None


def moe_balance_loss(logits, topk_ids, coef: float = 1.0, score="softmax", seqs: int = 1, token_mask=None,
                     workspace=None, stream=None) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """Balance loss and route counts of ``seqs`` sequences of equal length (see
    include/moe_q4.h): logits [seqs * T, E] bf16, fp16 or fp32 with contiguous
    rows, topk_ids int32 [seqs * T, k], token_mask bool or uint8 [seqs * T] (0
    leaves a token out).

    Returns (loss fp32 [seqs], counts int32 [seqs, E], tokens int32 [seqs]).
    The loss carries a gradient to logits where logits requires one; a step
    recorded into a graph calls :func:`moe_balance_loss_backward` itself
    (backward() refuses there).  ``stream`` is as :func:`moe_router_topk`'s.
    """
    if stream is not None and isinstance(logits, torch.Tensor):
        with on_stream(stream, logits):
            return moe_balance_loss(logits, topk_ids, coef, score, seqs, token_mask, workspace)
    if isinstance(logits, torch.Tensor) and logits.requires_grad and torch.is_grad_enabled():
        return _BalanceFunction.apply(logits, topk_ids, coef, score, seqs, token_mask, workspace)
    return _balance(logits, topk_ids, coef, score, seqs, token_mask, workspace)


def moe_balance_loss_backward(logits, counts, tokens, dloss, k: int, coef: float = 1.0, score="softmax",
                              token_mask=None, dlogits=None, stream=None) -> torch.Tensor:
    """Gradient of :func:`moe_balance_loss`, the counts held fixed: dloss fp32
    [seqs] and the forward's counts and tokens -> dlogits in logits' type."""
    if stream is not None and isinstance(logits, torch.Tensor):
        with on_stream(stream, logits):
            return moe_balance_loss_backward(logits, counts, tokens, dloss, k, coef, score, token_mask, dlogits)
    zp, ld = matrix(logits, DTYPES, "logits")
    rows, E = logits.shape
    dev = logits.device
    if not isinstance(counts, torch.Tensor) or counts.dim() != 2:
        raise ValueError("counts [seqs, E] expected")
    S, T = _tokens_of(logits, counts.shape[0])
    cp = array(counts, torch.int32, (S, E), "counts", dev)
    np_ = array(tokens, torch.int32, (S,), "tokens", dev)
    gp = array(dloss, torch.float32, (S,), "dloss", dev)
    mp = _mask_ptr(token_mask, rows, dev)
    d, dp, ldd = _gradient(logits, dlogits)
    args = (zp, DTYPES[logits.dtype], ld, mp, cp, np_, gp, S, T, int(k), E, _score(score), coef, dp, ldd)
    st = call(_q.lib().moe_balance_loss_backward, args, dev, current_handle(dev))
    if st:
        raise _q.MoeQ4Error(st, "moe_balance_loss_backward")
    return d
