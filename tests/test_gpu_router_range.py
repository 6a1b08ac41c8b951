"""The router's selection and the balance loss with sigmoid scores of very
negative logits (needs an MI355X): fp32 holds none of the scores, their
ratios are ordinary numbers.  Bounds as in test_gpu_router; a score below
2^-126, fp32's smallest normal number, may be 0, so a weight that is such a
score times `scale` is off by scale * 2^-126 at most."""

import numpy as np
import pytest
import torch

import quantized_expert_gather_amd as q
from tests import operator_refs as R
from tests import test_gpu_router as T

pytestmark = pytest.mark.gpu
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def low_logits(rows, E, dtype, seed=0):
    z = T.logits(rows, E, F32, seed=seed)
    for i, at in enumerate((-20.0, -80.0, -87.0, -95.0, -104.0, -120.0, -300.0, -700.0)):
        if 2 * i + 1 < rows:
            z[2 * i + 1] += at          # low rows among ordinary ones
    if rows > 17:
        z[17, 1:] = -500.0
        z[17, 0] = float("-inf")
    return z.to(dtype)


def check_topk(z, k, bias, norm, scale=1.5):
    z64 = z.double().numpy()
    ids, w = R.route(z64, k, None if bias is None else bias.double().numpy(), "sigmoid", norm, scale)
    gi, gw = q.moe_router_topk(z.cuda(), k, select_bias=None if bias is None else bias.cuda(), score="sigmoid", renormalize=norm,
                               scale=scale)
    assert np.array_equal(gi.cpu().numpy(), ids)
    assert (np.abs(gw.double().cpu().numpy() - w) <= T.rel(z64) * np.abs(w) + scale * 2.0 ** -126).all()


@pytest.mark.parametrize("E,k", [(8, 2), (64, 6), (256, 8), (300, 40), (1024, 8), (1500, 8)])
def test_topk_of_low_logits(E, k):
    for dtype in (F32, BF16, F16):
        z = low_logits(24, E, dtype, seed=E)
        for bias in (None, 0.1 * torch.randn(E, generator=torch.Generator().manual_seed(4)), torch.zeros(E)):
            for norm in (True, False):
                check_topk(z, k, bias, norm)


@pytest.mark.parametrize("E,k", [(8, 2), (64, 6), (256, 8), (1500, 8)])
def test_topk_backward_of_low_logits(E, k):
    for dtype in (F32, BF16):
        z = low_logits(24, E, dtype, seed=E)
        g = torch.randn(24, k, generator=torch.Generator().manual_seed(2))
        ids, _ = q.moe_router_topk(z.cuda(), k, score="sigmoid")
        ids[1, 0] = -1
        dz = q.moe_router_topk_backward(z.cuda(), ids, g.cuda(), score="sigmoid", scale=1.5)
        z64, i64, g64 = z.double().numpy(), ids.cpu().numpy().astype(np.int64), g.double().numpy()
        ref = R.route_backward(z64, i64, g64, "sigmoid", True, 1.5)
        w = np.abs(R.route_weights(z64, i64, "sigmoid", True, 1.5))
        dot = (w * np.abs(g64)).sum(-1, keepdims=True)
        scale = np.zeros_like(z64)
        for t, j in zip(*np.nonzero(i64 >= 0)):
            scale[t, i64[t, j]] += w[t, j] * (np.abs(g64[t, j]) + dot[t, 0])
        T.close_gradient(dz.double().cpu().numpy(), ref, scale, dtype, T.rel(z64))


@pytest.mark.parametrize("S,rows,E,k", [(1, 24, 8, 2), (2, 24, 64, 6), (1, 24, 256, 8), (3, 300, 300, 4), (1, 24, 1500, 8)])
def test_balance_of_low_logits(S, rows, E, k):
    for dtype in (F32, BF16, F16):
        z = torch.cat([low_logits(rows, E, dtype, seed=E + i) for i in range(S)])
        T.check_balance(S, rows, E, k, dtype, "sigmoid", z=z)
    mask = torch.ones(S * rows, dtype=torch.bool)
    mask[2:7] = False
    T.check_balance(S, rows, E, k, F32, "sigmoid", z=low_logits(S * rows, E, F32), mask=mask)


def test_a_call_on_a_given_stream_carries_its_gradient():
    z = T.logits(40, 24, F32, seed=3).cuda()
    c = torch.randn(40, 4, generator=torch.Generator().manual_seed(1)).cuda()
    grads = []
    for side in (None, torch.cuda.Stream(), torch.cuda.Stream().cuda_stream):
        zi = z.clone().requires_grad_()
        torch.cuda.synchronize()
        ids, w = q.moe_router_topk(zi, 4, stream=side)
        loss, _, _ = q.moe_balance_loss(zi, ids, stream=side)
        assert w.requires_grad and loss.requires_grad and not ids.requires_grad
        torch.cuda.synchronize()
        torch.autograd.backward([w, loss], [c, torch.ones_like(loss)])
        torch.cuda.synchronize()
        grads.append(zi.grad)
    assert torch.equal(grads[0], grads[1]) and torch.equal(grads[0], grads[2]) and grads[0].abs().max() > 0
    with torch.no_grad():
        assert not q.moe_router_topk(zi, 4, stream=torch.cuda.Stream())[1].requires_grad
