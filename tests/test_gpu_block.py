"""The operators beside the expert layer used together with it, as a model's
feed-forward block and its router's training step use them (needs an MI355X)."""

import numpy as np
import pytest
import torch

import oracle
import quantized_expert_gather_amd as q
import synth
from tests import operator_refs as R

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("codec", ["affine4_g64", "mxfp4"])
@pytest.mark.parametrize("L", [1, 5, 48])
def test_feed_forward_block(codec, L):
    """x -> 4-bit router projection -> selection -> experts, plus a dense 4-bit projection of x."""
    E, k, H, I = 16, 4, 512, 256
    print("[case] block", codec, L, flush=True)
    x, _, _, bank = synth.random_problem_q(codec, L, k, E, H, I, seed=3)
    x = (x.float() / H ** 0.5).to(torch.bfloat16)  # N(0,1) weights: logits and gates of order one
    wr = R.linear_weights(codec, E, H, 21)
    wd = R.linear_weights(codec, H, H, 22)
    one = lambda m: [None if t is None else t[0].cuda() for t in m]  # noqa: E731
    xd, bk = x.cuda(), bank.to(torch.device("cuda"))
    z = q.moe_linear_codec_forward(codec, xd, *one(wr), out_dtype=torch.float32)
    ids, w = q.moe_router_topk(z, k, score="sigmoid", scale=1.5)
    y = q.forward_bank_codec(xd, ids, w, bk, out_dtype=torch.float32)
    dense = q.moe_linear_codec_forward(codec, xd, *one(wd), out_dtype=torch.float32)
    got = (y + dense).double().cpu().numpy()
    zr, zb = R.linear_reference(codec, x, *wr, None)
    ri, rw = R.route(z.double().cpu().numpy(), k, None, "sigmoid", True, 1.5)  # the choice follows the logits as computed
    assert (np.abs(z.double().cpu().numpy() - zr) <= zb + 2.0 ** -24 * np.abs(zr)).all()
    assert np.array_equal(ids.cpu().numpy(), ri)
    ref = oracle.forward_pairs_q(codec, x, ri.astype(np.int32), rw.astype(np.float32), bank)
    ref = ref + R.linear_reference(codec, x, *wd, None)[0]
    err = np.linalg.norm(got - ref, axis=1) / np.linalg.norm(ref, axis=1)
    assert err.max() <= 1e-3  # the expert layer's contract


def test_router_training_step_from_the_layer():
    """The router's gradient through the layer's weights: out = sum_j w_j y_j, so dw_j = <dout, y_j>, with y_j from one-route calls."""
    L, E, k, H, I = 6, 8, 2, 256, 128
    x, _, _, bank = synth.random_problem(L, k, E, H, I, seed=5)
    x = (x.float() / 16).to(torch.bfloat16)
    bk, xd = bank.to(torch.device("cuda")), x.cuda()
    g = torch.Generator().manual_seed(2)
    wr = (0.1 * torch.randn(H, E, generator=g)).cuda().requires_grad_()
    dout = torch.randn(L, H, generator=g).cuda()
    z = xd.float() @ wr
    ids, w = q.moe_router_topk(z, k)
    ys = [q.forward_bank(xd, ids[:, j:j + 1].contiguous(), torch.ones(L, 1, device="cuda"), bk, out_dtype=torch.float32)
          for j in range(k)]
    dw = torch.stack([(dout * y).sum(-1) for y in ys], -1)
    loss, counts, _ = q.moe_balance_loss(z, ids, coef=0.1)
    torch.autograd.backward([w, loss], [dw, torch.ones(1, device="cuda")])

    def objective(wm):  # in 64 bits, the choice and the counts held fixed
        zz = x.double().numpy() @ wm
        ww = R.route_weights(zz, ids.cpu().numpy().astype(np.int64), "softmax", True, 1.0)
        p = R.softmax(zz)
        bal = 0.1 * E / (k * L) * (counts[0].cpu().numpy() * p.mean(0)).sum()
        return (ww * dw.double().cpu().numpy()).sum() + bal
    base = wr.detach().double().cpu().numpy()
    grad = wr.grad.double().cpu().numpy()
    rng = np.random.default_rng(0)
    for _ in range(4):
        d = rng.normal(size=base.shape)
        h = 1e-4
        diff = (objective(base + h * d) - objective(base - h * d)) / (2 * h)
        # fp32 products of 256 and 6 terms on the way to the gradient; the difference itself is good to h^2
        assert abs(diff - (grad * d).sum()) <= 1e-4 * np.abs(grad * d).sum()
