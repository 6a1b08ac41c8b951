"""The router's selection and the balance loss on the GPU against 64-bit
references (needs an MI355X).

Bounds.  An exponential of a difference d of fp32 numbers is 2^(d log2 e): off by
at most 2^-24 |d| for the difference's rounding, as much for the product's and
half of it for the constant's, and two steps of its own; sums over a
row take at most 16 + 6 + 16 roundings on a path (a thread's values, the
lanes, the waves) and quotients two more.  With 5 D for a quotient's two
exponentials a probability is off by at most 2^-24 (5 D + 80) of itself, D the
largest difference; a gradient multiplies three such numbers at most."""

import numpy as np
import pytest
import torch

import quantized_expert_gather_amd as q
from tests import operator_refs as R

pytestmark = pytest.mark.gpu
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def logits(T, E, dtype, seed=0, spread=2.0):
    g = torch.Generator().manual_seed(seed)
    return (spread * torch.randn(T, E, generator=g)).to(dtype)


def rel(z):
    f = z[np.isfinite(z)]
    return 2.0 ** -24 * (5 * (f.max() - f.min() if f.size else 0) + 80)


def check_topk(z, k, bias, score, norm, scale=1.5):
    print("[case] topk", tuple(z.shape), z.dtype, k, bias is not None, score, norm, flush=True)
    z64 = z.double().numpy()
    ids, w = R.route(z64, k, None if bias is None else bias.double().numpy(), score, norm, scale)
    gi, gw = q.moe_router_topk(z.cuda(), k, select_bias=None if bias is None else bias.cuda(), score=score, renormalize=norm,
                               scale=scale)
    assert gi.dtype == torch.int32 and gw.dtype == F32
    gi, gw = gi.cpu().numpy(), gw.double().cpu().numpy()
    assert np.array_equal(gi, ids), np.argwhere(gi != ids)[:4]
    assert (np.abs(gw - w) <= rel(z64) * np.abs(w) + 2.0 ** -126).all()
    return gi


@pytest.mark.parametrize("E,k", [(1, 1), (2, 1), (8, 2), (8, 8), (60, 4), (64, 6), (65, 6), (128, 64), (250, 8), (256, 8),
                                 (288, 8), (511, 16), (1000, 33), (1024, 8), (1025, 8), (4096, 10), (16384, 64)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("norm", [True, False])
def test_topk_sizes(E, k, score, norm):
    for dtype in (F32, BF16, F16):
        z = logits(7, E, dtype, seed=E + k)
        check_topk(z, k, None, score, norm)
        check_topk(z, k, 0.3 * torch.randn(E, generator=torch.Generator().manual_seed(5)), score, norm)


@pytest.mark.parametrize("T", [1, 2, 5, 1023])
def test_topk_token_counts(T):
    check_topk(logits(T, 96, F32), 5, None, "softmax", True)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_topk_ties_go_to_the_lower_expert(score):
    z = torch.randint(-2, 3, (200, 300), generator=torch.Generator().manual_seed(1)).float()
    z[0] = 0.0
    z[1, ::2] = -0.0
    z[1, 1::2] = 0.0
    check_topk(z, 40, None, score, True)
    check_topk(z, 40, torch.zeros(300), score, True)
    check_topk(z.to(BF16), 40, torch.randint(0, 2, (300,), generator=torch.Generator().manual_seed(2)).float(), score, False)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_topk_scores_that_fp32_cannot_tell_apart(score):
    # logits a few steps apart under a bias: fp32 scores collide, 64-bit ones do not
    g = torch.Generator().manual_seed(3)
    z = 0.25 + torch.randint(0, 40, (300, 256), generator=g).float() * 2.0 ** -25
    z = z[:, torch.randperm(256, generator=g)]
    b = torch.randint(0, 3, (256,), generator=g).float() * 2.0 ** -24 + 0.5
    check_topk(z, 8, b, score, True)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,k", [(64, 4), (64, 16), (256, 7), (256, 8), (288, 31), (1024, 64), (1500, 8), (9, 8), (8, 8)])
def test_topk_close_pairs_at_every_place(score, E, k):
    # biases that bring experts' scores within a few steps of one another, in
    # pairs and in runs, at places that differ from row to row
    g = torch.Generator().manual_seed(E + k)
    T = 96
    z = torch.randn(T, E, generator=g)
    n = min(E, 48)
    z[:, :n] = z[0, :n]                        # the same logits in every row
    b = 0.05 * torch.randn(E, generator=g)
    total = 1.0 if score == "sigmoid" else None
    p = torch.sigmoid(z[0].double()) if total else torch.softmax(z[0].double(), -1)
    for i in range(0, n - 3, 4):               # experts i, i + 1 close; in every third group i + 2 and i + 3 too
        for j in range(1, 4 if i % 12 == 0 else 2):
            b[i + j] = (p[i] + b[i].double() - p[i + j]).float()
    if score == "softmax":
        z = z[:1].repeat(T, 1)                 # close scores need the same sum: rows differ by a shift
        z = z + torch.randint(-3, 4, (T, 1), generator=g).float()
    check_topk(z, k, b, score, True)
    check_topk(z, k, b, score, False)


def test_topk_masked_experts_and_nan():
    inf = float("inf")
    z = logits(9, 130, F32, seed=4)
    z[0, :] = -inf
    z[1, 3:] = -inf          # fewer experts left than routes
    z[2, 10] = float("nan")
    z[3, :] = float("nan")
    z[4, ::2] = torch.finfo(F32).min
    z[5, 1:] = torch.finfo(F32).min
    z[6, 7] = torch.finfo(F32).max / 2
    z64 = z.double().numpy()
    for score in ("softmax", "sigmoid"):
        for norm in (True, False):
            ids, w = R.route(z64, 6, None, score, norm, 1.0)
            gi, gw = q.moe_router_topk(z.cuda(), 6, score=score, renormalize=norm)
            gi, gw = gi.cpu().numpy(), gw.double().cpu().numpy()
            assert np.array_equal(gi, ids)
            ok = np.isfinite(w) & (np.arange(9) != 3)[:, None]
            if norm or score == "sigmoid":
                ok[2] = True
            else:
                assert np.isnan(gw[2]).all()
                ok[2] = False
            lim = 2.0 ** -24 * 200 * np.abs(w) + 2.0 ** -126
            assert (np.abs(gw - w)[ok] <= lim[ok]).all()
            assert (gw[0] == 0).all() and (gw[1, 3:] == 0).all()
    # a bias of -inf takes experts out of the choice
    b = torch.zeros(130)
    b[::2] = -inf
    check_topk(logits(20, 130, F32, seed=8), 9, b, "sigmoid", True)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E", [40, 130, 1500])
@pytest.mark.parametrize("T", [9, 7000])
def test_topk_choice_of_bad_rows_with_a_bias(score, E, T):
    inf = float("inf")
    z = logits(T, E, F32, seed=4)
    z[0, 10] = float("nan")
    z[1, :] = -inf
    z[2, :] = float("nan")
    z[3, 5] = inf
    z[4, 3:] = -inf
    z[5, :] = 0.25
    b = 0.1 * torch.randn(E, generator=torch.Generator().manual_seed(E))
    b[7] = -inf
    for bias in (b, torch.zeros(E)):
        ids, _ = R.route(z.double().numpy(), 6, bias.double().numpy(), score, True, 1.0)
        gi, gw = q.moe_router_topk(z.cuda(), 6, select_bias=bias.cuda(), score=score)
        assert np.array_equal(gi.cpu().numpy(), ids)
        assert torch.isfinite(gw[6:]).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("E", [64, 100, 1500])
def test_topk_strided_logits(dtype, E):
    z = logits(6, E, dtype)
    wide = torch.full((6, E + 7), 50.0, dtype=dtype, device="cuda")
    wide[:, 3:3 + E] = z.cuda()
    i0, w0 = q.moe_router_topk(z.cuda(), 4)
    i1, w1 = q.moe_router_topk(wide[:, 3:3 + E], 4)
    assert torch.equal(i0, i1) and torch.equal(w0, w1)
    d0 = q.moe_router_topk_backward(z.cuda(), i0, w0)
    room = torch.full((8, E + 5), 9.0, dtype=dtype, device="cuda")
    q.moe_router_topk_backward(wide[:, 3:3 + E], i0, w0, dlogits=room[1:7, 2:2 + E])
    assert torch.equal(room[1:7, 2:2 + E], d0)
    room[1:7, 2:2 + E] = 9.0
    assert (room == 9.0).all()


def test_topk_into_given_tensors():
    z = logits(5, 40, F32).cuda()
    ids, w = torch.empty(5, 3, dtype=torch.int32, device="cuda"), torch.empty(5, 3, device="cuda")
    a, b = q.moe_router_topk(z, 3, topk_ids=ids, topk_weights=w)
    assert a is ids and b is w
    c, d = q.moe_router_topk(z, 3)
    assert torch.equal(a, c) and torch.equal(b, d)


def close_gradient(got, ref, scale, dtype, tol):
    lim = 3 * tol * scale + R.HALF_STEP[dtype] * (np.abs(ref) + 3 * tol * scale) + R.HALF_TINY[dtype]
    bad = ~(np.abs(got - ref) <= lim)
    assert not bad.any(), (int(bad.sum()), float(np.abs(got - ref)[bad].max()))


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (3, 8, 2), (5, 60, 6), (70, 64, 8), (33, 256, 8), (9, 288, 6), (4, 1024, 64),
                                   (3, 1030, 8), (2, 16384, 16)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("norm", [True, False])
def test_topk_backward(T, E, k, score, norm):
    for dtype in (F32, BF16, F16):
        print("[case] topk backward", T, E, k, score, norm, dtype, flush=True)
        z = logits(T, E, dtype, seed=T)
        g = torch.randn(T, k, generator=torch.Generator().manual_seed(2))
        ids, _ = q.moe_router_topk(z.cuda(), k, score=score)
        if T > 2 and k > 1:
            ids[1, 1] = ids[1, 0]    # the same expert twice
            ids[2, 0] = -1           # routes left out
            ids[2, 1] = E
        dz = q.moe_router_topk_backward(z.cuda(), ids, g.cuda(), score=score, renormalize=norm, scale=1.5)
        assert dz.dtype == dtype
        z64, i64, g64 = z.double().numpy(), ids.cpu().numpy().astype(np.int64), g.double().numpy()
        i64 = np.where((i64 < 0) | (i64 >= E), -1, i64)
        ref = R.route_backward(z64, i64, g64, score, norm, 1.5)
        w = np.abs(R.route_weights(z64, i64, score, norm, 1.5))
        dot = (w * np.abs(g64)).sum(-1, keepdims=True)
        scale = np.zeros_like(z64)
        if score == "softmax" and not norm:
            scale += R.softmax(z64) * dot
        for t, j in zip(*np.nonzero(i64 >= 0)):
            scale[t, i64[t, j]] += w[t, j] * (np.abs(g64[t, j]) + dot[t, 0])
        close_gradient(dz.double().cpu().numpy(), ref, scale, dtype, rel(z64))


def test_topk_backward_of_masked_rows_is_zero():
    z = torch.full((3, 20), float("-inf"))
    z[1, 4] = 1.0
    for score in ("softmax", "sigmoid"):
        for norm in (True, False):
            ids, _ = q.moe_router_topk(z.cuda(), 3, score=score, renormalize=norm)
            dz = q.moe_router_topk_backward(z.cuda(), ids, torch.ones(3, 3).cuda(), score=score, renormalize=norm)
            assert (dz[[0, 2]] == 0).all() and torch.isfinite(dz).all()


# ---- balance loss ----

def routes(T, E, k, seed=0):
    g = torch.Generator().manual_seed(seed)
    return torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]).to(torch.int32) if T else \
        torch.empty(0, k, dtype=torch.int32)


def check_balance(S, T, E, k, dtype, score, mask=None, seed=0, coef=0.7, ids=None, z=None):
    print("[case] balance", S, T, E, k, dtype, score, mask is not None, flush=True)
    z = logits(S * T, E, dtype, seed=seed) if z is None else z
    ids = routes(S * T, E, k, seed) if ids is None else ids
    mk = None if mask is None else mask.numpy()
    z64 = z.double().numpy()
    loss, counts, tokens = R.balance(z64, ids.numpy(), coef, score, S, mk)
    md = None if mask is None else mask.cuda()
    gl, gc, gt = q.moe_balance_loss(z.cuda(), ids.cuda(), coef=coef, score=score, seqs=S, token_mask=md)
    assert gl.shape == (S,) and gc.shape == (S, E) and gt.shape == (S,)
    assert np.array_equal(gc.cpu().numpy(), counts) and np.array_equal(gt.cpu().numpy(), tokens)
    # every addend of the loss is positive: a relative bound, with the sums over tokens and workgroups
    tol = rel(z64) + 2.0 ** -24 * (400 + T / 256)
    assert (np.abs(gl.double().cpu().numpy() - loss) <= tol * loss + 2.0 ** -126).all()
    g = torch.randn(S, generator=torch.Generator().manual_seed(9)) * (1024 if dtype == F16 else 1)
    dz = q.moe_balance_loss_backward(z.cuda(), gc, gt, g.cuda(), k, coef=coef, score=score, token_mask=md)
    ref = R.balance_backward(z64, counts, tokens, g.double().numpy(), k, coef, score, mk)
    p = R.softmax(z64) if score == "softmax" else R.sigmoid(z64) / R.sigmoid(z64).sum(-1, keepdims=True)
    n = np.maximum(tokens, 1).astype(float)
    a = np.abs(np.repeat(g.double().numpy()[:, None] * coef * E * counts / (k * n[:, None] ** 2), T, 0))
    scale = p * (a + (a * p).sum(-1, keepdims=True))
    close_gradient(dz.double().cpu().numpy(), ref, scale, dtype, rel(z64))
    if mask is not None:
        assert (dz.cpu()[mask == 0] == 0).all()


@pytest.mark.parametrize("S,T,E,k", [(1, 1, 1, 1), (1, 1, 8, 2), (1, 3, 60, 4), (1, 257, 64, 6), (3, 50, 100, 8),
                                     (2, 300, 288, 8), (1, 1000, 256, 8), (5, 17, 512, 3), (1, 40, 1024, 2), (2, 9, 1500, 8),
                                     (1, 3, 16384, 8), (300, 2, 16, 2)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_balance_sizes(S, T, E, k, score):
    for dtype in (F32, BF16, F16):
        check_balance(S, T, E, k, dtype, score)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E", [64, 90, 1100])
def test_balance_masks(score, E):
    S, T = 4, 45
    lens = torch.tensor([45, 0, 1, 20])
    mask = (torch.arange(T) < lens[:, None]).reshape(-1)
    check_balance(S, T, E, 4, F32, score, mask=mask)
    check_balance(S, T, E, 4, BF16, score, mask=mask.to(torch.uint8))
    holes = torch.rand(S * T, generator=torch.Generator().manual_seed(1)) < 0.5
    check_balance(S, T, E, 4, F32, score, mask=holes)


def test_balance_masked_tokens_may_hold_anything():
    S, T, E, k = 2, 30, 70, 3
    z, ids = logits(S * T, E, F32), routes(S * T, E, k)
    mask = torch.ones(S * T, dtype=torch.bool)
    mask[5:9] = False
    mask[40:] = False
    z2, ids2 = z.clone(), ids.clone()
    z2[~mask] = float("nan")
    ids2[~mask] = 1 << 30
    a = q.moe_balance_loss(z.cuda(), ids.cuda(), seqs=S, token_mask=mask.cuda())
    b = q.moe_balance_loss(z2.cuda(), ids2.cuda(), seqs=S, token_mask=mask.cuda())
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    g = torch.ones(S).cuda()
    da = q.moe_balance_loss_backward(z.cuda(), a[1], a[2], g, k, token_mask=mask.cuda())
    db = q.moe_balance_loss_backward(z2.cuda(), a[1], a[2], g, k, token_mask=mask.cuda())
    assert torch.equal(da, db)


def test_balance_masked_experts_and_routes():
    z = logits(50, 40, F32)
    z[:, 7] = float("-inf")
    z[3] = float("-inf")
    ids = routes(50, 40, 4)
    ids[0, 0] = -1
    ids[1, 1] = 40
    ids[2, 2] = ids[2, 1]
    check_balance(1, 50, 40, 4, F32, "softmax", ids=ids, z=z)


def test_balance_no_tokens():
    loss, counts, tokens = q.moe_balance_loss(torch.empty(0, 8, device="cuda"), torch.empty(0, 2, dtype=torch.int32, device="cuda"),
                                              seqs=1)
    assert loss.tolist() == [0.0] and (counts == 0).all() and tokens.tolist() == [0]


def test_balance_runs_are_equal():
    z, ids = logits(3000, 256, BF16).cuda(), routes(3000, 256, 8).cuda()
    a = q.moe_balance_loss(z, ids)
    for _ in range(3):
        b = q.moe_balance_loss(z, ids)
        assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_many_logits():
    # a row offset past 2^32 bytes; one row of every run is checked
    T, E = 1_050_000, 1024
    z = torch.zeros(T, E, device="cuda")
    z[-1, 77] = 3.0
    z[-1, 5] = 2.0
    ids, w = q.moe_router_topk(z, 2)
    assert ids[-1].tolist() == [77, 5] and ids[-2].tolist() == [0, 1]
    dz = q.moe_router_topk_backward(z, ids, w, renormalize=False)
    assert dz[-1, 77] != 0 and torch.isfinite(dz[-1]).all()
    loss, counts, tokens = q.moe_balance_loss(z, ids)
    assert counts[0, 77] == 1 and counts[0, 0] == T - 1 and tokens[0] == T
    d = q.moe_balance_loss_backward(z, counts, tokens, torch.ones(1, device="cuda"), 2)
    assert torch.isfinite(d[-1]).all() and (d[-1, 0] > 0)


# ---- gradients through torch, streams, graphs ----

@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_autograd(score):
    T, H, E, k = 64, 32, 20, 4
    g = torch.Generator().manual_seed(6)
    x, wr, c = torch.randn(T, H, generator=g), 0.3 * torch.randn(H, E, generator=g), torch.randn(T, k, generator=g)
    mask = torch.rand(T, generator=g) < 0.8
    wd = wr.clone().cuda().requires_grad_()
    z = x.cuda() @ wd
    ids, w = q.moe_router_topk(z, k, score=score, scale=2.0)
    loss, counts, tokens = q.moe_balance_loss(z, ids, coef=0.5, score=score, seqs=2, token_mask=mask.cuda())
    assert not ids.requires_grad and not counts.requires_grad
    ((w * c.cuda()).sum() + loss.mean()).backward()
    w64 = wr.double().requires_grad_()
    z64 = x.double() @ w64
    p = torch.softmax(z64, -1) if score == "softmax" else torch.sigmoid(z64)
    ch = p.gather(-1, ids.cpu().long())
    wt = 2.0 * ch / ch.sum(-1, keepdim=True)
    pn = p / p.sum(-1, keepdim=True)
    tot = (pn * mask[:, None]).view(2, T // 2, E).sum(1)
    n = mask.view(2, -1).sum(-1).double()
    bl = 0.5 * E / (k * n * n) * (counts.cpu().double() * tot).sum(-1)
    ((wt * c).sum() + bl.mean()).backward()
    # the logits come from an fp32 product of 32 terms; the weight gradient adds 64 tokens
    assert (wd.grad.cpu().double() - w64.grad).abs().max() <= 2e-5 * w64.grad.abs().max()


def test_backward_of_a_captured_step_is_refused(monkeypatch):
    z = logits(8, 16, F32).cuda().requires_grad_()
    ids, w = q.moe_router_topk(z, 2)
    loss, _, _ = q.moe_balance_loss(z, ids)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
    with pytest.raises(RuntimeError, match="moe_router_topk_backward"):
        w.sum().backward()
    with pytest.raises(RuntimeError, match="moe_balance_loss_backward"):
        loss.sum().backward()
    assert z.grad is None


def test_autograd_does_not_touch_plain_calls():
    z = logits(4, 8, F32).cuda().requires_grad_()
    with torch.no_grad():
        assert not q.moe_router_topk(z, 2)[1].requires_grad
    assert not q.moe_router_topk(z.detach(), 2)[1].requires_grad


def test_streams_and_graphs():
    T, E, k, S = 128, 96, 6, 4
    z, g, dl = logits(T, E, BF16).cuda(), torch.randn(T, k).cuda(), torch.ones(S).cuda()
    bias = torch.randn(E).cuda() * 0.1

    def step(stream=None, ws=None):
        ids, w = q.moe_router_topk(z, k, select_bias=bias, score="sigmoid", stream=stream)
        dz = q.moe_router_topk_backward(z, ids, g, score="sigmoid", stream=stream)
        loss, counts, tokens = q.moe_balance_loss(z, ids, score="sigmoid", seqs=S, stream=stream, workspace=ws)
        db = q.moe_balance_loss_backward(z, counts, tokens, dl, k, score="sigmoid", stream=stream)
        return ids, w, dz, loss, counts, tokens, db
    ref = [t.clone() for t in step()]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    other = step(side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(ref, other))
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        out = step()
    for rep in range(3):
        for t in out:
            t.zero_()
        gr.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(ref, out)), rep
        again = step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(ref, again))
