"""Host-side checks of the operators beside the expert layer (no GPU): every
refusal returns before any GPU work, so the pointers here are fake."""

import numpy as np
import pytest
import torch

import quantized_expert_gather_amd as q
from tests import operator_refs as R

BASE, STRIDE = 1 << 40, 1 << 36


def fake(i, off=0):
    return BASE + i * STRIDE + off


def linear(codec=0, x=None, xd=0, ldx=None, w=None, s=None, b=None, bias=0, L=2, N=24, K=128, out=None, od=0, ldo=None,
           ws=None, wn=1 << 34):
    p = lambda v, i: fake(i) if v is None else v  # noqa: E731
    return q.lib().moe_linear_codec_forward(codec, p(x, 0), xd, K if ldx is None else ldx, p(w, 1), p(s, 2), p(b, 3), bias,
                                            L, N, K, p(out, 5), od, N if ldo is None else ldo, p(ws, 6), wn, None)


@pytest.mark.parametrize("kw,status", [
    (dict(L=-1), q.MOE_Q4_ERR_SHAPE),
    (dict(N=0), q.MOE_Q4_ERR_SHAPE),
    (dict(K=0), q.MOE_Q4_ERR_SHAPE),
    (dict(ldx=127), q.MOE_Q4_ERR_SHAPE),
    (dict(ldo=23), q.MOE_Q4_ERR_SHAPE),
    (dict(K=96), q.MOE_Q4_ERR_UNSUPPORTED),
    (dict(codec=1, K=48), q.MOE_Q4_ERR_UNSUPPORTED),
    (dict(codec=3, K=16), q.MOE_Q4_ERR_UNSUPPORTED),
    (dict(codec=4), q.MOE_Q4_ERR_UNSUPPORTED),  # 8-bit codecs
    (dict(codec=5), q.MOE_Q4_ERR_UNSUPPORTED),
    (dict(codec=9), q.MOE_Q4_ERR_UNSUPPORTED),
    (dict(xd=1), q.MOE_Q4_ERR_UNSUPPORTED),
    (dict(od=3), q.MOE_Q4_ERR_UNSUPPORTED),
    (dict(L=q.MOE_Q4_LINEAR_MAX_L + 1), q.MOE_Q4_ERR_UNSUPPORTED),
    (dict(K=q.MOE_Q4_LINEAR_MAX_K + 64), q.MOE_Q4_ERR_UNSUPPORTED),
    (dict(ldx=q.MOE_Q4_LINEAR_MAX_LDX + 8), q.MOE_Q4_ERR_UNSUPPORTED),
    (dict(N=q.MOE_Q4_LINEAR_MAX_N + 1), q.MOE_Q4_ERR_UNSUPPORTED),
    (dict(L=40, K=64, ws=fake(0)), q.MOE_Q4_ERR_ALIAS),
    (dict(L=40, K=64, ws=fake(2)), q.MOE_Q4_ERR_ALIAS),
    (dict(L=40, K=64, ws=fake(4, 256), bias=fake(4, 512)), q.MOE_Q4_ERR_ALIAS),
    (dict(x=0), q.MOE_Q4_ERR_NULL),
    (dict(w=0), q.MOE_Q4_ERR_NULL),
    (dict(s=0), q.MOE_Q4_ERR_NULL),
    (dict(b=0), q.MOE_Q4_ERR_NULL),
    (dict(out=0), q.MOE_Q4_ERR_NULL),
    (dict(x=fake(0, 8)), q.MOE_Q4_ERR_ALIGN),
    (dict(ldx=132), q.MOE_Q4_ERR_ALIGN),
    (dict(w=fake(1, 8)), q.MOE_Q4_ERR_ALIGN),
    (dict(s=fake(2, 1)), q.MOE_Q4_ERR_ALIGN),
    (dict(b=fake(3, 1)), q.MOE_Q4_ERR_ALIGN),
    (dict(codec=3, s=fake(2, 1)), q.MOE_Q4_ERR_ALIGN),
    (dict(bias=fake(4, 2)), q.MOE_Q4_ERR_ALIGN),
    (dict(out=fake(5, 1)), q.MOE_Q4_ERR_ALIGN),
    (dict(od=1, out=fake(5, 2)), q.MOE_Q4_ERR_ALIGN),
    (dict(out=fake(0)), q.MOE_Q4_ERR_ALIAS),
    (dict(out=fake(0, 256 + 128), ldx=256), q.MOE_Q4_ERR_ALIAS),   # between x's strided rows' ends
    (dict(out=fake(1, 24 * 64 - 2)), q.MOE_Q4_ERR_ALIAS),
    (dict(out=fake(2)), q.MOE_Q4_ERR_ALIAS),
    (dict(out=fake(3)), q.MOE_Q4_ERR_ALIAS),
    (dict(out=fake(4), bias=fake(4, 4)), q.MOE_Q4_ERR_ALIAS),
    (dict(L=0), q.MOE_Q4_OK),
    (dict(L=0, x=0, w=0, out=0), q.MOE_Q4_OK),
])
def test_linear_refusals(kw, status):
    assert linear(**kw) == status


def test_linear_workspace_bytes():
    assert q.moe_linear_codec_workspace_bytes("mxfp4", 1, 4096, 4096) == 0  # a single token needs none
    for codec in ("affine4_g64", "affine4_g32", "mxfp4", "nvfp4"):
        for L in (1, 16, 17, 96, 2048):
            n = q.moe_linear_codec_workspace_bytes(codec, L, 2050, 4096)
            assert n >= 0 and n % 256 == 0
            if n:
                assert linear(codec=q.CODECS[codec][0], L=L, N=2050, K=4096, wn=n - 1) == q.MOE_Q4_ERR_WORKSPACE
                assert linear(codec=q.CODECS[codec][0], L=L, N=2050, K=4096, ws=0) == q.MOE_Q4_ERR_WORKSPACE
                assert linear(codec=q.CODECS[codec][0], L=L, N=2050, K=4096, ws=fake(6, 64)) == q.MOE_Q4_ERR_ALIGN
    assert q.moe_linear_codec_workspace_bytes("mxfp4", -1, 4, 64) == 0
    assert q.moe_linear_codec_workspace_bytes(9, 1, 4, 64) == 0


def topk(z=None, dt=1, ld=None, bias=0, T=4, k=3, E=10, score=0, norm=1, ids=None, w=None):
    p = lambda v, i: fake(i) if v is None else v  # noqa: E731
    return q.lib().moe_router_topk(p(z, 0), dt, E if ld is None else ld, bias, T, k, E, score, norm, 1.0, p(ids, 2), p(w, 3),
                                   None)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), q.MOE_Q4_ERR_SHAPE),
    (dict(k=0), q.MOE_Q4_ERR_SHAPE),
    (dict(k=11), q.MOE_Q4_ERR_SHAPE),
    (dict(ld=9), q.MOE_Q4_ERR_SHAPE),
    (dict(E=16385), q.MOE_Q4_ERR_UNSUPPORTED),
    (dict(k=65, E=100), q.MOE_Q4_ERR_UNSUPPORTED),
    (dict(dt=3), q.MOE_Q4_ERR_UNSUPPORTED),
    (dict(score=2), q.MOE_Q4_ERR_UNSUPPORTED),
    (dict(norm=2), q.MOE_Q4_ERR_UNSUPPORTED),
    (dict(T=q.MOE_Q4_ROUTER_MAX_T + 1, E=1, k=1), q.MOE_Q4_ERR_UNSUPPORTED),
    (dict(z=0), q.MOE_Q4_ERR_NULL),
    (dict(ids=0), q.MOE_Q4_ERR_NULL),
    (dict(w=0), q.MOE_Q4_ERR_NULL),
    (dict(z=fake(0, 2)), q.MOE_Q4_ERR_ALIGN),
    (dict(dt=0, z=fake(0, 1)), q.MOE_Q4_ERR_ALIGN),
    (dict(bias=fake(1, 2)), q.MOE_Q4_ERR_ALIGN),
    (dict(ids=fake(2, 2)), q.MOE_Q4_ERR_ALIGN),
    (dict(w=fake(3, 1)), q.MOE_Q4_ERR_ALIGN),
    (dict(ids=fake(0, 156)), q.MOE_Q4_ERR_ALIAS),
    (dict(w=fake(2, 44)), q.MOE_Q4_ERR_ALIAS),
    (dict(w=fake(1), bias=fake(1, 8)), q.MOE_Q4_ERR_ALIAS),
    (dict(T=0, z=0), q.MOE_Q4_OK),
])
def test_topk_refusals(kw, status):
    assert topk(**kw) == status


def topk_back(z=None, dt=1, ld=None, T=4, k=3, E=10, score=0, norm=1, ids=None, g=None, d=None, ldd=None):
    p = lambda v, i: fake(i) if v is None else v  # noqa: E731
    return q.lib().moe_router_topk_backward(p(z, 0), dt, E if ld is None else ld, p(ids, 2), p(g, 3), T, k, E, score, norm,
                                            1.0, p(d, 4), E if ldd is None else ldd, None)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), q.MOE_Q4_ERR_SHAPE), (dict(k=0), q.MOE_Q4_ERR_SHAPE), (dict(ldd=9), q.MOE_Q4_ERR_SHAPE),
    (dict(ld=9), q.MOE_Q4_ERR_SHAPE), (dict(k=65, E=70), q.MOE_Q4_ERR_UNSUPPORTED), (dict(dt=9), q.MOE_Q4_ERR_UNSUPPORTED),
    (dict(g=0), q.MOE_Q4_ERR_NULL), (dict(d=0), q.MOE_Q4_ERR_NULL), (dict(d=fake(4, 2)), q.MOE_Q4_ERR_ALIGN),
    (dict(T=q.MOE_Q4_ROUTER_MAX_T + 1, k=1), q.MOE_Q4_ERR_UNSUPPORTED),
    (dict(d=fake(0)), q.MOE_Q4_ERR_ALIAS), (dict(d=fake(3, 44)), q.MOE_Q4_ERR_ALIAS), (dict(d=fake(2)), q.MOE_Q4_ERR_ALIAS),
    (dict(T=0), q.MOE_Q4_OK),
])
def test_topk_backward_refusals(kw, status):
    assert topk_back(**kw) == status


def balance(z=None, dt=1, ld=None, ids=None, mask=0, S=2, T=5, k=2, E=8, score=0, loss=None, counts=None, tokens=None,
            ws=None, wn=1 << 30):
    p = lambda v, i: fake(i) if v is None else v  # noqa: E731
    return q.lib().moe_balance_loss(p(z, 0), dt, E if ld is None else ld, p(ids, 1), mask, S, T, k, E, score, 1.0,
                                    p(loss, 3), p(counts, 4), p(tokens, 5), p(ws, 6), wn, None)


@pytest.mark.parametrize("kw,status", [
    (dict(S=-1), q.MOE_Q4_ERR_SHAPE), (dict(T=-1), q.MOE_Q4_ERR_SHAPE), (dict(k=9), q.MOE_Q4_ERR_SHAPE),
    (dict(ld=7), q.MOE_Q4_ERR_SHAPE), (dict(E=16385, k=1), q.MOE_Q4_ERR_UNSUPPORTED),
    (dict(S=65536, T=1), q.MOE_Q4_ERR_UNSUPPORTED), (dict(dt=4), q.MOE_Q4_ERR_UNSUPPORTED),
    (dict(score=7), q.MOE_Q4_ERR_UNSUPPORTED), (dict(z=0), q.MOE_Q4_ERR_NULL), (dict(ids=0), q.MOE_Q4_ERR_NULL),
    (dict(loss=0), q.MOE_Q4_ERR_NULL), (dict(counts=0), q.MOE_Q4_ERR_NULL), (dict(tokens=0), q.MOE_Q4_ERR_NULL),
    (dict(ws=0), q.MOE_Q4_ERR_WORKSPACE), (dict(wn=64), q.MOE_Q4_ERR_WORKSPACE), (dict(ws=fake(6, 128)), q.MOE_Q4_ERR_ALIGN),
    (dict(z=fake(0, 2)), q.MOE_Q4_ERR_ALIGN), (dict(counts=fake(0, 64)), q.MOE_Q4_ERR_ALIAS),
    (dict(loss=fake(6)), q.MOE_Q4_ERR_ALIAS), (dict(tokens=fake(4, 60)), q.MOE_Q4_ERR_ALIAS),
    (dict(mask=fake(2), loss=fake(2, 8)), q.MOE_Q4_ERR_ALIAS),
    (dict(T=q.MOE_Q4_ROUTER_MAX_T + 1), q.MOE_Q4_ERR_UNSUPPORTED), (dict(ws=fake(0)), q.MOE_Q4_ERR_ALIAS),
    (dict(ws=fake(1)), q.MOE_Q4_ERR_ALIAS), (dict(ws=fake(2), mask=fake(2, 8)), q.MOE_Q4_ERR_ALIAS), (dict(S=0), q.MOE_Q4_OK),
])
def test_balance_refusals(kw, status):
    assert balance(**kw) == status


def balance_back(z=None, dt=1, ld=None, mask=0, counts=None, tokens=None, g=None, S=2, T=5, k=2, E=8, score=0, d=None,
                 ldd=None):
    p = lambda v, i: fake(i) if v is None else v  # noqa: E731
    return q.lib().moe_balance_loss_backward(p(z, 0), dt, E if ld is None else ld, mask, p(counts, 2), p(tokens, 3), p(g, 4),
                                             S, T, k, E, score, 1.0, p(d, 5), E if ldd is None else ldd, None)


@pytest.mark.parametrize("kw,status", [
    (dict(S=-1), q.MOE_Q4_ERR_SHAPE), (dict(ldd=7), q.MOE_Q4_ERR_SHAPE), (dict(k=0), q.MOE_Q4_ERR_SHAPE),
    (dict(score=-1), q.MOE_Q4_ERR_UNSUPPORTED), (dict(counts=0), q.MOE_Q4_ERR_NULL), (dict(d=0), q.MOE_Q4_ERR_NULL),
    (dict(d=fake(5, 1)), q.MOE_Q4_ERR_ALIGN), (dict(d=fake(0)), q.MOE_Q4_ERR_ALIAS), (dict(d=fake(4)), q.MOE_Q4_ERR_ALIAS),
    (dict(mask=fake(1), d=fake(1, 8)), q.MOE_Q4_ERR_ALIAS), (dict(T=0), q.MOE_Q4_OK), (dict(S=0), q.MOE_Q4_OK),
])
def test_balance_backward_refusals(kw, status):
    assert balance_back(**kw) == status


def test_tile_plans_keep_their_sums_small():
    # (nvfp4 needs room for nothing but the sums of a split K: 16 at most)
    for L in (17, 33, 65, 129, 300, 1000, 5000):
        for N in (1, 63, 64, 500, 4096, 20000):
            for K in (32, 128, 160, 2048, 14336):
                n = q.moe_linear_codec_workspace_bytes("nvfp4", L, N, K)
                assert n % 256 == 0 and n <= 16 * L * N * 4 + 256, (L, N, K)


def test_balance_workspace_grows_with_experts():
    assert q.moe_balance_loss_workspace_bytes(1, 1000, 64) % 256 == 0
    assert 0 < q.moe_balance_loss_workspace_bytes(1, 1000, 64) < q.moe_balance_loss_workspace_bytes(1, 1000, 256)
    assert q.moe_balance_loss_workspace_bytes(0, 10, 64) == 0
    assert q.moe_balance_loss_workspace_bytes(1, 10, 16385) == 0


def test_bindings_refuse_host_tensors():
    x = torch.zeros(2, 64, dtype=torch.bfloat16)
    w, s, b = torch.zeros(8, 8, dtype=torch.int32), torch.zeros(8, 1, dtype=torch.bfloat16), torch.zeros(8, 1, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        q.moe_linear_codec_forward("affine4_g64", x, w, s, b)
    with pytest.raises(ValueError):
        q.moe_linear_codec_forward("affine8_g64", x, w, s, b)
    z = torch.zeros(4, 8)
    with pytest.raises(ValueError):
        q.moe_router_topk(z, 2)
    with pytest.raises(ValueError):
        q.moe_balance_loss(z, torch.zeros(4, 2, dtype=torch.int32))


def test_given_outputs_are_refused_where_a_gradient_is_due():
    z = torch.zeros(4, 8, requires_grad=True)
    ids, w = torch.empty(4, 2, dtype=torch.int32), torch.empty(4, 2)
    for kw in (dict(topk_ids=ids), dict(topk_weights=w), dict(topk_ids=ids, topk_weights=w)):
        with pytest.raises(RuntimeError, match="gradient"):
            q.moe_router_topk(z, 2, **kw)
        with torch.no_grad(), pytest.raises(ValueError, match="device"):  # past that check
            q.moe_router_topk(z, 2, **kw)


# ---- the references themselves ----

@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("norm", [True, False])
def test_route_reference_gradient_against_differences(score, norm):
    rng = np.random.default_rng(3)
    z = rng.normal(size=(5, 11))
    ids, w = R.route(z, 4, None, score, norm, 1.7)
    ids = ids.copy()
    ids[1, 2] = ids[1, 0]   # the same expert twice
    ids[2, 3] = -1          # a route left out
    g = rng.normal(size=ids.shape)
    dz = R.route_backward(z, ids, g, score, norm, 1.7)
    h = 1e-5
    for t in range(z.shape[0]):
        for e in range(z.shape[1]):
            up, dn = z.copy(), z.copy()
            up[t, e] += h
            dn[t, e] -= h
            d = ((R.route_weights(up, ids, score, norm, 1.7) - R.route_weights(dn, ids, score, norm, 1.7)) * g).sum() / (2 * h)
            assert abs(d - dz[t, e]) < 1e-8


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_balance_reference_gradient_against_differences(score):
    rng = np.random.default_rng(4)
    z = rng.normal(size=(12, 7))
    ids = np.stack([rng.permutation(7)[:3] for _ in range(12)])
    mask = np.array([1, 1, 1, 0, 1, 1, 0, 0, 1, 1, 1, 1])
    loss, counts, tokens = R.balance(z, ids, 0.5, score, 3, mask)
    dl = rng.normal(size=3)
    dz = R.balance_backward(z, counts, tokens, dl, 3, 0.5, score, mask)
    h = 1e-5
    for t in range(12):
        for e in range(7):
            up, dn = z.copy(), z.copy()
            up[t, e] += h
            dn[t, e] -= h
            d = ((R.balance(up, ids, 0.5, score, 3, mask)[0] - R.balance(dn, ids, 0.5, score, 3, mask)[0]) * dl).sum() / (2 * h)
            assert abs(d - dz[t, e]) < 1e-8


def test_route_reference_orders_ties_and_nan():
    z = np.array([[1.0, 3.0, 3.0, np.nan, -np.inf, 3.0]])
    assert R.route(z, 6, None, "softmax", True, 1.0)[0].tolist() == [[1, 2, 5, 0, 4, 3]]
