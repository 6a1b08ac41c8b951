"""The gated block's gradient in fp16 where dg = dh u silu'(g) and du = dh
silu(g) pass fp16's range and the gradients do not, and the weights' gradients
of a few tokens far apart (needs an MI355X).

fp16's dg and du are numbers over a power of two that puts the call's largest
at 2^14 or above: half a step of fp16 each, and at least 2^-25 of that unit, so
2^-39 of the largest one.  Everything else is as in around_refs."""

import pytest
import torch

import quantized_expert_gather_amd as q
from tests import around_refs as R

pytestmark = pytest.mark.gpu
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
MOST = 65504.0


def problem(T, H, I, sx, sw, sd, seed=0, positive=False):
    g = torch.Generator().manual_seed(seed + 5 * T + 3 * H + I)
    r = lambda *s: torch.rand(*s, generator=g) + 0.5 if positive else torch.randn(*s, generator=g)  # noqa: E731
    x = (sx * r(T, H)).to(F16)
    wg, wu = ((sw * r(I, H) / H ** (1.0 if positive else 0.5)).to(F16) for _ in range(2))
    return x, wg, wu, (sd * r(T, I)).clamp(-MOST, MOST).to(F16)


def reference(x, wg, wu, dh):
    """The gradients in 64 bits and their fp32 bounds: around_refs' without fp16's least step."""
    half = R.HALF[F16]
    g, u, h, bg, bu, _ = R.glu(x, wg, wu)
    x, wg, wu, dh = (t.double() for t in (x, wg, wu, dh))
    s = torch.sigmoid(g)
    slope = s * (1 + g * (1 - s))
    dg, du = dh * u * slope, dh * g * s
    e = (2 * g.abs() + 12) * R.U
    bdg = dh.abs() * (u.abs() * (0.5 * bg + e * (s + (g * s * (1 - s)).abs())) + slope.abs() * bu)
    bdu = dh.abs() * (1.1 * bg + e * (g * s).abs())
    least = 2.0 ** -39 * max(dg.abs().max(), du.abs().max())
    bdg, bdu = bdg + half * (dg.abs() + bdg) + least, bdu + half * (du.abs() + bdu) + least
    T, I = g.shape
    refs = dg @ wg + du @ wu, dg.T @ x, du.T @ x
    bounds = (bdg @ wg.abs() + bdu @ wu.abs() + (2 * I + 24) * R.U * (dg.abs() @ wg.abs() + du.abs() @ wu.abs()),
              bdg.T @ x.abs() + (T + 24) * R.U * (dg.abs().T @ x.abs()), bdu.T @ x.abs() + (T + 24) * R.U * (du.abs().T @ x.abs()))
    return refs, bounds, max(dg.abs().max(), du.abs().max())


def check(got, ref, bound, share=0.9):
    """Within the bound where fp16 holds the gradient, which `share` of it must be."""
    assert got.dtype == F16 and got.shape == ref.shape
    got = got.double().cpu()
    fits = ref.abs() + bound < MOST
    assert fits.double().mean() >= share
    tol = bound + R.HALF[F16] * (ref.abs() + bound) + R.TINY[F16]
    assert ((got - ref).abs() <= tol)[fits].all()  # (an infinity or NaN is not)
    # zeros would not do: most are further from 0 than their bound
    assert (ref.abs() > 2 * tol)[fits].double().mean() > 0.5


SIZES = [(1, 72, 64), (7, 128, 64), (40, 1416, 64), (260, 136, 200), (700, 264, 136)]


@pytest.mark.parametrize("T,H,I", SIZES)
@pytest.mark.parametrize("saved", [True, False])
@pytest.mark.parametrize("sd", [2e3, 2e4])
def test_dx_of_large_dg(T, H, I, saved, sd):
    """dg and du up to 10^7, weights that bring dx back into fp16."""
    print("[case] glu range dx", T, H, I, saved, sd, flush=True)
    x, wg, wu, dh = problem(T, H, I, 2000.0, 0.01, sd)
    refs, bounds, most = reference(x, wg, wu, dh)
    assert most > 2 * MOST
    keep = None
    if saved:
        keep = torch.empty(2, T, I, device="cuda")
        q.moe_glu(x.cuda(), wg.cuda(), wu.cuda(), saved=keep)
    dx, _, _ = q.moe_glu_backward(x.cuda(), wg.cuda(), wu.cuda(), dh.cuda(), saved=keep)
    check(dx, refs[0], bounds[0], 0.5)


@pytest.mark.parametrize("T,H,I", SIZES + [(3000, 72, 64)])
@pytest.mark.parametrize("saved", [True, False])
def test_dw_of_large_dg(T, H, I, saved):
    """dg and du up to 10^6, inputs that bring the weights' gradients back into fp16."""
    print("[case] glu range dw", T, H, I, saved, flush=True)
    x, wg, wu, dh = problem(T, H, I, 0.01, 1000.0, 1e4)
    refs, bounds, most = reference(x, wg, wu, dh)
    assert most > 2 * MOST
    keep = None
    if saved:
        keep = torch.empty(2, T, I, device="cuda")
        q.moe_glu(x.cuda(), wg.cuda(), wu.cuda(), saved=keep)
    _, dwg, dwu = q.moe_glu_backward(x.cuda(), wg.cuda(), wu.cuda(), dh.cuda(), saved=keep)
    check(dwg, refs[1], bounds[1], 0.85)
    check(dwu, refs[2], bounds[2], 0.85)


@pytest.mark.parametrize("T,H,I", [(40, 72, 64), (700, 264, 136), (8192, 64, 40)])
@pytest.mark.parametrize("sd", [2e-6, 2e-5, 1e-3])
def test_small_dg(T, H, I, sd):
    """dg and du of 10^-8 to 10^-5, summed over many tokens or with weights of some size."""
    print("[case] glu range small", T, H, I, sd, flush=True)
    x, wg, wu, dh = problem(T, H, I, 1.0, 0.02, sd, positive=True)
    refs, bounds, _ = reference(x, wg, wu, dh)
    _, dwg, dwu = q.moe_glu_backward(x.cuda(), wg.cuda(), wu.cuda(), dh.cuda())
    if T > 100 or sd > 1e-4:
        check(dwg, refs[1], bounds[1], 1.0)
        check(dwu, refs[2], bounds[2], 1.0)
    x, wg, wu, dh = problem(T, H, I, 2e-4, 100.0, sd, positive=True)
    refs, bounds, _ = reference(x, wg, wu, dh)
    check(q.moe_glu_backward(x.cuda(), wg.cuda(), wu.cuda(), dh.cuda())[0], refs[0], bounds[0], 1.0)


@pytest.mark.parametrize("T", [30, 500])
def test_channels_and_tokens_of_different_sizes(T):
    """dg and du of one call from 10^-4 to 10^5: a token's and a channel's own sums hold."""
    x, wg, wu, dh = problem(T, 136, 64, 1.0, 1.0, 1.0)
    up = 2.0 ** torch.arange(-12, 4).repeat(4)
    wu = (wu * up[:, None]).to(F16)
    dh = (dh * 2.0 ** torch.arange(-4, 6).repeat(T // 10)[:, None]).to(F16)
    refs, bounds, _ = reference(x, wg, wu, dh)
    for got, ref, bound in zip(q.moe_glu_backward(x.cuda(), wg.cuda(), wu.cuda(), dh.cuda()), refs, bounds):
        check(got, ref, bound, 1.0)


def test_zeros_and_values_that_are_none():
    x, wg, wu, dh = (t.cuda() for t in problem(50, 72, 64, 1.0, 1.0, 1e3))
    for t in q.moe_glu_backward(x, wg, wu, torch.zeros_like(dh)):
        assert (t == 0).all()
    clean = q.moe_glu_backward(x, wg, wu, dh)
    bad = dh.clone()
    bad[3], bad[4, 5] = float("inf"), float("nan")
    got = q.moe_glu_backward(x, wg, wu, bad)
    rows = [0, 1, 2] + list(range(5, 50))
    assert torch.isfinite(clean[0]).all() and torch.equal(got[0][rows], clean[0][rows])
    assert not torch.isfinite(got[0][3]).any() and torch.isnan(got[0][4]).all()
    only = torch.zeros_like(dh)
    only[7, 3] = float("inf")  # nothing finite beside it
    dx, dwg, dwu = q.moe_glu_backward(x, wg, wu, only)
    rows = [i for i in range(50) if i != 7]
    assert (dx[rows] == 0).all() and (dwg[:3] == 0).all() and (dwg[4:] == 0).all() and not torch.isfinite(dwu[3]).all()


def test_graphs_take_the_scale_of_their_own_values():
    x, wg, wu, dh = (t.cuda() for t in problem(40, 136, 64, 1.0, 1.0, 1.0))
    ws = torch.empty(q.moe_glu_backward_workspace_bytes(40, 136, 64, saved=False), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    q.moe_glu_backward(x, wg, wu, dh, workspace=ws)
    with torch.cuda.graph(graph):
        got = q.moe_glu_backward(x, wg, wu, dh, workspace=ws)
    base = dh.clone()
    for size in (1.0, 2.0 ** 13, 2.0 ** -10, 0.0):
        dh.copy_(base * size)
        for t in got:
            t.zero_()
        ws.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, q.moe_glu_backward(x, wg, wu, dh)):
            assert torch.equal(a.isfinite(), b.isfinite()) and torch.equal(a[a.isfinite()], b[b.isfinite()])


@pytest.mark.parametrize("T,H,I", [(300_000, 8192, 8), (5000, 264, 72), (700, 1032, 136)])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_weight_gradients_of_a_few_tokens(T, H, I, dtype):
    """dh is 0 but for a few tokens, at both ends and about 4 GB on in x: the weights' gradients are sums of that many
    terms, and their bounds those terms'."""
    print("[case] glu few tokens", T, H, I, dtype, flush=True)
    mid = min(T // 2, (1 << 32) // (2 * H))
    rows = torch.tensor([0, 1, mid - 1, mid, mid + 1, T - 65, T - 64, T - 2, T - 1])
    g = torch.Generator(device="cuda").manual_seed(T)
    x = torch.empty(T, H, device="cuda", dtype=dtype)
    for i in range(0, T, 20_000):
        x[i:i + 20_000] = torch.randn(min(20_000, T - i), H, generator=g, device="cuda")
    _, wg, wu, _ = problem(8, H, I, 1.0, 1.0, 1.0)
    wg, wu = wg.to(dtype), wu.to(dtype)
    some = torch.randn(len(rows), I, generator=g, device="cuda").to(dtype)
    dh = torch.zeros(T, I, device="cuda", dtype=dtype)
    dh[rows.cuda()] = some
    dx, dwg, dwu = q.moe_glu_backward(x, wg.cuda(), wu.cuda(), dh)
    few = x[rows.cuda()].cpu(), wg, wu, some.cpu()
    refs, bounds = R.glu_backward(*few)
    R.check(dx[rows.cuda()], refs[0], bounds[0], dtype)
    for got, which in ((dwg, 1), (dwu, 2)):
        R.check(got, refs[which], bounds[which], dtype)
        for i in range(len(rows)):  # the check finds each token's loss (one element off is enough, and a tenth of them are)
            keep = [j for j in range(len(rows)) if j != i]
            lost = R.glu_backward(few[0][keep], wg, wu, few[3][keep])[0][which]
            tol = bounds[which] + R.HALF[dtype] * (refs[which].abs() + bounds[which])
            assert ((lost - refs[which]).abs() > tol).double().mean() > 0.1
