"""The gated block and its gradient on the GPU against 64-bit references (needs an MI355X)."""

import pytest
import torch

import quantized_expert_gather_amd as q
from tests import around_refs as R

pytestmark = pytest.mark.gpu
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def problem(T, H, I, dtype, seed=0):
    g = torch.Generator().manual_seed(seed + 5 * T + 3 * H + I)
    x = torch.randn(T, H, generator=g).to(dtype)
    wg, wu = ((torch.randn(I, H, generator=g) / H ** 0.5).to(dtype) for _ in range(2))
    return x, wg, wu, torch.randn(T, I, generator=g).to(dtype)


def check_forward(T, H, I, dtype):
    print("[case] glu", T, H, I, dtype, flush=True)
    x, wg, wu, _ = problem(T, H, I, dtype)
    g, u, h, bg, bu, bh = R.glu(x, wg, wu)
    saved = torch.full((2, T, I), 9.0, device="cuda")
    got = q.moe_glu(x.cuda(), wg.cuda(), wu.cuda(), saved=saved)
    R.check(got, h, bh, dtype)
    R.check(saved[0], g, bg)
    R.check(saved[1], u, bu)
    assert torch.equal(q.moe_glu(x.cuda(), wg.cuda(), wu.cuda()), got)


def check_backward(T, H, I, dtype, saved):
    print("[case] glu backward", T, H, I, dtype, saved, flush=True)
    x, wg, wu, dh = problem(T, H, I, dtype)
    refs, bounds = R.glu_backward(x, wg, wu, dh)
    d = [t.cuda() for t in (x, wg, wu)]
    keep = None
    if saved:
        keep = torch.empty(2, T, I, device="cuda")
        q.moe_glu(*d, saved=keep)
    for got, ref, bound in zip(q.moe_glu_backward(*d, dh.cuda(), saved=keep), refs, bounds):
        R.check(got, ref, bound, dtype)


@pytest.mark.parametrize("T", [1, 2, 16, 17, 32, 33, 64, 65, 100, 129, 260])
@pytest.mark.parametrize("H,I", [(8, 8), (64, 72), (136, 128), (520, 264)])
def test_forward_sizes(T, H, I):
    check_forward(T, H, I, BF16)


@pytest.mark.parametrize("T,H,I", [(4, 1024, 2048), (48, 2056, 200), (96, 512, 1416), (700, 264, 2600), (1500, 200, 1400)])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_forward_larger(T, H, I, dtype):
    check_forward(T, H, I, dtype)


# For each of the products the smallest sizes at which each tile shape was
# chosen, without and with parts of the sum's axis.
SHAPES = [(2065, 72, 2704), (131, 8272, 6304), (1537, 64, 1264), (5538, 5760, 144), (1799, 456, 1680), (132, 7976, 3136),
          (1442, 200, 1416), (612, 4632, 1624), (897, 64, 1104), (2778, 3512, 80), (45, 1480, 64), (3416, 3464, 64),
          (2739, 672, 5816), (1681, 2360, 64), (5575, 272, 3112), (2720, 2160, 200), (2776, 648, 3112), (1944, 2064, 72),
          (4287, 136, 2992), (1233, 1544, 64), (2694, 136, 1696), (38, 64, 712), (34, 2136, 2696), (4344, 200, 8208),
          (39, 1416, 1368), (5932, 144, 5688), (459, 1360, 2112), (5937, 200, 4264), (193, 1168, 1656), (3529, 136, 4232),
          (37, 904, 1032), (3481, 152, 1432), (1540, 64, 72), (134, 7056, 6496), (5436, 144, 5472)]


@pytest.mark.parametrize("T,H,I", SHAPES)
def test_tile_shapes(T, H, I):
    print("[case] glu shapes", T, H, I, flush=True)
    dtype = BF16 if T % 2 else F16
    x, wg, wu, dh = (t.cuda() for t in problem(T, H, I, dtype))  # (the references, in 64 bits, there too)
    g, u, h, bg, bu, bh = (t.cpu() for t in R.glu(x, wg, wu))
    saved = torch.full((2, T, I), 9.0, device="cuda")
    R.check(q.moe_glu(x, wg, wu, saved=saved), h, bh, dtype)
    R.check(saved[0], g, bg)
    R.check(saved[1], u, bu)
    refs, bounds = R.glu_backward(x, wg, wu, dh)
    got = q.moe_glu_backward(x, wg, wu, dh, saved=saved)
    for a, ref, bound in zip(got, refs, bounds):
        R.check(a, ref.cpu(), bound.cpu(), dtype)
    for a, b in zip(got, q.moe_glu_backward(x, wg, wu, dh, saved=saved)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("T", [1, 7, 33, 64, 130])
@pytest.mark.parametrize("H,I", [(8, 8), (72, 136), (264, 200)])
@pytest.mark.parametrize("saved", [True, False])
def test_backward_sizes(T, H, I, saved):
    check_backward(T, H, I, BF16, saved)


@pytest.mark.parametrize("T,H,I", [(40, 1024, 520), (513, 776, 256), (1000, 136, 1032), (300, 2056, 1416)])
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("saved", [True, False])
def test_backward_larger(T, H, I, dtype, saved):
    check_backward(T, H, I, dtype, saved)


def test_backward_against_differences():
    x, wg, wu, dh = problem(5, 16, 8, F16)
    dx, dwg, dwu = (t.double().cpu() for t in q.moe_glu_backward(x.cuda(), wg.cuda(), wu.cuda(), dh.cuda()))
    x, wg, wu, dh = (t.double() for t in (x, wg, wu, dh))
    f = lambda a, b, c: (R.glu(a, b, c)[2] * dh).sum()  # noqa: E731
    for which, grad in ((0, dx), (1, dwg), (2, dwu)):
        for i, j in ((0, 0), (3, 11), (4, 15)):
            a, b = [x.clone(), wg.clone(), wu.clone()], [x.clone(), wg.clone(), wu.clone()]
            a[which][i, j] += 1e-5
            b[which][i, j] -= 1e-5
            # two roundings to fp16 of numbers near 1, the first summed over up to 16
            assert abs((f(*a) - f(*b)) / 2e-5 - grad[i, j]) < 16 * 2.0 ** -11 * (1 + grad.abs().max())


def test_strides_and_given_outputs():
    for T in (6, 150):
        x, wg, wu, dh = problem(T, 136, 72, BF16)
        both = torch.cat((wg, wu)).cuda()  # halves of one matrix
        xb = torch.zeros(T, 160, dtype=BF16, device="cuda")
        xb[:, 8:144] = x.cuda()
        eb = torch.zeros(T, 81, dtype=BF16, device="cuda")
        eb[:, 5:77] = dh.cuda()
        out, dxb = torch.full((T, 90), 3.0, dtype=BF16, device="cuda"), torch.full((T, 150), 3.0, dtype=BF16, device="cuda")
        q.moe_glu(xb[:, 8:144], both[:72], both[72:], out=out[:, 1:73])
        _, _, h, _, _, bh = R.glu(x, wg, wu)
        R.check(out[:, 1:73], h, bh)
        assert (out[:, 0] == 3).all() and (out[:, 73:] == 3).all()
        grads = torch.empty(2, 72, 136, dtype=BF16, device="cuda")
        q.moe_glu_backward(xb[:, 8:144], both[:72], both[72:], eb[:, 5:77], dx=dxb[:, 7:143], dwg=grads[0], dwu=grads[1])
        refs, bounds = R.glu_backward(x, wg, wu, dh)
        for got, ref, bound in zip((dxb[:, 7:143], grads[0], grads[1]), refs, bounds):
            R.check(got, ref, bound)
        assert (dxb[:, :7] == 3).all() and (dxb[:, 143:] == 3).all()


@pytest.mark.parametrize("recompute", [False, True])
@pytest.mark.parametrize("T", [3, 200])
def test_autograd(recompute, T):
    x, wg, wu, dh = problem(T, 128, 64, BF16)
    leaves = [t.cuda().requires_grad_() for t in (x, wg, wu)]
    q.moe_glu(*leaves, recompute=recompute).backward(dh.cuda())
    refs, bounds = R.glu_backward(x, wg, wu, dh)
    for leaf, ref, bound in zip(leaves, refs, bounds):
        R.check(leaf.grad, ref, bound)
    for which in range(3):  # one alone
        one = [t.cuda().requires_grad_(i == which) for i, t in enumerate((x, wg, wu))]
        q.moe_glu(*one, recompute=recompute).backward(dh.cuda())
        assert torch.equal(one[which].grad, leaves[which].grad)
        assert all(t.grad is None for i, t in enumerate(one) if i != which)


def test_offsets_past_32_bits():
    """Rows of x past 4 GB.  dw's sum of 300000 terms a result: (T + 24) 2^-24 of
    their magnitudes, as everywhere."""
    T, H, I = 300_000, 8192, 8
    print("[case] glu offsets", T, H, I, flush=True)
    _, wg, wu, _ = problem(8, H, I, BF16)
    x = torch.empty(T, H, device="cuda", dtype=BF16)
    for i in range(0, T, 20_000):
        x[i:i + 20_000] = torch.randn(min(20_000, T - i), H, device="cuda")
    dh = torch.randn(T, I, device="cuda").to(BF16)
    d = [x, wg.cuda(), wu.cuda()]
    h = q.moe_glu(*d)
    dx, dwg, dwu = q.moe_glu_backward(*d, dh)
    wsum, bsum, mag = [0.0, 0.0], [0.0, 0.0], 0.0
    for i in range(0, T, 20_000):
        part = slice(i, min(i + 20_000, T))
        (rx, *rw), (bx, *bw) = R.glu_backward(x[part], d[1], d[2], dh[part])
        for k in range(2):
            wsum[k] = wsum[k] + rw[k]
            bsum[k] = bsum[k] + bw[k]
        if i in (0, 140_000, 280_000):
            R.check(dx[part], rx.cpu(), bx.cpu(), BF16)
            _, _, rh, _, _, bh = R.glu(x[part], d[1], d[2])
            R.check(h[part], rh.cpu(), bh.cpu(), BF16)
        g, u, *_ = R.glu(x[part], d[1], d[2])
        s = torch.sigmoid(g)
        for e in (dh[part].double() * u * s * (1 + g * (1 - s)), dh[part].double() * g * s):
            mag = mag + e.abs().T @ x[part].double().abs()
    for k, got in enumerate((dwg, dwu)):  # (a part's own bound has its number of tokens' roundings alone)
        R.check(got, wsum[k].cpu(), (bsum[k] + T * R.U * mag).cpu(), BF16)


def test_a_norm_and_the_block_as_they_are_used():
    """Norm with the residual, the block behind it and the sum carried on, and all
    gradients through autograd; each step against 64 bits at its own inputs."""
    T, H, I = 203, 264, 136
    x, wg, wu, dh = problem(T, H, I, BF16)
    g = torch.Generator().manual_seed(3)
    res, w, dtotal = torch.randn(T, H, generator=g), 1 + torch.randn(H, generator=g) / 4, torch.randn(T, H, generator=g)
    leaves = [t.cuda().requires_grad_() for t in (x, res, w, wg, wu)]
    y, total = q.moe_rms_norm(leaves[0], leaves[2], leaves[1])
    y.retain_grad()
    h = q.moe_glu(y, leaves[3], leaves[4])
    torch.autograd.backward([h, total], [dh.cuda(), dtotal.cuda()])
    sums = R.total_of(x, res)
    assert torch.equal(total.detach().cpu(), sums)
    R.check(y.detach(), *R.norm(sums, w, 1e-6), BF16)
    mid = y.detach().cpu()
    R.check(h.detach(), *(R.glu(mid, wg, wu)[i] for i in (2, 5)), BF16)
    refs, bounds = R.glu_backward(mid, wg, wu, dh)
    for t, ref, bound in zip((y, leaves[3], leaves[4]), refs, bounds):
        R.check(t.grad, ref, bound, BF16)
    dx, bound, dw, wbound = R.norm_backward(sums, w, y.grad.cpu(), dtotal, 1e-6)
    R.check(leaves[1].grad, dx, bound)
    R.check(leaves[0].grad, dx, bound, BF16)
    R.check(leaves[2].grad, dw, wbound)


@pytest.mark.parametrize("T", [5, 140])
def test_infinities_and_nan_stay_with_their_rows(T):
    x, wg, wu, _ = problem(T, 200, 64, BF16)
    _, _, h, _, _, bh = R.glu(x, wg, wu)
    x, wg = x.clone(), wg.clone()
    x[1, 199] = float("inf")
    x[2, 0] = float("nan")
    wg[63, 199] = float("nan")
    got = q.moe_glu(x.cuda(), wg.cuda(), wu.cuda()).cpu()
    assert torch.isnan(got[2]).all() and torch.isnan(got[:, 63]).all()
    rows = [0] + list(range(3, T))
    R.check(got[rows][:, :63], h[rows][:, :63], bh[rows][:, :63])


@pytest.mark.parametrize("T,H,I", [(6, 72, 64), (140, 72, 64), (140, 200, 520), (1500, 328, 1400), (2600, 136, 2600)])
@pytest.mark.parametrize("odd", [float("nan"), float("inf")])
def test_a_first_rows_nan_or_infinity_stays_with_it(T, H, I, odd):
    """Odd numbers of steps, and rows that end inside one: what stands in for the rest is no other row's."""
    x, wg, wu, dh = (t.cuda() for t in problem(T, H, I, F16))
    clean = q.moe_glu(x, wg, wu)
    dclean = q.moe_glu_backward(x, wg, wu, dh)[0]
    bad, dbad = x.clone(), dh.clone()
    bad[0], dbad[0, :] = odd, odd
    got, dx = q.moe_glu(bad, wg, wu), q.moe_glu_backward(x, wg, wu, dbad)[0]
    assert torch.equal(got[1:], clean[1:]) and torch.equal(dx[1:], dclean[1:])
    assert not torch.isfinite(got[0]).all() and not torch.isfinite(dx[0]).any()
    w = wg.clone()
    w[0] = odd
    assert torch.equal(q.moe_glu(x, w, wu)[:, 1:], clean[:, 1:])


@pytest.mark.parametrize("T", [3, 90])
def test_an_infinity_gives_one(T):
    """The last inputs of rows that end inside a step: inf times a weight, not inf times zero."""
    x, wg, wu, _ = problem(T, 72, 64, BF16)
    x[1] = 0
    x[1, 71] = float("inf")
    wg[:, 71], wu[:, 71] = 1, 2
    got = q.moe_glu(x.cuda(), wg.cuda(), wu.cuda()).cpu()
    assert (got[1] == float("inf")).all() and torch.isfinite(got[0]).all() and torch.isfinite(got[2:]).all()


def test_large_gates():
    x, wg, wu, dh = problem(70, 64, 64, BF16)
    x = x * 60  # gates of a few hundred: the sigmoid is 0 or 1
    g, u, h, bg, bu, bh = R.glu(x, wg, wu)
    R.check(q.moe_glu(x.cuda(), wg.cuda(), wu.cuda()), h, bh)
    refs, bounds = R.glu_backward(x, wg, wu, dh)
    for got, ref, bound in zip(q.moe_glu_backward(x.cuda(), wg.cuda(), wu.cuda(), dh.cuda()), refs, bounds):
        R.check(got, ref, bound)


def test_no_tokens():
    x, wg, wu, dh = (t.cuda() for t in problem(2, 64, 40, F16))
    assert q.moe_glu(x[:0], wg, wu).shape == (0, 40)
    dx, dwg, dwu = q.moe_glu_backward(x[:0], wg, wu, dh[:0])
    assert dx.shape == (0, 64) and (dwg == 0).all() and (dwu == 0).all() and dwg.shape == (40, 64)


@pytest.mark.parametrize("T", [4, 96, 300])
def test_graph_stream_and_repeats(T):
    x, wg, wu, dh = (t.cuda() for t in problem(T, 1024, 512, BF16))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    keep = torch.empty(2, T, 512, device="cuda")
    h = q.moe_glu(x, wg, wu, saved=keep, stream=side)
    a = q.moe_glu_backward(x, wg, wu, dh, saved=keep, stream=side)
    torch.cuda.synchronize()
    ws = torch.empty(q.moe_glu_backward_workspace_bytes(T, 1024, 512), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    saved = torch.empty(2, T, 512, device="cuda")
    with torch.cuda.graph(graph):
        hg = q.moe_glu(x, wg, wu, saved=saved)
        b = q.moe_glu_backward(x, wg, wu, dh, saved=saved, workspace=ws)
    for _ in range(3):
        for t in (hg, saved, *b):
            t.zero_()
        ws.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(hg, h) and all(torch.equal(s, t) for s, t in zip(a, b))
        c = q.moe_glu_backward(x, wg, wu, dh, saved=keep)
        assert all(torch.equal(s, t) for s, t in zip(a, c))


def test_saved_projections_at_any_start():
    for T, I in ((200, 64), (1500, 1408)):  # rows of whole 64 bytes, at a start that is none
        x, wg, wu, _ = (t.cuda() for t in problem(T, 136, I, BF16))
        keep, room = torch.empty(2, T, I, device="cuda"), torch.full((2 * T * I + 64,), 7.0, device="cuda")
        h = q.moe_glu(x, wg, wu, saved=keep)
        part = room[4:4 + 2 * T * I].view(2, T, I)
        assert torch.equal(q.moe_glu(x, wg, wu, saved=part), h) and torch.equal(part, keep)
        assert (room[:4] == 7).all() and (room[4 + 2 * T * I:] == 7).all()


def test_two_streams_at_once():
    """Calls of both streams between each other, each with its own workspace."""
    p, r = [[t.cuda() for t in problem(T, 1032, 520, F16)] for T in (300, 70)]
    def run(a):
        keep = torch.empty(2, a[0].shape[0], 520, device="cuda")
        return [q.moe_glu(*a[:3], saved=keep), *q.moe_glu_backward(*a, saved=keep)]
    refs = [run(p), run(r)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(8):
        for i, a in enumerate((p, r)):
            with torch.cuda.stream(streams[i]):
                got[i].append(run(a))
    torch.cuda.synchronize()
    for i in range(2):
        for g in got[i]:
            assert all(torch.equal(s, t) for s, t in zip(g, refs[i]))


def test_backward_of_a_captured_step_is_refused(monkeypatch):
    x, wg, wu, dh = (t.cuda() for t in problem(4, 64, 64, BF16))
    x.requires_grad_()
    h = q.moe_glu(x, wg, wu)
    y = q.moe_rms_norm(x)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
    with pytest.raises(RuntimeError, match="moe_glu_backward"):
        h.backward(dh)
    with pytest.raises(RuntimeError, match="moe_rms_norm_backward"):
        y.backward(x.detach())
