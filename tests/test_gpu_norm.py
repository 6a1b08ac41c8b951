"""The norm, its gradient and the quantization on the GPU against 64-bit
references (needs an MI355X)."""

import pytest
import torch

import quantized_expert_gather_amd as q
from tests import around_refs as R

pytestmark = pytest.mark.gpu
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
EPS = 1e-6


def rand(shape, dtype, seed, size=1.0):
    g = torch.Generator().manual_seed(seed)
    return (size * torch.randn(shape, generator=g)).to(dtype)


def dev(t):
    return None if t is None else t.cuda()


def check_norm(T, H, x=BF16, res=BF16, w=BF16, seed=0):
    print("[case] norm", T, H, x, res, w, flush=True)
    xv = rand((T, H), x, seed)
    rv = rand((T, H), res, seed + 1) if res else None
    wv = rand((H,), w, seed + 2) if w else None
    total = R.total_of(xv, rv)
    y, bound = R.norm(total, wv, EPS)
    got = q.moe_rms_norm(dev(xv), dev(wv), residual=dev(rv), eps=EPS)
    if res:
        got, gt = got
        assert gt.dtype == res and torch.equal(gt.cpu(), total)
    R.check(got, y, bound, x)
    got = q.moe_rms_norm_fp8(dev(xv), dev(wv), residual=dev(rv), eps=EPS)
    if res:
        assert torch.equal(got[2].cpu(), total)
    R.check_codes(got[0], got[1], y, slack=60 * R.U)


@pytest.mark.parametrize("H", [1, 7, 8, 64, 120, 127, 128, 129, 130, 500, 512, 513, 2047, 2048, 2050, 4096, 4104, 6144, 8192,
                               8193, 16384])
@pytest.mark.parametrize("T", [1, 5])
def test_norm_sizes(T, H):
    check_norm(T, H)


@pytest.mark.parametrize("T,H", [(37, 128), (513, 96), (600, 2050), (777, 4096), (520, 6144), (700, 8192), (530, 16383), (3000, 256)])
def test_norm_many_rows(T, H):
    check_norm(T, H)


@pytest.mark.parametrize("x", [BF16, F16, F32])
@pytest.mark.parametrize("res", ["none", "same", "f32"])
@pytest.mark.parametrize("w", [None, BF16, F16, F32])
def test_norm_types(x, res, w):
    for H in (192, 1000):
        check_norm(6, H, x, {"none": None, "same": x, "f32": F32}[res], w, seed=3)


@pytest.mark.parametrize("out", [BF16, F16, F32])
def test_norm_out_types_and_given_outputs(out):
    x, r, w = rand((9, 300), BF16, 1), rand((9, 300), BF16, 2), rand((300,), F32, 3)
    total = R.total_of(x, r)
    y, bound = R.norm(total, w, EPS)
    got, _ = q.moe_rms_norm(dev(x), dev(w), residual=dev(r), eps=EPS, out_dtype=out)
    R.check(got, y, bound, out)
    buf = torch.full((9, 320), 7.0, dtype=out, device="cuda")
    stream = dev(r)
    got, t = q.moe_rms_norm(dev(x), dev(w), residual=stream, eps=EPS, total=stream, out=buf[:, 4:304])
    assert t is stream and torch.equal(stream.cpu(), total)  # in place
    R.check(buf[:, 4:304], y, bound, out)
    assert (buf[:, :4] == 7).all() and (buf[:, 304:] == 7).all()


def test_norm_strided_rows_and_unaligned_starts():
    for off in (0, 1, 3):
        x = rand((5, 400), BF16, off)[:, off:off + 257]
        r = rand((5, 300), F32, off)[:, off:off + 257]
        w = rand((300,), F16, 2)[off:off + 257]
        total = R.total_of(x, r)
        y, bound = R.norm(total, w, EPS)
        xb, rb = torch.zeros(5, 400, dtype=BF16, device="cuda"), torch.zeros(5, 300, device="cuda")
        xb[:, off:off + 257], rb[:, off:off + 257] = x.cuda(), r.cuda()
        codes, scales = torch.empty(5, 333, dtype=torch.uint8, device="cuda").fill_(9), torch.empty(5, 3, device="cuda")
        got = q.moe_rms_norm_fp8(xb[:, off:off + 257], w.cuda().clone(), residual=rb[:, off:off + 257], eps=EPS,
                                 codes=codes.view(R.F8)[:, off:off + 257], scales=scales)
        R.check_codes(got[0], got[1], y)
        assert torch.equal(got[2].cpu(), total)
        rest = torch.cat((codes[:, :off], codes[:, off + 257:]), 1)
        assert (rest == 9).all()


def test_norm_offsets_past_32_bits():
    ld = (1 << 30) + 64
    big = torch.empty(2 * ld + 512, dtype=BF16, device="cuda")
    x = big.as_strided((3, 512), (ld, 1))
    v = rand((3, 512), BF16, 4)
    x.copy_(v)
    y, bound = R.norm(v, None, EPS)
    R.check(q.moe_rms_norm(x, eps=EPS), y, bound)
    out = torch.empty(2 * ld + 512, dtype=BF16, device="cuda").as_strided((3, 512), (ld, 1))
    q.moe_rms_norm(x, eps=EPS, out=out)
    R.check(out, y, bound)
    codes, scales = q.moe_quantize_fp8(x)
    R.check_codes(codes, scales, v, slack=4 * R.U)


def test_norm_of_more_rows_than_a_launch_holds():
    T = (1 << 25) + 40  # of 8 channels, 16 a workgroup, 2^21 workgroups a launch
    print("[case] norm launches", T, flush=True)
    x = torch.randint(1, 5, (T, 8), device="cuda", dtype=torch.int8).to(BF16)
    got = q.moe_rms_norm(x)
    for i in (slice(0, 40), slice((1 << 25) - 40, (1 << 25) + 40)):
        y, bound = R.norm(x[i].cpu(), None, 1e-6)
        R.check(got[i], y, bound, BF16)
    v = torch.rsqrt(x.float().square().mean(1) + 1e-6)
    assert ((got[:, 0].float() - x[:, 0].float() * v).abs() <= 2.0 ** -8 * got[:, 0].float() * 1.01).all()


def test_norm_zeros_infinities_and_nan():
    x = rand((6, 384), F32, 5)
    x[1] = 0
    x[2, 130] = float("inf")
    x[3, 5] = float("nan")
    x[4] *= 1e-30
    y = q.moe_rms_norm(x.cuda(), eps=EPS).cpu()
    assert (y[1] == 0).all() and (y[2, :130] == 0).all() and torch.isnan(y[2, 130])
    assert torch.isnan(y[3]).all()
    for t in (0, 5):
        ref, bound = R.norm(x[t:t + 1], None, EPS)
        R.check(y[t:t + 1], ref, bound)
    ref, bound = R.norm(x[4:5], None, EPS)  # the squares vanish beside eps
    assert ((y[4:5] - ref).abs() <= 50 * R.U * ref.abs()).all()
    codes, scales = q.moe_rms_norm_fp8(x.cuda(), eps=EPS)
    codes, scales = codes.cpu().float(), scales.cpu()
    assert (codes[1] == 0).all() and (scales[1] == 2.0 ** -126).all()
    assert torch.isnan(codes[3]).all() and torch.isnan(codes[2, 130]) and (codes[2, :128] == 0).all()
    R.check_codes(codes[:1].to(R.F8), scales[:1], R.norm(x[:1], None, EPS)[0])


@pytest.mark.parametrize("T,H", [(1, 1), (3, 100), (5, 128), (40, 129), (1, 6144), (700, 512), (1030, 2050), (600, 4096), (9, 16384),
                                 (2000, 96), (515, 8000)])
def test_norm_backward_sizes(T, H):
    print("[case] norm backward", T, H, flush=True)
    check_backward(T, H, BF16, BF16, BF16, True)


@pytest.mark.parametrize("T,H", [(20011, 100), (70000, 16), (9001, 500), (3000, 1030), (2500, 4090), (1500, 4104), (600, 9001)])
def test_norm_backward_many_rows(T, H):
    print("[case] norm backward rows", T, H, flush=True)
    check_backward(T, H, F32, BF16, F32, True, seed=5)


def check_backward(T, H, r, dy, w, dtotal, seed=0):
    rv, yv = rand((T, H), r, seed), rand((T, H), dy, seed + 1)
    wv = rand((H,), w, seed + 2) if w else None
    tv = rand((T, H), r, seed + 3) if dtotal else None
    dx, bx, dw, bw = R.norm_backward(rv, wv, yv, tv, EPS, rounds=T)
    gx, gw = q.moe_rms_norm_backward(dev(rv), dev(wv), dev(yv), dtotal=dev(tv), eps=EPS)
    R.check(gx, dx, bx, r)
    assert (gw is None) == (w is None)
    if w:
        R.check(gw, dw, bw, w)


@pytest.mark.parametrize("r", [BF16, F16, F32])
@pytest.mark.parametrize("dy", [BF16, F16, F32])
@pytest.mark.parametrize("w", [None, BF16, F16, F32])
def test_norm_backward_types(r, dy, w):
    print("[case] norm backward", r, dy, w, flush=True)
    for dtotal in (False, True):
        check_backward(13, 333, r, dy, w, dtotal, seed=4)


def test_norm_backward_against_differences():
    r, w, dy = rand((3, 40), F32, 1).double(), rand((40,), F32, 2).double(), rand((3, 40), F32, 3).double()
    gx, gw = q.moe_rms_norm_backward(r.float().cuda(), w.float().cuda(), dy.float().cuda(), eps=EPS)
    f = lambda a, b: (R.norm(a, b, EPS)[0] * dy).sum()  # noqa: E731
    h = 1e-5
    for t, c in ((0, 0), (1, 17), (2, 39)):
        e = torch.zeros_like(r)
        e[t, c] = h
        assert abs((f(r + e, w) - f(r - e, w)) / (2 * h) - gx.cpu()[t, c]) < 2e-5  # gradients near 1: 120 roundings of fp32
    for c in (0, 21):
        e = torch.zeros_like(w)
        e[c] = h
        assert abs((f(r, w + e) - f(r, w - e)) / (2 * h) - gw.cpu()[c]) < 2e-5


@pytest.mark.parametrize("res", [None, BF16, F32])
def test_norm_autograd(res):
    x, w = rand((33, 256), BF16, 1).cuda().requires_grad_(), rand((256,), F32, 2).cuda().requires_grad_()
    r = rand((33, 256), res, 3).cuda().requires_grad_() if res else None
    dy, dt = rand((33, 256), BF16, 4), rand((33, 256), res or BF16, 5)
    got = q.moe_rms_norm(x, w, residual=r, eps=EPS)
    y, total = got if res else (got, None)
    outs, grads = ([y, total], [dy.cuda(), dt.cuda()]) if res else ([y], [dy.cuda()])
    torch.autograd.backward(outs, grads)
    tv = R.total_of(x.detach().cpu(), None if r is None else r.detach().cpu())
    dx, bx, dw, bw = R.norm_backward(tv, w.detach().cpu(), dy, dt if res else None, EPS, rounds=33)
    R.check(w.grad, dw, bw)
    if res:
        R.check(r.grad, dx, bx)
    if res != F32:
        R.check(x.grad, dx, bx)
    else:  # rounded to fp32, then to x's type
        R.check(x.grad, dx, bx + R.U * dx.abs())
    if res:  # one of the two results alone
        for only in (0, 1):
            for t in (x, w, r):
                t.grad = None
            out = q.moe_rms_norm(x, w, residual=r, eps=EPS)
            torch.autograd.backward([out[only]], [grads[only]])
            if only:
                assert torch.equal(r.grad, grads[1]) and w.grad is None
            else:
                dx1, bx1, _, _ = R.norm_backward(tv, w.detach().cpu(), dy, None, EPS)
                R.check(r.grad, dx1, bx1)


def test_norm_deterministic():
    r, dy, w = rand((900, 1000), BF16, 1).cuda(), rand((900, 1000), BF16, 2).cuda(), rand((1000,), F32, 3).cuda()
    a = q.moe_rms_norm_backward(r, w, dy, eps=EPS)
    for _ in range(3):
        b = q.moe_rms_norm_backward(r, w, dy, eps=EPS)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("x", [BF16, F16, F32])
@pytest.mark.parametrize("rows", [1, 128])
@pytest.mark.parametrize("T,K", [(1, 1), (1, 128), (3, 129), (127, 100), (128, 256), (129, 300), (260, 1024), (1000, 16), (5, 16384)])
def test_quantize(x, rows, T, K):
    print("[case] quantize", x, rows, T, K, flush=True)
    v = rand((T, K), x, T + K, size=3.0)
    codes, scales = q.moe_quantize_fp8(v.cuda(), block_rows=rows)
    R.check_codes(codes, scales, v, rows, slack=4 * R.U)


def test_quantize_keeps_the_largest_and_strides():
    v = rand((130, 500), F32, 8)
    buf = torch.empty(130, 600, dtype=torch.uint8, device="cuda").fill_(3)
    x = torch.zeros(130, 520, device="cuda")
    x[:, 7:507] = v.cuda()
    codes, scales = q.moe_quantize_fp8(x[:, 7:507], block_rows=128, codes=buf.view(R.F8)[:, 11:511])
    R.check_codes(codes, scales, v, 128, slack=4 * R.U)
    assert (buf[:, :11] == 3).all() and (buf[:, 511:] == 3).all()
    assert codes.cpu().float().abs().max() == 448
    z = torch.zeros(2, 128)
    z[1, 3] = float("nan")
    codes, scales = q.moe_quantize_fp8(z.cuda())
    assert (scales.cpu() == 2.0 ** -126).all() and torch.isnan(codes.cpu().float()[1, 3]) and (codes.cpu().float()[0] == 0).all()
    z[1, 3] = float("inf")
    codes, scales = q.moe_quantize_fp8(z.cuda())
    assert torch.isinf(scales.cpu()[1, 0]) and torch.isnan(codes.cpu().float()[1, 3])


def test_norm_empty():
    x = torch.empty(0, 256, dtype=BF16, device="cuda")
    w = torch.ones(256, device="cuda")
    y, t = q.moe_rms_norm(x, w, residual=x)
    assert y.shape == t.shape == (0, 256)
    c, s = q.moe_rms_norm_fp8(x, w)
    assert c.shape == (0, 256) and s.shape == (0, 2)
    dx, dw = q.moe_rms_norm_backward(x, w, x)
    assert dx.shape == (0, 256) and (dw == 0).all()
    c, s = q.moe_quantize_fp8(x, block_rows=128)
    assert c.shape == (0, 256) and s.shape == (0, 2)


def test_norm_graph_and_stream():
    x, r, w = (rand(s, BF16, i).cuda() for i, s in enumerate(((64, 768), (64, 768), (768,))))
    dy = rand((64, 768), BF16, 7).cuda()
    ws = torch.empty(q.moe_rms_norm_backward_workspace_bytes(64, 768), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    a = q.moe_rms_norm(x, w, residual=r, stream=side)
    b = q.moe_rms_norm_fp8(x, w, residual=r, stream=side.cuda_stream)
    c = q.moe_rms_norm_backward(a[1], w, dy, workspace=ws, stream=side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, t = q.moe_rms_norm(x, w, residual=r)
        codes, scales, _ = q.moe_rms_norm_fp8(x, w, residual=r)
        dx, dw = q.moe_rms_norm_backward(t, w, dy, workspace=ws)
    for i in range(3):
        for o in (y, t, dx, dw, scales):
            o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, a[0]) and torch.equal(t, a[1]) and torch.equal(scales, b[1])
        assert torch.equal(codes.view(torch.uint8), b[0].view(torch.uint8))
        assert torch.equal(dx, c[0]) and torch.equal(dw, c[1])
