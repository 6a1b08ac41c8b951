"""The 8-bit product with scales for blocks of 128 on the GPU against a 64-bit
reference (needs an MI355X)."""

import pytest
import torch

import quantized_expert_gather_amd as q
from tests import around_refs as R

pytestmark = pytest.mark.gpu
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def problem(L, N, K, bias=False, seed=0):
    g = torch.Generator().manual_seed(seed + L * 7 + N * 3 + K)
    kb = -(-K // 128)
    x = (140 * torch.randn(L, K, generator=g)).clamp(-448, 448).to(R.F8)
    w = (105 * torch.randn(N, K, generator=g)).clamp(-448, 448).to(R.F8)
    sx = torch.exp(torch.randn(L, kb, generator=g)) / 140
    sw = torch.exp(0.3 * torch.randn(-(-N // 128), kb, generator=g)) / 105
    return x, sx, w, sw, torch.randn(N, generator=g) if bias else None


def check(L, N, K, out=F32, bias=False, seed=0):
    print("[case] fp8", L, N, K, out, bias, flush=True)
    p = problem(L, N, K, bias, seed)
    ref, bound = R.linear_fp8(*p, out=out)
    got = q.moe_linear_fp8_forward(*(None if t is None else t.cuda() for t in p), out_dtype=out)
    R.check(got, ref, bound, out)


@pytest.mark.parametrize("L", [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 100, 128, 129, 257])
@pytest.mark.parametrize("N,K", [(1, 16), (16, 128), (17, 144), (130, 112), (128, 1024), (250, 2064)])
@pytest.mark.parametrize("out", [BF16, F32])
def test_sizes(L, N, K, out):
    check(L, N, K, out)


@pytest.mark.parametrize("L,N,K", [(1, 4099, 4112), (7, 2050, 512), (96, 2050, 4096), (40, 520, 8192), (300, 1000, 1040),
                                   (700, 5000, 512), (1100, 2300, 400), (2049, 4097, 272)])
@pytest.mark.parametrize("out", [F16, F32])
def test_larger(L, N, K, out):
    check(L, N, K, out, bias=True)


def test_scales_are_each_block_s_own():
    """One token and one row at a time have values in one block only."""
    L, N, K = 70, 300, 512
    x, sx, w, sw, _ = problem(L, N, K, seed=5)
    for b in range(4):
        xb = torch.zeros_like(x.view(torch.uint8))
        xb[:, b * 128:(b + 1) * 128] = x.view(torch.uint8)[:, b * 128:(b + 1) * 128]
        ref, bound = R.linear_fp8(xb.view(R.F8), sx, w, sw, None)
        for l in (70, 3):
            got = q.moe_linear_fp8_forward(xb.view(R.F8)[:l].cuda(), sx[:l].cuda(), w.cuda(), sw.cuda(), out_dtype=F32)
            R.check(got, ref[:l], bound[:l])


def test_strides_and_given_outputs():
    for L in (5, 90):
        x, sx, w, sw, bias = problem(L, 131, 272, True)
        xb = torch.zeros(L, 320, dtype=torch.uint8, device="cuda")
        xb[:, 16:288] = x.view(torch.uint8).cuda()
        out = torch.full((L, 150), 5.0, dtype=BF16, device="cuda")
        q.moe_linear_fp8_forward(xb.view(R.F8)[:, 16:288], sx.cuda(), w.cuda(), sw.cuda(), bias.cuda(), out=out[:, 3:134])
        ref, bound = R.linear_fp8(x, sx, w, sw, bias, BF16)
        R.check(out[:, 3:134], ref, bound, BF16)
        assert (out[:, :3] == 5).all() and (out[:, 134:] == 5).all()


# Each tile shape, without and with parts of the inputs, and the products by
# rows with 16 and 32 of w's rows a workgroup.
@pytest.mark.parametrize("L,N,K", [(3283, 3795, 64), (5524, 643, 7184), (2322, 2571, 64), (1817, 259, 5488), (51, 67, 2448), (1181, 771, 5408),
                                   (33, 67, 1680), (9, 6149, 272), (16, 131, 4112), (17, 4099, 400), (32, 4099, 4096), (32, 131, 2064)])
@pytest.mark.parametrize("out", [BF16, F32])
def test_tile_shapes(L, N, K, out):
    print("[case] fp8 shapes", L, N, K, out, flush=True)
    p = [t.cuda() for t in problem(L, N, K, True)]  # (the references, in 64 bits, there too)
    ref, bound = R.linear_fp8(*p, out)
    got = q.moe_linear_fp8_forward(*p, out_dtype=out)
    R.check(got, ref.cpu(), bound.cpu(), out)
    assert torch.equal(got, q.moe_linear_fp8_forward(*p, out_dtype=out))


def test_more_outputs_than_a_launch_holds():
    N = (1 << 26) + 300
    print("[case] fp8 launches", N, flush=True)
    x, sx, _, _, _ = problem(2, 64, 16)
    w = torch.randint(0, 0x7F, (N, 16), device="cuda", dtype=torch.uint8).view(R.F8)  # 0x7f is NaN
    sw = torch.rand((N + 127) // 128, 1, device="cuda") + 0.5
    got = q.moe_linear_fp8_forward(x.cuda(), sx.cuda(), w, sw, out_dtype=F32)
    for a in (0, (1 << 26) - 256, (1 << 26) + 172):  # (from a block's beginning to 128 on)
        a -= a % 128
        ref, bound = R.linear_fp8(x, sx, w[a:a + 128].cpu(), sw[a // 128:a // 128 + 1].cpu(), None)
        R.check(got[:, a:a + 128], ref, bound)
    assert torch.isfinite(got).all()


def test_offsets_past_32_bits():
    L, K = 600_000, 8192
    print("[case] fp8 offsets", L, K, flush=True)
    x = torch.randint(0, 0x7F, (L, K), device="cuda", dtype=torch.uint8).view(R.F8)
    sx = torch.rand(L, K // 128, device="cuda") + 0.5
    _, _, w, sw, _ = problem(1, 8, K)
    got = q.moe_linear_fp8_forward(x, sx, w.cuda(), sw.cuda(), out_dtype=F32)
    for i in (slice(0, 70), slice(L // 2, L // 2 + 70), slice(L - 70, L)):
        ref, bound = R.linear_fp8(x[i].cpu(), sx[i].cpu(), w, sw, None)
        R.check(got[i], ref, bound)


@pytest.mark.parametrize("L", [4, 200])
def test_nan_codes_and_scales_stay_with_their_outputs(L):
    x, sx, w, sw, _ = problem(L, 300, 640)
    ref, bound = R.linear_fp8(x, sx, w, sw, None)
    x, sx, w, sw = x.clone(), sx.clone(), w.clone(), sw.clone()
    x.view(torch.uint8)[2, 639] = 0x7F
    w.view(torch.uint8)[299, 0] = 0xFF
    sx[1, 4] = float("nan")
    sw[0, 2] = float("inf")
    got = q.moe_linear_fp8_forward(x.cuda(), sx.cuda(), w.cuda(), sw.cuda(), out_dtype=F32).cpu()
    assert torch.isnan(got[2]).all() and torch.isnan(got[:, 299]).all() and torch.isnan(got[1]).all()
    assert not torch.isfinite(got[:, :128]).any()
    rows = [0] + list(range(3, L))
    R.check(got[rows][:, 128:299], ref[rows][:, 128:299], bound[rows][:, 128:299])


@pytest.mark.parametrize("L,N,K", [(4, 300, 144), (30, 4096, 656), (200, 300, 144), (200, 300, 640), (600, 2600, 400), (1300, 2600, 656)])
@pytest.mark.parametrize("out", [BF16, F32])
def test_a_first_rows_nan_stays_with_it(L, N, K, out):
    """Odd numbers of steps, and rows that end inside one: what stands in for the rest is no other row's."""
    x, sx, w, sw = (t.cuda() for t in problem(L, N, K)[:4])
    clean = q.moe_linear_fp8_forward(x, sx, w, sw, out_dtype=out)
    bad, wbad = x.clone(), w.clone()
    bad.view(torch.uint8)[0] = 0x7F
    wbad.view(torch.uint8)[0] = 0xFF
    got = q.moe_linear_fp8_forward(bad, sx, w, sw, out_dtype=out)
    assert torch.isnan(got[0]).all() and torch.equal(got[1:], clean[1:])
    got = q.moe_linear_fp8_forward(x, sx, wbad, sw, out_dtype=out)
    assert torch.isnan(got[:, 0]).all() and torch.equal(got[:, 1:], clean[:, 1:])


def test_zero_and_subnormal_codes():
    x, sx, w, sw, _ = problem(40, 64, 256)
    x = (x.float() / 2 ** 13).to(R.F8)  # mostly subnormal
    w = (w.float() / 2 ** 12).to(R.F8)
    x[3], w[5] = 0, 0
    ref, bound = R.linear_fp8(x, sx, w, sw, None)
    for l in (40, 9):
        R.check(q.moe_linear_fp8_forward(x[:l].cuda(), sx[:l].cuda(), w.cuda(), sw.cuda(), out_dtype=F32), ref[:l], bound[:l])


def test_no_tokens():
    x, sx, w, sw, _ = problem(3, 40, 128)
    out = q.moe_linear_fp8_forward(x[:0].cuda(), sx[:0].cuda(), w.cuda(), sw.cuda())
    assert out.shape == (0, 40) and out.dtype == BF16


@pytest.mark.parametrize("L", [1, 48, 300])
def test_graph_stream_and_repeats(L):
    p = [None if t is None else t.cuda() for t in problem(L, 1000, 2048, True)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    a = q.moe_linear_fp8_forward(*p, stream=side)
    torch.cuda.synchronize()
    ws = torch.empty(max(256, q.moe_linear_fp8_workspace_bytes(L, 1000, 2048)), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b = q.moe_linear_fp8_forward(*p, workspace=ws)
    for _ in range(3):
        b.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(a, b)
        assert torch.equal(q.moe_linear_fp8_forward(*p), a)


def test_norm_into_product():
    """A layer's input: residual, norm and codes, then the product; against the whole in 64 bits."""
    for L in (1, 40, 300):
        g = torch.Generator().manual_seed(L)
        x, r = torch.randn(L, 768, generator=g).to(BF16), torch.randn(L, 768, generator=g).to(BF16)
        nw, w = 1 + 0.1 * torch.randn(768, generator=g), torch.randn(520, 768, generator=g) / 768 ** 0.5
        wc, ws = q.moe_quantize_fp8(w.cuda(), block_rows=128)
        codes, scales, total = q.moe_rms_norm_fp8(x.cuda(), nw.cuda(), residual=r.cuda())
        got = q.moe_linear_fp8_forward(codes, scales, wc, ws, out_dtype=F32)
        ref, bound = R.linear_fp8(codes.cpu(), scales.cpu(), wc.cpu(), ws.cpu(), None)
        R.check(got, ref, bound)
        y, _ = R.norm(R.total_of(x, r), nw, 1e-6)
        # codes are off by 2^-4 of a value at most, or 2^-10 of the block's scale; both factors'
        ay, aw = y.abs() + R.scales(y, 1).repeat_interleave(128, 1) * 2.0 ** -6, w.double().abs()
        aw = aw + R.scales(w, 128).repeat_interleave(128, 0)[:520].repeat_interleave(128, 1) * 2.0 ** -6
        assert ((got.double().cpu() - y @ w.double().T).abs() <= (2 * 2.0 ** -4 + 2.0 ** -8 + 1e-4) * (ay @ aw.T)).all()
