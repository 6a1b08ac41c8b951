"""Rounding of the norm's and the quantization's codes, and the norm's weight
gradient where a few rows alone count (needs an MI355X)."""

import pytest
import torch

import quantized_expert_gather_amd as q
from tests import around_refs as R

pytestmark = pytest.mark.gpu
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def codes_of(v, s, rows):
    """Codes of the quotients: one division, rounded to fp32, and one rounding to nearest even."""
    i, j = R.blocks_of(v, rows)
    return (v.float() / s[i, j]).to(R.F8).view(torch.uint8)


def same_codes(codes, scales, v, rows=1):
    assert torch.equal(scales.cpu(), R.scales(v.float(), rows).float())  # (max / 448 in 64 bits rounded once, and in 32)
    assert torch.equal(codes.cpu().view(torch.uint8), codes_of(v, scales.cpu(), rows))


# 16-bit inputs give quotients that are exact ties, or round to one, about once in 2000 (fp16 less often, fp32 hardly ever).
@pytest.mark.parametrize("x", [BF16, F16, F32])
@pytest.mark.parametrize("rows", [1, 128])
@pytest.mark.parametrize("size", [1.0, 2e-4, 300.0])
def test_codes_are_the_quotients(x, rows, size):
    g = torch.Generator().manual_seed(11)
    v = (size * torch.randn(260, 2064, generator=g)).to(x)
    codes, scales = q.moe_quantize_fp8(v.cuda(), block_rows=rows)
    same_codes(codes, scales, v, rows)


@pytest.mark.parametrize("rows", [1, 128])
@pytest.mark.parametrize("size", [1e-36, 1e-34, 1e-30, 1e30, 1e37])
def test_codes_of_small_and_large_blocks(rows, size):
    """Blocks down to where the scale is the least there is, and to fp32's largest numbers."""
    g = torch.Generator().manual_seed(12)
    for x in (BF16, F32):
        v = (size * torch.randn(130, 1040, generator=g)).to(x)
        codes, scales = q.moe_quantize_fp8(v.cuda(), block_rows=rows)
        same_codes(codes, scales, v, rows)


def test_every_tie_goes_to_the_even_code():
    """Blocks whose scale is 3 x 2^-9: the codes' midpoints times it are exact in fp32."""
    mids = torch.cat([(16 + 2 * torch.arange(8) + 1) / 16 * 2.0 ** e for e in range(-6, 8)] + [(2 * torch.arange(8) + 1) * 2.0 ** -10])
    v = torch.zeros(mids.numel(), 128)
    v[:, 0] = 448.0
    v[:, 1], v[:, 2] = mids, -mids
    v = v * (3 * 2.0 ** -9)
    codes, scales = q.moe_quantize_fp8(v.cuda())
    assert (scales.cpu() == 3 * 2.0 ** -9).all()
    same_codes(codes, scales, v)
    assert (codes.cpu().view(torch.uint8)[:, 1:3] % 2 == 0).all()


@pytest.mark.parametrize("T,H", [(40, 96), (40, 500), (700, 2050), (5, 6144), (600, 4096), (3, 16384)])
def test_norm_s_codes_are_the_quotients(T, H):
    """The codes of y in fp32, which the fp32 output has."""
    g = torch.Generator().manual_seed(T + H)
    x, r = torch.randn(T, H, generator=g).to(BF16).cuda(), torch.randn(T, H, generator=g).to(BF16).cuda()
    w = (1 + torch.randn(H, generator=g) / 8).to(BF16).cuda()
    y, _ = q.moe_rms_norm(x, w, residual=r, out_dtype=F32)
    codes, scales, _ = q.moe_rms_norm_fp8(x, w, residual=r)
    same_codes(codes, scales, y.cpu())


def test_values_beside_an_infinity():
    v = torch.ones(2, 256)
    v[0, 5] = float("inf")
    v[1, 200] = float("-inf")
    codes, scales = q.moe_quantize_fp8(v.cuda())
    c, s = codes.cpu().float(), scales.cpu()
    assert torch.isnan(c[0, 5]) and torch.isnan(c[1, 200]) and torch.isinf(s[0, 0]) and torch.isinf(s[1, 1])
    c[0, 5] = c[1, 200] = 0
    assert (c[0, :128] == 0).all() and (c[1, 128:] == 0).all() and (c[0, 128:] == 448).all() and (c[1, :128] == 448).all()


# Rows of every launch shape: several a workgroup, one after another, and a last round that is not full.
@pytest.mark.parametrize("T,H", [(20011, 100), (70000, 16), (9001, 500), (3000, 1030), (2500, 4090), (1500, 4104), (600, 9001)])
@pytest.mark.parametrize("where", ["last", "first", "spread"])
def test_weight_gradient_of_a_few_rows(T, H, where):
    """dy is 0 but in a few rows, so dw is a sum of that many terms and its bound theirs: a lost row shows."""
    g = torch.Generator().manual_seed(T + H)
    rows = {"last": range(T - 4, T), "first": range(4), "spread": [0, T // 3, T // 2, T - 299, T - 17, T - 16, T - 2, T - 1]}[where]
    rows = torch.tensor(list(rows))
    r, w = torch.randn(T, H, generator=g), torch.randn(H, generator=g)
    dy = torch.zeros(T, H)
    dy[rows] = 2.0 ** torch.arange(len(rows)).float().unsqueeze(1) * (1 + torch.rand(len(rows), H, generator=g))
    _, dw = q.moe_rms_norm_backward(r.cuda(), w.cuda(), dy.cuda())
    _, _, ref, bound = R.norm_backward(r[rows], w, dy[rows], None, 1e-6, rounds=len(rows))
    R.check(dw, ref, bound)
    for i in range(len(rows)):  # the check finds each row's loss
        rest = torch.cat((rows[:i], rows[i + 1:]))
        lost = R.norm_backward(r[rest], w, dy[rest], None, 1e-6)[2]
        assert ((lost - ref).abs() > bound + R.U * (ref.abs() + bound)).double().mean() > 0.9
