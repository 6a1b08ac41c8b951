"""Dense 4-bit products whose scales, biases or activations span a wide range,
on both sides of the rule that gives a call to the few tokens' or the many
tokens' kernel (needs an MI355X).

The bound is operator_refs.linear_reference's: fp32 sums of exact products,
relative to the magnitudes that meet.  Where the large scales meet zeros of x
(or the large x zeros of the weights) these magnitudes are the small ones', so
nothing may be lost beside a row's or a token's largest value."""

import numpy as np
import pytest
import torch

import quantized_expert_gather_amd as q
from tests import operator_refs as R

pytestmark = pytest.mark.gpu

AFFINE = ["affine4_g64", "affine4_g32"]
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
# affine sizes that are past the rule (many groups; split K) and one short input
AFFINE_TILES = [(1500, 1400, 256), (300, 110, 16448), (40, 50, 64)]


def by_tiles(codec, L, N, K):
    """Whether an affine call goes to the many tokens' kernel, by the room for its copy of the tokens."""
    return q.moe_linear_codec_workspace_bytes(codec, L, N, K) >= 2 * L * K


def forward(codec, x, w, s, b, ot=F32, bias=None):
    return q.moe_linear_codec_forward(codec, x.cuda(), w[0].cuda(), s[0].cuda(), None if b is None else b[0].cuda(),
                                      bias=bias, out_dtype=ot)


def check(out, ref, bound, dtype=F32):
    got = out.double().cpu().numpy()
    lim = bound + R.HALF_STEP[dtype] * (np.abs(ref) + bound) + R.HALF_TINY[dtype]
    bad = ~(np.abs(got - ref) <= lim)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4].tolist(), got[bad][:4], ref[bad][:4])


def activations(L, K, dtype, seed=7):
    return torch.randn(L, K, generator=torch.Generator().manual_seed(seed)).to(dtype)


# ---- mxfp4 with fp16 tokens: block exponents far apart in one row ----

@pytest.mark.parametrize("xt", [F16, BF16])
@pytest.mark.parametrize("L,N,K", [(16, 48, 256), (17, 48, 256), (300, 300, 4160), (200, 131, 288)])
def test_mxfp4_blocks_far_below_their_rows_largest(xt, L, N, K):
    print("[case] mxfp4 blocks far apart", xt, L, N, K, flush=True)
    w, s, _ = R.linear_weights("mxfp4", N, K, 31)
    x = activations(L, K, xt)
    x[:, :32] = 0                       # nothing meets the large block
    for i, d in enumerate((30, 34, 35, 36, 37, 40, 48, 60, 100)):
        s[0, i, :] = 120
        s[0, i, 0] = 120 + d
        s[0, i + 9, 1:] = 120           # the small block in the middle
        s[0, i + 9, 2] = 120 - d
    s[0, 20, 0], s[0, 20, 3], s[0, 20, 4] = 200, 150, 110
    s[0, 21, 1:] = 0                    # 2^-127 under zero codes, as for a block of zeros
    w[0, 21, 4:] = 0
    s[0, 22, 5] = 0
    w[0, 22, 20:24] = int(np.uint32(0x88888888).view(np.int32))  # and minus zeros
    ref, bound = R.linear_reference("mxfp4", x, w, s, None, None)
    check(forward("mxfp4", x, w, s, None), ref, bound + K * 2.0 ** -126)


def test_mxfp4_large_block_meets_some_tokens_only():
    L, N, K = 150, 70, 512
    w, s, _ = R.linear_weights("mxfp4", N, K, 32)
    x = activations(L, K, F16)
    x[::2, :32] = 0
    s[0, 3, 0] = 180
    s[0, 3, 1:] = 121
    s[0, 69, 0] = 171
    s[0, 69, 7] = 255                   # a NaN beside it stays its row's
    ref, bound = R.linear_reference("mxfp4", x, w, s, None, None)
    out = forward("mxfp4", x, w, s, None)
    assert torch.isnan(out[:, 69]).all()
    check(out[:, :69], ref[:, :69], bound[:, :69])


# ---- affine: scales far below the biases, and far apart in a row ----

@pytest.mark.parametrize("codec", AFFINE)
@pytest.mark.parametrize("xt", [BF16, F16])
@pytest.mark.parametrize("L,N,K", AFFINE_TILES + [(5, 50, 256)])
def test_affine_scales_far_below_the_biases(codec, xt, L, N, K):
    print("[case] affine scales far below biases", codec, xt, L, N, K, flush=True)
    assert by_tiles(codec, L, N, K) == (L > 5)
    w, s, b = R.linear_weights(codec, N, K, 33)
    x = activations(L, K, xt)
    g = torch.Generator().manual_seed(3)
    rb = torch.randn(b[0].shape, generator=g)
    for i, e in enumerate((-126, -120, -110, -100, -90, -70, -60, -50, -40, -24)):
        s[0, i] = 2.0 ** e              # a row of constants whose scale was kept from being zero
        b[0, i] = rb[i].to(BF16)
    s[0, 10] = 0.0
    b[0, 10] = rb[10].to(BF16)
    s[0, 11] = 0.0
    b[0, 11] = (rb[11] * 2.0 ** 75).to(BF16)
    b[0, 12] = (rb[12] * 2.0 ** 80).to(BF16)
    s[0, 13] = 2.0 ** -100
    b[0, 13] = (rb[13] * 2.0 ** -20).to(BF16)
    ref, bound = R.linear_reference(codec, x, w, s, b, None)
    check(forward(codec, x, w, s, b), ref, bound + K * 2.0 ** -126)


@pytest.mark.parametrize("codec", AFFINE)
@pytest.mark.parametrize("xt", [BF16, F16])
@pytest.mark.parametrize("L,N,K", AFFINE_TILES[:2] + [(16, 50, 256)])
def test_affine_scales_far_below_their_rows_largest(codec, xt, L, N, K):
    print("[case] affine scales far apart", codec, xt, L, N, K, flush=True)
    assert by_tiles(codec, L, N, K) == (L > 16)
    w, s, b = R.linear_weights(codec, N, K, 34)
    gs = R.GROUPS[codec]
    x = activations(L, K, xt)
    x[:, :gs] = 0                       # nothing meets the large scale
    for i, d in enumerate(range(20, 40)):
        s[0, i, 1:] = (s[0, i, 1:].float() * 2.0 ** -d).to(BF16)
        b[0, i, 1:] = (b[0, i, 1:].float() * 2.0 ** -d).to(BF16)
    s[0, 20, 2] = 2.0 ** -126
    b[0, 20, 2] = 0.0
    ref, bound = R.linear_reference(codec, x, w, s, b, None)
    check(forward(codec, x, w, s, b), ref, bound + K * 2.0 ** -126)


@pytest.mark.parametrize("codec", AFFINE)
@pytest.mark.parametrize("L,N,K", AFFINE_TILES[:2] + [(16, 50, 256)])
def test_bf16_activations_far_below_their_tokens_largest(codec, L, N, K):
    print("[case] tokens far apart", codec, L, N, K, flush=True)
    assert by_tiles(codec, L, N, K) == (L > 16)
    w, s, b = R.linear_weights(codec, N, K, 35)
    gs = R.GROUPS[codec]
    x = activations(L, K, BF16)
    for i, d in enumerate(range(22, 46)):
        t = i % L
        x[t, :gs] = (x[t, :gs].float() * 2.0 ** d).to(BF16)
    s[0, ::2, 0] = 0.0                  # half of the rows do not look at the large ones
    b[0, ::2, 0] = 0.0
    s[0, 4, 0] = s[0, 4, 1] * 2.0 ** -20
    b[0, 4, 0] = b[0, 4, 1] * 2.0 ** -20
    ref, bound = R.linear_reference(codec, x, w, s, b, None)
    check(forward(codec, x, w, s, b), ref, bound)


@pytest.mark.parametrize("codec", AFFINE)
@pytest.mark.parametrize("xt", [BF16, F16])
@pytest.mark.parametrize("ot", [BF16, F16, F32])
@pytest.mark.parametrize("L", [9, 40])
def test_group_sums_count_in_full(codec, xt, ot, L):
    # codes and biases of 0: every weight is 0 and so is the result.  The sum of a group's x, 985089, takes three bf16
    # terms; every partial sum is a whole number of at most 8 * 985089 < 2^24, exact in fp32.
    N, K = 20, 64
    w = torch.zeros(1, N, K // 8, dtype=torch.int32)
    s, b = torch.ones(1, N, K // R.GROUPS[codec], dtype=BF16), torch.zeros(1, N, K // R.GROUPS[codec], dtype=BF16)
    x = torch.zeros(L, K)
    x[:, :30] = 32768.0
    x[:, 30], x[:, 31] = 2048.0, 1.0
    out = forward(codec, x.to(xt), w, s, b, ot=ot)
    assert (out == 0).all(), out.unique()
