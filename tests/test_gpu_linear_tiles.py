"""Affine products that are sure to go to the many tokens' kernel: types,
alignments, biases, replays, and its way for tiles of wide rows (needs an
MI355X).  Every case asserts that the rule sends it there."""

import numpy as np
import pytest
import torch

import quantized_expert_gather_amd as q
from tests import operator_refs as R
from tests.test_gpu_linear import check, problem
from tests.test_gpu_linear_range import by_tiles

pytestmark = pytest.mark.gpu

AFFINE = ["affine4_g64", "affine4_g32"]
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
SIZES = [(1500, 1400, 256), (300, 110, 16448)]  # many groups of tokens; K split


def on_device(m):
    return [None if t is None else t[0].cuda() for t in m]


@pytest.mark.parametrize("codec", AFFINE)
@pytest.mark.parametrize("L,N,K", SIZES)
@pytest.mark.parametrize("xt", [BF16, F16])
@pytest.mark.parametrize("ot", [BF16, F16, F32])
def test_types(codec, L, N, K, xt, ot):
    assert by_tiles(codec, L, N, K)
    x, w, s, b, bias = problem(codec, L, N, K, xt, True)
    ref, bound = R.linear_reference(codec, x, w, s, b, bias)
    check(q.moe_linear_codec_forward(codec, x.cuda(), *on_device((w, s, b)), bias=bias.cuda(), out_dtype=ot), ref, bound, L, N, ot)


@pytest.mark.parametrize("codec", AFFINE)
@pytest.mark.parametrize("L,N,K", SIZES)
@pytest.mark.parametrize("ot", [BF16, F16, F32])
def test_biases_far_above_the_scales(codec, L, N, K, ot):
    assert by_tiles(codec, L, N, K)
    x, w, s, b, _ = problem(codec, L, N, K, BF16, False)
    b = torch.randn(b.shape, generator=torch.Generator().manual_seed(3)).to(BF16)
    s = s / 64
    ref, bound = R.linear_reference(codec, x, w, s, b, None)
    check(q.moe_linear_codec_forward(codec, x.cuda(), *on_device((w, s, b)), out_dtype=ot), ref, bound, L, N, ot)


@pytest.mark.parametrize("codec", AFFINE)
@pytest.mark.parametrize("skip_s,skip_b", [(1, 1), (1, 0), (0, 1), (4, 6)])
@pytest.mark.parametrize("L,N,K", [(1500, 1201, 320), (300, 110, 16448)])
def test_unaligned_scale_arrays(codec, skip_s, skip_b, L, N, K):
    assert by_tiles(codec, L, N, K)
    x, w, s, b, _ = problem(codec, L, N, K, BF16, False)
    ref, bound = R.linear_reference(codec, x, w, s, b, None)

    def shifted(t, skip):
        room = torch.full((t.numel() + skip + 9,), float("nan"), dtype=t.dtype, device="cuda")
        room[skip:skip + t.numel()] = t.flatten().cuda()
        return room[skip:skip + t.numel()].view(t.shape[1:])
    out = q.moe_linear_codec_forward(codec, x.cuda(), w[0].cuda(), shifted(s, skip_s), shifted(b, skip_b), out_dtype=F32)
    check(out, ref, bound, L, N, F32)


@pytest.mark.parametrize("codec", AFFINE)
def test_small_fp16_activations(codec):
    L, N, K = 1500, 1400, 256
    assert by_tiles(codec, L, N, K)
    x, w, s, b, _ = problem(codec, L, N, K, F16, False)
    x = (x.float() * 2.0 ** -17).to(F16)  # subnormal numbers
    ref, bound = R.linear_reference(codec, x, w, s, b, None)
    check(q.moe_linear_codec_forward(codec, x.cuda(), *on_device((w, s, b)), out_dtype=F32), ref, bound, L, N, F32)


@pytest.mark.parametrize("codec", AFFINE)
@pytest.mark.parametrize("L,N,K", SIZES)
def test_runs_prepared_calls_and_graphs(codec, L, N, K):
    assert by_tiles(codec, L, N, K)
    x, w, s, b, bias = problem(codec, L, N, K, BF16, True)
    a = [x.cuda(), *on_device((w, s, b))]
    kw = dict(bias=bias.cuda())
    first = q.moe_linear_codec_forward(codec, *a, **kw)
    assert torch.equal(first, q.moe_linear_codec_forward(codec, *a, **kw))
    calls = [q.PreparedLinear(codec, *a, **kw, stream=torch.cuda.Stream()) for _ in range(2)]
    graphs = []
    torch.cuda.synchronize()
    for c in calls:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=c._keep[-1]):
            c()
        graphs.append(g)
    for rep in range(3):
        for c in calls:
            c.out.fill_(float("nan"))
        torch.cuda.synchronize()
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(c.out, first) for c in calls), rep
        assert torch.equal(first, q.moe_linear_codec_forward(codec, *a, **kw))


def wide(codec, L, N, K, xt):
    """A product in which every tile has a row that is wide, with x zero where the large scales are."""
    x, w, s, b, _ = problem(codec, L, N, K, xt, False)
    gs = R.GROUPS[codec]
    x[:, :gs] = 0
    if codec == "mxfp4":
        s[0, ::7, 0] = 170
    else:
        s[0, ::7, 1:] = (s[0, ::7, 1:].float() * 2.0 ** -40).to(BF16)
        b[0, ::7, 1:] = (b[0, ::7, 1:].float() * 2.0 ** -40).to(BF16)
    return x, w, s, b


# short last steps of K, ends of the tokens and of the rows inside a tile, K split
@pytest.mark.parametrize("codec,xt,L,N,K", [(c, t, *z) for c in AFFINE for t in (BF16, F16) for z in
                                            ((1501, 1403, 320), (20, 70, 64), (300, 110, 16448), (800, 1203, 576))] +
                         [(c, BF16, *z) for c in ("affine4_g32",) for z in ((1501, 1403, 352), (40, 77, 96), (333, 45, 32))] +
                         [("mxfp4", F16, *z) for z in ((1501, 1403, 352), (40, 77, 96), (333, 45, 32), (300, 700, 4160))])
def test_wide_rows_with_strides(codec, xt, L, N, K):
    print("[case] wide rows", codec, xt, L, N, K, flush=True)
    assert codec == "mxfp4" or by_tiles(codec, L, N, K)
    if K == 32 or (codec == "affine4_g64" and K == 64):
        x, w, s, b, _ = problem(codec, L, N, K, xt, False)  # one group: nothing is wide
    else:
        x, w, s, b = wide(codec, L, N, K, xt)
    ref, bound = R.linear_reference(codec, x, w, s, b, None)
    room_x = torch.full((L, K + 24), float("nan"), dtype=xt, device="cuda")
    room_x[:, 8:8 + K] = x.cuda()
    room = torch.full((L + 2, N + 9), 7.0, device="cuda")
    out = room[1:L + 1, 4:4 + N]
    a = (room_x[:, 8:8 + K], *on_device((w, s, b)))
    q.moe_linear_codec_forward(codec, *a, out=out)
    check(out, ref, bound, L, N, F32)
    first = out.clone()
    assert torch.equal(q.moe_linear_codec_forward(codec, *a, out_dtype=F32), first)
    room[1:L + 1, 4:4 + N] = 7.0
    assert (room == 7.0).all()


@pytest.mark.parametrize("codec,L,N,K", [("affine4_g64", 1500, 1400, 256), ("affine4_g32", 1500, 1400, 256), ("mxfp4", 200, 300, 512)])
def test_wide_rows_keep_bad_tokens_and_rows_apart(codec, L, N, K):
    x, w, s, b = wide(codec, L, N, K, F16)
    clean = q.moe_linear_codec_forward(codec, x.cuda(), *on_device((w, s, b)), out_dtype=F32)
    ref, bound = R.linear_reference(codec, x, w, s, b, None)
    check(clean, ref, bound, L, N, F32)
    x[1, 70], x[2, 200], x[L - 1, K - 1] = float("nan"), float("inf"), float("-inf")
    s[0, 17, 2] = 255 if codec == "mxfp4" else float("nan")
    out = q.moe_linear_codec_forward(codec, x.cuda(), *on_device((w, s, b)), out_dtype=F32)
    rows, cols = [1, 2, L - 1], [17]
    assert not torch.isfinite(out[rows]).any() and not torch.isfinite(out[:, cols]).any()
    keep_r = torch.tensor(np.setdiff1d(np.arange(L), rows), device="cuda")
    keep_c = torch.tensor(np.setdiff1d(np.arange(N), cols), device="cuda")
    assert torch.equal(out[keep_r][:, keep_c], clean[keep_r][:, keep_c])


def test_wide_rows_in_a_graph():
    codec, L, N, K = "affine4_g32", 1500, 1400, 256
    x, w, s, b = wide(codec, L, N, K, BF16)
    a = [x.cuda(), *on_device((w, s, b))]
    first = q.moe_linear_codec_forward(codec, *a, out_dtype=F32)
    side = torch.cuda.Stream()
    p = q.PreparedLinear(codec, *a, out_dtype=F32, stream=side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        p()
    for rep in range(3):
        p.out.fill_(float("nan"))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(p.out, first), rep
        assert torch.equal(q.moe_linear_codec_forward(codec, *a, out_dtype=F32), first)


def test_activations_of_a_wide_token_and_uneven_rows_with_strides():
    # the two marks that send a tile the wide rows' way only together
    codec, L, N, K = "affine4_g64", 1501, 1403, 320
    for uneven in (False, True):
        x, w, s, b, _ = problem(codec, L, N, K, BF16, False)
        x[::50, :64] = (x[::50, :64].float() * 2.0 ** 40).to(BF16)
        if uneven:
            s[0, ::5, 0] = 0.0
            b[0, ::5, 0] = 0.0
        ref, bound = R.linear_reference(codec, x, w, s, b, None)
        room_x = torch.full((L, K + 24), float("nan"), dtype=BF16, device="cuda")
        room_x[:, 8:8 + K] = x.cuda()
        out = q.moe_linear_codec_forward(codec, room_x[:, 8:8 + K], *on_device((w, s, b)), out_dtype=F32)
        check(out, ref, bound, L, N, F32)
