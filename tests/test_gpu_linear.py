"""The dense 4-bit product on the GPU against 64-bit references (needs an
MI355X).  The bounds are derived in operator_refs.linear_reference; rounding
to the output type adds half a step."""

import numpy as np
import pytest
import torch

import quantized_expert_gather_amd as q
from tests import operator_refs as R

pytestmark = pytest.mark.gpu

CODECS = ["affine4_g64", "affine4_g32", "mxfp4", "nvfp4"]
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def problem(codec, L, N, K, xt, bias, seed=1):
    w, s, b = R.linear_weights(codec, N, K, seed)
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(L, K, generator=g).to(xt)
    bv = torch.randn(N, generator=g) if bias else None
    return x, w, s, b, bv


def dev(t):
    return None if t is None else t.cuda()


def check(out, ref, bound, L, N, dtype):
    got = out.double().cpu().numpy()
    lim = bound + R.HALF_STEP[dtype] * (np.abs(ref) + bound) + R.HALF_TINY[dtype]
    bad = ~(np.abs(got - ref) <= lim)
    assert not bad.any(), (int(bad.sum()), float(np.nanmax(np.abs(got - ref) / lim)))


def run(codec, L, N, K, xt, ot, bias=False, seed=1):
    print("[case] linear", codec, L, N, K, xt, ot, bias, flush=True)
    x, w, s, b, bv = problem(codec, L, N, K, xt, bias, seed)
    ref, bound = R.linear_reference(codec, x, w, s, b, bv)
    out = q.moe_linear_codec_forward(codec, dev(x), dev(w[0]), dev(s[0]), dev(b[0]) if b is not None else None, bias=dev(bv),
                                     out_dtype=ot)
    torch.cuda.synchronize()
    assert out.shape == (L, N) and out.dtype == ot
    check(out, ref, bound, L, N, ot)


@pytest.mark.parametrize("codec", CODECS)
@pytest.mark.parametrize("L,N,K", [(1, 1, 64), (1, 16, 64), (2, 17, 128), (3, 33, 192), (1, 250, 1024), (5, 100, 2112),
                                   (16, 64, 4096), (1, 48, 6144), (9, 31, 8256), (4, 20, 16448), (15, 4099, 320)])
def test_few_tokens(codec, L, N, K):
    run(codec, L, N, K, BF16 if N % 2 else F16, F32, bias=N % 3 == 0)


@pytest.mark.parametrize("codec", ["affine4_g32", "mxfp4", "nvfp4"])
@pytest.mark.parametrize("L,N,K", [(1, 3, 32), (2, 18, 96), (7, 50, 160), (3, 40, 4128), (40, 70, 224), (130, 200, 1056)])
def test_inputs_that_end_inside_a_step(codec, L, N, K):
    run(codec, L, N, K, BF16, F32)
    run(codec, L, N, K, F16, F16)


@pytest.mark.parametrize("codec", CODECS)
@pytest.mark.parametrize("L,N,K", [(17, 64, 256), (32, 129, 512), (33, 16, 1024), (64, 257, 4160), (96, 2050, 2048),
                                   (100, 1, 640), (127, 128, 128), (129, 130, 1024), (300, 515, 1088), (513, 384, 2048),
                                   (1000, 256, 64)])
def test_many_tokens(codec, L, N, K):
    run(codec, L, N, K, F16 if N % 2 else BF16, F32, bias=N % 2 == 0)


@pytest.mark.parametrize("codec", CODECS)
@pytest.mark.parametrize("L,N,K", [(20, 16500, 64), (40, 33000, 128), (64, 16401, 192), (150, 8200, 320), (260, 5003, 448)])
def test_many_tokens_and_many_outputs(codec, L, N, K):
    run(codec, L, N, K, BF16 if N % 2 else F16, F16 if N % 2 else F32, bias=True)


@pytest.mark.parametrize("codec", CODECS)
@pytest.mark.parametrize("xt", [BF16, F16])
@pytest.mark.parametrize("L,N,K", [(1, 40, 384), (4, 3000, 320), (16, 70, 448), (3, 100, 2240), (9, 50, 4160), (2, 33, 6208),
                                   (6, 20, 8256)])
def test_few_tokens_of_long_and_odd_inputs(codec, xt, L, N, K):
    run(codec, L, N, K, xt, F32)


@pytest.mark.parametrize("codec", CODECS)
@pytest.mark.parametrize("L,K", [(2, 4224), (7, 6144), (3, 8320)])
def test_unaligned_scale_rows_of_long_inputs(codec, L, K):
    x, w, s, b, _ = problem(codec, L, 21, K, BF16, False)
    ref, bound = R.linear_reference(codec, x, w, s, b, None)

    def shifted(t):
        if t is None:
            return None
        skip = 2 if codec == "nvfp4" else 1
        room = torch.zeros(t.numel() + skip, dtype=t.dtype, device="cuda")
        room[skip:] = t.flatten().cuda()
        return room[skip:].view(t.shape[1:])
    out = q.moe_linear_codec_forward(codec, x.cuda(), w[0].cuda(), shifted(s), shifted(b), out_dtype=F32)
    check(out, ref, bound, L, 21, F32)


@pytest.mark.parametrize("codec", CODECS)
@pytest.mark.parametrize("xt", [BF16, F16])
@pytest.mark.parametrize("ot", [BF16, F16, F32])
def test_types(codec, xt, ot):
    for L in (1, 6, 50, 200):
        run(codec, L, 72, 512, xt, ot, bias=True)


@pytest.mark.parametrize("codec", CODECS)
@pytest.mark.parametrize("L", [1, 4, 16, 40, 200])
def test_strided_rows_and_untouched_surroundings(codec, L):
    N, K = 75, 320
    x, w, s, b, _ = problem(codec, L, N, K, BF16, False)
    ref, bound = R.linear_reference(codec, x, w, s, b, None)
    wide = torch.full((L, K + 24), float("nan"), dtype=BF16, device="cuda")
    wide[:, 8:8 + K] = x.cuda()
    room = torch.full((L + 2, N + 9), 7.0, device="cuda")
    out = room[1:L + 1, 4:4 + N]
    got = q.moe_linear_codec_forward(codec, wide[:, 8:8 + K], w[0].cuda(), s[0].cuda(), dev(b[0]) if b is not None else None,
                                     out=out)
    assert got is out
    check(out, ref, bound, L, N, F32)
    room[1:L + 1, 4:4 + N] = 7.0
    assert (room == 7.0).all()


@pytest.mark.parametrize("codec", CODECS)
@pytest.mark.parametrize("L", [1, 20, 150])
def test_scales_at_the_ends_of_their_range(codec, L):
    N, K = 40, 256
    x, w, s, b, _ = problem(codec, L, N, K, BF16, False)
    if codec.startswith("affine"):
        s[0, 1] = 0.0
        s[0, 2, ::2] = -s[0, 2, ::2]
        s[0, 3] *= 2.0 ** -90
        b[0, 3] *= 2.0 ** -90
        s[0, 4] *= 2.0 ** 90
        b[0, 4] *= 2.0 ** 90
    elif codec == "mxfp4":
        s[0, 1] = 0      # 2^-127
        s[0, 2] = 240
        s[0, 3, 1] = 1
    else:
        s[0, 1] = 0      # a scale of zero
        s[0, 2] = 1      # the smallest subnormal
        s[0, 3] = 0x7E   # 448
        s[0, 4] = 0xB8   # negative
    ref, bound = R.linear_reference(codec, x, w, s, b, None)
    out = q.moe_linear_codec_forward(codec, x.cuda(), w[0].cuda(), s[0].cuda(), dev(b[0]) if b is not None else None,
                                     out_dtype=F32)
    # products of a 2^-127 block lie below fp32's smallest normal number: each may round to it or to zero
    got = out.double().cpu().numpy()
    assert (np.abs(got - ref) <= bound + R.HALF_STEP[F32] * np.abs(ref) + K * 2.0 ** -126).all()


@pytest.mark.parametrize("codec", ["affine4_g64", "affine4_g32"])
@pytest.mark.parametrize("L", [2, 9, 40, 200])
@pytest.mark.parametrize("ot", [F16, F32])
def test_biases_far_above_the_scales(codec, L, ot):
    x, w, s, b, _ = problem(codec, L, 70, 256, BF16, False)
    g = torch.Generator().manual_seed(3)
    b = torch.randn(b.shape, generator=g).to(BF16)
    s = s / 64
    ref, bound = R.linear_reference(codec, x, w, s, b, None)
    out = q.moe_linear_codec_forward(codec, x.cuda(), w[0].cuda(), s[0].cuda(), b[0].cuda(), out_dtype=ot)
    check(out, ref, bound, L, 70, ot)


@pytest.mark.parametrize("codec,nan", [("mxfp4", 255), ("nvfp4", 0x7F)])
@pytest.mark.parametrize("L", [1, 20, 150])
def test_nan_scales_reach_their_row_only(codec, nan, L):
    N, K = 35, 320
    x, w, s, b, _ = problem(codec, L, N, K, BF16, False)
    s[0, 5, 1] = nan
    s[0, 34, -1] = nan
    out = q.moe_linear_codec_forward(codec, x.cuda(), w[0].cuda(), s[0].cuda(), out_dtype=F32).cpu()
    rows = torch.isnan(out).all(0)
    assert rows.nonzero().flatten().tolist() == [5, 34]
    assert torch.isfinite(out[:, ~rows]).all()


@pytest.mark.parametrize("codec", CODECS)
@pytest.mark.parametrize("L", [3, 40, 200])
def test_nan_activations_reach_their_token_only(codec, L):
    N, K = 50, 256
    x, w, s, b, _ = problem(codec, L, N, K, F16, False)
    x[1, 70] = float("nan")
    out = q.moe_linear_codec_forward(codec, x.cuda(), w[0].cuda(), s[0].cuda(), dev(b[0]) if b is not None else None).cpu()
    bad = torch.isnan(out).all(1)
    assert bad.nonzero().flatten().tolist() == [1]
    assert torch.isfinite(out[~bad]).all()


def test_small_fp16_values_are_not_flushed():
    # subnormal fp16 activations, and nvfp4 weights that are subnormal in fp16
    for codec in CODECS:
        for L in (2, 40):
            x, w, s, b, _ = problem(codec, L, 32, 128, F16, False)
            x = (x.float() * 2.0 ** -17).to(F16)
            ref, bound = R.linear_reference(codec, x, w, s, b, None)
            out = q.moe_linear_codec_forward(codec, x.cuda(), w[0].cuda(), s[0].cuda(), dev(b[0]) if b is not None else None,
                                             out_dtype=F32)
            check(out, ref, bound, L, 32, F32)


def test_unaligned_scale_rows():
    # scale arrays that start on odd 16-bit words (any byte for mxfp4)
    for codec in CODECS:
        for L in (2, 40, 200):
            x, w, s, b, _ = problem(codec, L, 33, 256, BF16, False)
            ref, bound = R.linear_reference(codec, x, w, s, b, None)

            def shifted(t):
                if t is None:
                    return None
                skip = 2 if codec == "nvfp4" else 1
                room = torch.zeros(t.numel() + skip, dtype=t.dtype, device="cuda")
                room[skip:] = t.flatten().cuda()
                return room[skip:].view(t.shape[1:])
            out = q.moe_linear_codec_forward(codec, x.cuda(), w[0].cuda(), shifted(s), shifted(b), out_dtype=F32)
            check(out, ref, bound, L, 33, F32)


def test_no_tokens():
    w, s, b = R.linear_weights("affine4_g64", 8, 64, 1)
    out = q.moe_linear_codec_forward("affine4_g64", torch.empty(0, 64, dtype=BF16, device="cuda"), w[0].cuda(), s[0].cuda(),
                                     b[0].cuda())
    assert out.shape == (0, 8)


@pytest.mark.parametrize("L", [1, 12, 64, 400])
def test_runs_are_equal_and_prepared_calls_match(L):
    x, w, s, b, bv = problem("affine4_g32", L, 300, 2048, BF16, True)
    a = [t.cuda() for t in (x, w[0], s[0], b[0])]
    one = q.moe_linear_codec_forward("affine4_g32", *a, bias=bv.cuda())
    two = q.moe_linear_codec_forward("affine4_g32", *a, bias=bv.cuda())
    p = q.PreparedLinear("affine4_g32", *a, bias=bv.cuda())
    three = p().clone()
    assert torch.equal(one, two) and torch.equal(one, three)
    a[0].mul_(2)
    four = p()
    assert torch.equal(four, q.moe_linear_codec_forward("affine4_g32", *a, bias=bv.cuda()))


@pytest.mark.parametrize("L", [2, 64, 300])
def test_other_streams(L):
    x, w, s, b, _ = problem("mxfp4", L, 500, 4096, BF16, False)
    a = [t.cuda() for t in (x, w[0], s[0])]
    ref = q.moe_linear_codec_forward("mxfp4", *a)
    torch.cuda.synchronize()
    sides = [torch.cuda.Stream() for _ in range(2)]
    outs = [q.moe_linear_codec_forward("mxfp4", *a, stream=sd) for sd in sides for _ in range(3)]
    outs.append(q.moe_linear_codec_forward("mxfp4", *a, stream=sides[0].cuda_stream))
    torch.cuda.synchronize()
    assert all(torch.equal(o, ref) for o in outs)


@pytest.mark.parametrize("L", [2, 40])
def test_a_streams_outputs_share_no_memory_with_pending_work(L):
    x, w, s, b, _ = problem("affine4_g64", L, 300, 512, BF16, False)
    a = [t.cuda() for t in (x, w[0], s[0], b[0])]
    ref = q.moe_linear_codec_forward("affine4_g64", *a)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for make in (lambda: q.moe_linear_codec_forward("affine4_g64", *a, stream=side),
                 lambda: q.PreparedLinear("affine4_g64", *a, stream=side)()):
        old = [torch.empty_like(ref) for _ in range(4)]
        torch.cuda._sleep(20_000_000)
        for t in old:
            t.fill_(float("nan"))  # still to come when the call below is made
        del old, t
        out = make()
        torch.cuda.synchronize()
        assert torch.equal(out, ref)


def test_a_stream_of_another_device_is_refused():
    x, w, s, b, _ = problem("mxfp4", 1, 16, 128, BF16, False)

    class Elsewhere(torch.cuda.Stream):
        device = torch.device("cuda", 1)
    with pytest.raises(ValueError, match="stream"):
        q.moe_linear_codec_forward("mxfp4", x.cuda(), w[0].cuda(), s[0].cuda(), stream=Elsewhere())


@pytest.mark.parametrize("codec", CODECS)
@pytest.mark.parametrize("L", [3, 12, 40, 200])
def test_infinite_activations_reach_their_token_only(codec, L):
    x, w, s, b, _ = problem(codec, L, 40, 256, BF16, False)
    x[1, 30] = float("inf")
    x[2, 200] = float("-inf")
    a = [t.cuda() for t in (w[0], s[0])] + [b[0].cuda() if b is not None else None]
    out = q.moe_linear_codec_forward(codec, x.cuda(), *a)
    bad = ~torch.isfinite(out).any(1)
    assert bad.nonzero().flatten().tolist() == [1, 2]
    x[1:3] = 0
    keep = [t for t in range(L) if t not in (1, 2)]
    assert torch.equal(out[keep], q.moe_linear_codec_forward(codec, x.cuda(), *a)[keep])


@pytest.mark.parametrize("L", [1, 48, 260])
def test_replays_in_graphs(L):
    x, w, s, b, _ = problem("affine4_g64", L, 200, 1024, BF16, False)
    a = [t.cuda() for t in (x, w[0], s[0], b[0])]
    calls = [q.PreparedLinear("affine4_g64", *a, stream=torch.cuda.Stream()) for _ in range(2)]
    graphs = []
    for c in calls:
        side = c._keep[-1]
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            c()
        graphs.append(g)
    for rep in range(3):
        for c in calls:
            c.out.fill_(float("nan"))
        a[0].mul_(-1)
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        want = q.moe_linear_codec_forward("affine4_g64", *a)
        torch.cuda.synchronize()
        assert all(torch.equal(c.out, want) for c in calls), rep
    # x was negated three times; the matrix cores' sums are not odd in their inputs to the last bit
    r64, bound = R.linear_reference("affine4_g64", -x, w, s, b, None)
    check(want, r64, bound, L, 200, BF16)


def test_more_codes_than_32_bits_of_bytes():
    # 65537 rows of 65536 inputs: the last rows' codes lie past 2^31 bytes
    N, K = 65537 + 16, 65536
    w = torch.zeros(N, K // 8, dtype=torch.int32, device="cuda")
    s = torch.full((N, K // 32), 127, dtype=torch.uint8, device="cuda")
    w[-3:] = 0x22222222   # E2M1 1.0
    w[0] = 0x22222222
    for L in (1, 40):
        x = torch.zeros(L, K, dtype=BF16, device="cuda")
        x[:, -100:] = 1.0
        out = q.moe_linear_codec_forward("mxfp4", x, w, s, out_dtype=F32)
        want = torch.zeros(L, N, device="cuda")
        want[:, -3:] = 100.0
        want[:, 0] = 100.0
        assert torch.equal(out, want)


# ---- affine products that are large enough for the tiles (small ones of any number of tokens take the few tokens' way) ----

AFFINE = ["affine4_g64", "affine4_g32"]


@pytest.mark.parametrize("codec", AFFINE)
@pytest.mark.parametrize("xt", [BF16, F16])
@pytest.mark.parametrize("L,N,K", [(17, 4099, 4160), (33, 2900, 4160), (50, 2100, 5184), (70, 1700, 4224), (130, 1000, 4160),
                                   (200, 701, 4160), (600, 250, 4160), (1500, 100, 4224), (129, 2003, 2112), (40, 6000, 2240),
                                   (300, 14, 131072)])
def test_affine_tiles(codec, xt, L, N, K):
    run(codec, L, N, K, xt, F32, bias=N % 3 == 0)


@pytest.mark.parametrize("codec", AFFINE)
@pytest.mark.parametrize("L,N", [(20, 66000), (60, 33003), (200, 10501)])
@pytest.mark.parametrize("ot", [BF16, F16])
def test_affine_tiles_of_short_inputs(codec, L, N, ot):
    run(codec, L, N, 256, ot, ot, bias=True)


@pytest.mark.parametrize("codec", AFFINE)
@pytest.mark.parametrize("ot", [F16, F32])
def test_affine_tiles_with_extreme_rows(codec, ot):
    L, N, K = 150, 13203, 256
    x, w, s, b, _ = problem(codec, L, N, K, BF16, False)
    s[0, 1] = 0.0
    s[0, 2, ::2] = -s[0, 2, ::2]
    if ot == F32:
        s[0, 3] *= 2.0 ** -90
        b[0, 3] *= 2.0 ** -90
        s[0, 4] *= 2.0 ** 90
        b[0, 4] *= 2.0 ** 90
        x[5] *= 2.0 ** 20
        x[6] *= 2.0 ** -60
    b[0, 7] = b[0, 7] * 64
    x[8] = 0
    ref, bound = R.linear_reference(codec, x, w, s, b, None)
    out = q.moe_linear_codec_forward(codec, x.cuda(), w[0].cuda(), s[0].cuda(), b[0].cuda(), out_dtype=ot)
    check(out, ref, bound + K * 2.0 ** -126, L, N, ot)


@pytest.mark.parametrize("codec", AFFINE)
@pytest.mark.parametrize("xt", [BF16, F16])
def test_affine_tiles_keep_bad_tokens_and_rows_apart(codec, xt):
    L, N, K = 150, 13203, 256
    x, w, s, b, _ = problem(codec, L, N, K, xt, False)
    x[1, 70] = float("nan")
    x[2, 3] = float("inf")
    x[149, 255] = float("-inf")
    s[0, 17, 1] = float("nan")
    b[0, 40, 0] = float("inf")
    out = q.moe_linear_codec_forward(codec, x.cuda(), w[0].cuda(), s[0].cuda(), b[0].cuda(), out_dtype=F32).cpu()
    rows, cols = [1, 2, 149], [17, 40]
    assert not torch.isfinite(out[rows]).any() and not torch.isfinite(out[:, cols]).any()
    x[rows] = 0
    s[0, 17, 1] = 1.0
    b[0, 40, 0] = 0.0
    ref, bound = R.linear_reference(codec, x, w, s, b, None)
    keep_r, keep_c = np.setdiff1d(np.arange(L), rows), np.setdiff1d(np.arange(N), cols)
    got = out.double().numpy()[np.ix_(keep_r, keep_c)]
    r, bd = ref[np.ix_(keep_r, keep_c)], bound[np.ix_(keep_r, keep_c)]
    assert (np.abs(got - r) <= bd + R.HALF_STEP[F32] * (np.abs(r) + bd)).all()


@pytest.mark.parametrize("codec", AFFINE)
def test_affine_tiles_strided_runs_and_replays(codec):
    L, N, K = 150, 13203, 256
    x, w, s, b, _ = problem(codec, L, N, K, BF16, False)
    ref, bound = R.linear_reference(codec, x, w, s, b, None)
    wide = torch.full((L, K + 24), float("nan"), dtype=BF16, device="cuda")
    wide[:, 8:8 + K] = x.cuda()
    room = torch.full((L + 2, N + 9), 7.0, device="cuda")
    out = room[1:L + 1, 4:4 + N]
    a = (wide[:, 8:8 + K], w[0].cuda(), s[0].cuda(), b[0].cuda())
    q.moe_linear_codec_forward(codec, *a, out=out)
    check(out, ref, bound, L, N, F32)
    first = out.clone()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    p = q.PreparedLinear(codec, *a, out=out, stream=side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        p()
    for _ in range(3):
        out.fill_(float("nan"))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, first)
        assert torch.equal(q.moe_linear_codec_forward(codec, *a, out_dtype=F32), first)
    room[1:L + 1, 4:4 + N] = 7.0
    assert (room == 7.0).all()
