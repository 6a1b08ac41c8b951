"""Autograd around the norm, the quantization, the 8-bit product and the gated
block: what they write into given tensors, and what carries a gradient (needs
an MI355X)."""

import pytest
import torch

import quantized_expert_gather_amd as q
from tests import around_refs as R

pytestmark = pytest.mark.gpu
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def rand(shape, dtype=BF16, seed=0):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


# ---- given tensors ----

def test_a_stream_that_was_saved_cannot_be_added_to_unnoticed():
    """The residual in place, behind a product that needs it for its weight's gradient."""
    x, r, w = rand((6, 64)), rand((6, 64), seed=1), rand((64, 8), seed=2).requires_grad_()
    y = r @ w
    q.moe_rms_norm(x, residual=r, total=r)
    with pytest.raises(RuntimeError, match="inplace"):
        y.sum().backward()
    # and the sum that a norm of its own saved
    x.requires_grad_()
    y, total = q.moe_rms_norm(x, residual=r)
    with torch.no_grad():
        q.moe_rms_norm_fp8(x, residual=total, total=total)
    with pytest.raises(RuntimeError, match="inplace"):
        y.sum().backward()


def test_given_outputs_count_as_written():
    x, r, w, dy = rand((6, 256)), rand((6, 256), seed=1), rand((256,), seed=2), rand((6, 256), seed=3)
    wg, wu, dh = rand((64, 256), seed=4), rand((64, 256), seed=5), rand((6, 64), seed=6)
    e = lambda *s, dtype=BF16: torch.zeros(*s, dtype=dtype, device="cuda")  # noqa: E731
    total, out, codes, scales = e(6, 256), e(6, 256), e(6, 256, dtype=torch.uint8).view(R.F8), e(6, 2, dtype=F32)
    dx, dw, h, saved = e(6, 256), e(256), e(6, 64), e(2, 6, 64, dtype=F32)
    gx, dwg, dwu, p = e(6, 256), e(64, 256), e(64, 256), e(6, 64)
    wc, ws = q.moe_quantize_fp8(wg, block_rows=128)
    inputs = (x, r, w, dy, wg, wu, dh, wc, ws)
    before = [t._version for t in inputs]

    def writes(call, *given):
        v = [t._version for t in given]
        call()
        assert [t._version for t in given] == [i + 1 for i in v]

    writes(lambda: q.moe_rms_norm(x, w, residual=r, total=total, out=out), total, out)
    writes(lambda: q.moe_rms_norm_fp8(x, w, residual=r, total=total, codes=codes, scales=scales), total, codes, scales)
    writes(lambda: q.moe_rms_norm_backward(total, w, dy, dx=dx, dweight=dw), dx, dw)
    writes(lambda: q.moe_quantize_fp8(x, codes=codes, scales=scales), codes, scales)
    writes(lambda: q.moe_linear_fp8_forward(codes, scales, wc, ws, out=p), p)
    writes(lambda: q.moe_glu(x, wg, wu, out=h, saved=saved), h, saved)
    writes(lambda: q.moe_glu_backward(x, wg, wu, dh, saved=saved, dx=gx, dwg=dwg, dwu=dwu), gx, dwg, dwu)
    writes(lambda: q.moe_rms_norm(x, w, out=out, stream=torch.cuda.current_stream()), out)
    view = e(6, 300)
    writes(lambda: q.moe_rms_norm(x, w, out=view[:, 4:260]), view)  # a view counts for what it views
    assert [t._version for t in inputs] == before
    with torch.inference_mode():
        q.moe_rms_norm(x, w, residual=r, total=total, out=e(6, 256))


# ---- the residual stream beside codes ----

@pytest.mark.parametrize("res", [BF16, F32])
@pytest.mark.parametrize("which", ["x", "residual", "both"])
def test_the_stream_beside_codes_carries_its_gradient(res, which):
    x, r, w, dt = rand((6, 200)), rand((6, 200), res, 1), rand((200,), seed=2).requires_grad_(), rand((6, 200), res, 3)
    plain = q.moe_rms_norm_fp8(x, w, residual=r)  # (the weight has none of the stream's gradient)
    assert not plain[2].requires_grad
    leaves = [t for t, n in ((x, "x"), (r, "residual")) if which in (n, "both")]
    for t in leaves:
        t.requires_grad_()
    codes, scales, total = q.moe_rms_norm_fp8(x, w, residual=r)
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip((codes, scales, total.detach()), plain))
    assert total.requires_grad and not codes.requires_grad and not scales.requires_grad
    (2 * total).backward(dt)
    for t in leaves:
        assert torch.equal(t.grad, (2 * dt).to(t.dtype))
    assert w.grad is None
    # given codes stay possible, a given total does not; without grad mode it does
    given = torch.zeros(6, 200, dtype=torch.uint8, device="cuda").view(R.F8)
    got = q.moe_rms_norm_fp8(x, w, residual=r, codes=given)
    assert got[0] is given and torch.equal(given.view(torch.uint8), codes.view(torch.uint8)) and got[2].requires_grad
    with pytest.raises(RuntimeError, match="gradient"):
        q.moe_rms_norm_fp8(x, w, residual=r, total=torch.empty_like(dt))
    with torch.no_grad():
        assert not q.moe_rms_norm_fp8(x, w, residual=r, total=torch.empty_like(dt))[2].requires_grad
    assert not q.moe_rms_norm_fp8(x, w)[0].requires_grad


def test_a_layer_around_a_frozen_8_bit_projection():
    """The stream's gradient past the projection, beside the norm's that follows it."""
    x, r, w = rand((5, 256)).requires_grad_(), rand((5, 256), seed=1).requires_grad_(), rand((256,), seed=2)
    wc, ws = q.moe_quantize_fp8(rand((256, 256), seed=3), block_rows=128)
    codes, scales, total = q.moe_rms_norm_fp8(x, w, residual=r)
    p = q.moe_linear_fp8_forward(codes, scales, wc, ws)
    y, _ = q.moe_rms_norm(p, w, residual=total)
    dy = rand((5, 256), seed=4)
    y.backward(dy)
    d, _ = q.moe_rms_norm_backward((p.float() + total.detach().float()).to(BF16), w, dy)
    assert torch.equal(x.grad, d) and torch.equal(r.grad, d)


# ---- arguments that are no tensors, behind the checks of those that are ----

def test_arguments_that_are_no_tensors():
    x, w, dy = rand((4, 256)), rand((256,), seed=1), rand((4, 256), seed=2)
    wg, dh = rand((64, 256), seed=3), rand((4, 64), seed=4)
    c, s = q.moe_quantize_fp8(x)
    wc, ws = q.moe_quantize_fp8(wg, block_rows=128)
    g = wg.clone().requires_grad_()
    for call in (lambda: q.moe_rms_norm(x, 3.0), lambda: q.moe_rms_norm(x, w, residual=[1.0]), lambda: q.moe_rms_norm(x, w, out=[1.0]),
                 lambda: q.moe_rms_norm(x, w, residual=x, total=5), lambda: q.moe_rms_norm_fp8(x, codes=[1], scales=s),
                 lambda: q.moe_rms_norm_fp8(x, scales=[1]), lambda: q.moe_rms_norm_backward(x, w, [1.0]),
                 lambda: q.moe_rms_norm_backward(x, w, dy, dtotal=[1.0]), lambda: q.moe_rms_norm_backward(x, w, dy, workspace=bytes(4096)),
                 lambda: q.moe_rms_norm_backward(x, w, dy, dx=3), lambda: q.moe_rms_norm_backward(x, w, dy, dweight=3),
                 lambda: q.moe_quantize_fp8(x, codes=[1]), lambda: q.moe_quantize_fp8(x, scales=[1]),
                 lambda: q.moe_linear_fp8_forward(c, [1], wc, ws), lambda: q.moe_linear_fp8_forward(c, s, wc, [1]),
                 lambda: q.moe_linear_fp8_forward(c, s, wc, ws, bias=[1.0]), lambda: q.moe_linear_fp8_forward(c, s, wc, ws, out=[1.0]),
                 lambda: q.moe_linear_fp8_forward(c, s, wc, ws, workspace=bytes(64)), lambda: q.moe_glu(x, [1.0], wg),
                 lambda: q.moe_glu(x, g, 3), lambda: q.moe_glu(x, [1.0], g), lambda: q.moe_glu(x, wg, wg, out=[1.0]),
                 lambda: q.moe_glu(x, wg, wg, saved=[1.0]), lambda: q.moe_glu(x, wg, wg, workspace=bytes(64)),
                 lambda: q.moe_glu_backward(x, wg, wg, [1.0]), lambda: q.moe_glu_backward(x, wg, wg, dh, dx=[1.0]),
                 lambda: q.moe_glu_backward(x, wg, wg, dh, dwg=[1.0]), lambda: q.moe_glu_backward(x, wg, wg, dh, workspace=bytes(1 << 20))):
        with pytest.raises(TypeError):
            call()


def test_backward_of_a_captured_stream_is_refused(monkeypatch):
    x, r = rand((4, 128)).requires_grad_(), rand((4, 128), seed=1)
    total = q.moe_rms_norm_fp8(x, residual=r)[2]
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
    with pytest.raises(RuntimeError, match="graph-captured"):
        total.backward(r)
