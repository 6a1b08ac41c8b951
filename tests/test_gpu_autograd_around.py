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
