"""What the operators around the layer refuse of autograd, and what their
bindings say to arguments that are none (no GPU: every refusal comes first)."""

import pytest
import torch
import torch.autograd.forward_ad as fw

import quantized_expert_gather_amd as q

BF16 = torch.bfloat16


def calls(x, w, z):
    """Each differentiable result, with the named input in turn."""
    ids = torch.zeros(4, 2, dtype=torch.int32)
    wg = torch.zeros(8, 64, dtype=BF16)
    return {
        "norm x": (x, lambda t: q.moe_rms_norm(t, w)), "norm weight": (w, lambda t: q.moe_rms_norm(x, t)),
        "norm residual": (x, lambda t: q.moe_rms_norm(x, w, residual=t)), "norm stream": (x, lambda t: q.moe_rms_norm(t, w, out=x)),
        "codes x": (x, lambda t: q.moe_rms_norm_fp8(t, w, residual=x)), "codes residual": (x, lambda t: q.moe_rms_norm_fp8(x, w, residual=t)),
        "glu x": (x, lambda t: q.moe_glu(t, wg, wg)), "glu wg": (wg, lambda t: q.moe_glu(x, t, wg)),
        "glu wu": (wg, lambda t: q.moe_glu(x, wg, t)), "topk": (z, lambda t: q.moe_router_topk(t, 2)),
        "balance": (z, lambda t: q.moe_balance_loss(t, ids)),
    }


def arguments():
    return torch.zeros(4, 64, dtype=BF16), torch.ones(64), torch.zeros(4, 8)


@pytest.mark.parametrize("name", calls(*arguments()))
def test_forward_mode_is_refused(name):
    t, call = calls(*arguments())[name]
    with fw.dual_level():
        with pytest.raises(RuntimeError, match="forward-mode"):
            call(fw.make_dual(t, torch.ones_like(t)))
        with pytest.raises(ValueError, match="device"):  # without a tangent: the next check's
            call(t)


def test_arguments_that_are_no_tensors():
    x, w, z = arguments()
    g = torch.zeros(4, 64, dtype=BF16).requires_grad_()
    codes, s = torch.zeros(4, 64).to(torch.float8_e4m3fn), torch.zeros(4, 1)
    for call in (lambda: q.moe_rms_norm([1.0]), lambda: q.moe_rms_norm(None), lambda: q.moe_rms_norm([1.0], stream=0),
                 lambda: q.moe_rms_norm([1.0], w.clone().requires_grad_()), lambda: q.moe_rms_norm_fp8(3),
                 lambda: q.moe_rms_norm_backward([1.0], None, x), lambda: q.moe_quantize_fp8("x"),
                 lambda: q.moe_linear_fp8_forward([1], s, codes, s[:1]), lambda: q.moe_glu([1.0], x, x),
                 lambda: q.moe_glu(3, g, x), lambda: q.moe_glu_backward(None, x, x, x)):
        with pytest.raises(TypeError, match="must be a torch.Tensor"):
            call()
    for call in (lambda: q.moe_glu(g[0, 0], x, x), lambda: q.moe_glu(g, [1.0], x), lambda: q.moe_glu(g, x, None),
                 lambda: q.moe_rms_norm(x, out=[1.0]), lambda: q.moe_rms_norm(x, out=5, out_dtype=BF16)):
        with pytest.raises((TypeError, ValueError)):  # (x, on the host here, may be what is refused)
            call()
