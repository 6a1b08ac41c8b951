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
