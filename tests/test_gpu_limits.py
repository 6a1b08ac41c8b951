"""Calls whose rows or outputs need more threads than one launch holds, within
the documented limits (needs an MI355X)."""

import pytest
import torch

import quantized_expert_gather_amd as q

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


# 16 lanes a row (2^27 rows a launch), and a workgroup of 1024 threads a row (2^21)
@pytest.mark.parametrize("T,E,step", [((1 << 28) + 77, 4, 1 << 27), ((1 << 22) + 3, 1025, 1 << 21)])
def test_selection_of_more_rows_than_a_launch_holds(T, E, step):
    print("[case] selection", T, E, flush=True)
    z = torch.zeros(T, E, dtype=BF16, device="cuda")
    rows = torch.tensor(sorted({r for i in range(3) for r in (i * step - 1, i * step, i * step + 1) if 0 <= r < T} | {T - 1}),
                        device="cuda")
    z[rows, 2] = 1.0
    z[rows, 3] = torch.arange(len(rows), device="cuda").to(BF16) / 16
    ids, w = q.moe_router_topk(z, 1, score="sigmoid", renormalize=False)
    assert (ids[rows] == 2).all() and torch.equal(w[rows], torch.full_like(w[rows], w[rows[0], 0].item()))
    assert int((ids == 2).sum()) == len(rows) and int((w == 0.5).sum()) == T - len(rows)
    g = torch.ones(T, 1, device="cuda")
    dz = q.moe_router_topk_backward(z, ids, g, score="sigmoid", renormalize=False)
    p = torch.sigmoid(torch.tensor(1.0, dtype=torch.float64))
    assert ((dz[rows, 2].double().cpu() - p * (1 - p)).abs() <= 2.0 ** -8 * 0.2).all() and (dz[rows, 3] == 0).all()
    others = torch.ones(T, dtype=torch.bool, device="cuda")
    others[rows] = False
    assert bool(((dz[:, 0] == 0.25) == others).all()) and int((dz[:, 1] != 0).sum()) == 0


def test_short_products_of_more_outputs_than_a_launch_holds():
    # 16 tokens x 2^28 outputs of 32 inputs: 2^32 outputs
    L, N, K = 16, q.MOE_Q4_LINEAR_MAX_N, 32
    print("[case] short product", L, N, K, flush=True)
    w = torch.zeros(N, K // 8, dtype=torch.int32, device="cuda")
    s = torch.full((N, 1), 127, dtype=torch.uint8, device="cuda")
    cols = torch.tensor([0, 1, 255, 256, (1 << 27) - 1, 1 << 27, N - 256, N - 1], device="cuda")
    w[cols, 0] = 0x22222222   # E2M1 1.0, eight inputs
    x = torch.arange(1, L + 1, device="cuda").to(BF16).view(L, 1).expand(L, K).contiguous()
    out = q.moe_linear_codec_forward("mxfp4", x, w, s)
    want = (8.0 * torch.arange(1, L + 1, device="cuda")).to(BF16)
    for t in range(L):
        assert (out[t, cols] == want[t]).all(), t
        assert int((out[t] != 0).sum()) == len(cols), t
