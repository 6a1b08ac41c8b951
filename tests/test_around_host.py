"""Host-side checks of the norm, the quantization, the 8-bit block product and
the gated block (no GPU): every refusal returns before any GPU work, so the
pointers here are fake."""

import pytest
import torch

import quantized_expert_gather_amd as q
from tests import around_refs as R

BASE, STRIDE = 1 << 40, 1 << 36
SHAPE, UNSUP, NULL, ALIGN, ALIAS, WORK, OK = (q.MOE_Q4_ERR_SHAPE, q.MOE_Q4_ERR_UNSUPPORTED, q.MOE_Q4_ERR_NULL, q.MOE_Q4_ERR_ALIGN,
                                              q.MOE_Q4_ERR_ALIAS, q.MOE_Q4_ERR_WORKSPACE, q.MOE_Q4_OK)


def fake(i, off=0):
    return BASE + i * STRIDE + off


def p(v, i):
    return fake(i) if v is None else v


def norm(x=None, xd=0, ldx=None, res=None, rd=0, ldr=None, w=None, wd=0, T=4, H=200, eps=1e-6, total=None, ldt=None, y=None,
         yd=0, ldy=None, codes=None, ldc=None, scales=None):
    ld = lambda v: H if v is None else v  # noqa: E731
    return q.lib().moe_rms_norm(p(x, 0), xd, ld(ldx), p(res, 1), rd, ld(ldr), p(w, 2), wd, T, H, eps, p(total, 3), ld(ldt),
                                p(y, 4), yd, ld(ldy), p(codes, 5), ld(ldc), p(scales, 6), None)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), SHAPE), (dict(H=0), SHAPE), (dict(ldx=199), SHAPE), (dict(ldr=199), SHAPE), (dict(ldt=199), SHAPE),
    (dict(ldy=199), SHAPE), (dict(ldc=199), SHAPE), (dict(eps=-1.0), SHAPE), (dict(eps=float("nan")), SHAPE),
    (dict(H=16385), UNSUP), (dict(T=q.MOE_Q4_ROUTER_MAX_T + 1), UNSUP), (dict(xd=3), UNSUP), (dict(wd=-1), UNSUP),
    (dict(yd=4), UNSUP), (dict(rd=2), UNSUP), (dict(xd=1, rd=0), UNSUP), (dict(x=0), NULL), (dict(total=0), NULL),
    (dict(y=0, codes=0), NULL), (dict(scales=0), NULL), (dict(x=fake(0, 1)), ALIGN), (dict(xd=1, rd=1, x=fake(0, 2)), ALIGN),
    (dict(res=fake(1, 1)), ALIGN), (dict(total=fake(3, 1)), ALIGN), (dict(w=fake(2, 1)), ALIGN), (dict(y=fake(4, 1)), ALIGN),
    (dict(scales=fake(6, 2)), ALIGN), (dict(total=fake(0)), ALIAS), (dict(total=fake(1, 2)), ALIAS),
    (dict(total=fake(1), ldt=210), ALIAS), (dict(y=fake(0)), ALIAS), (dict(y=fake(1)), ALIAS), (dict(y=fake(3)), ALIAS),
    (dict(codes=fake(2)), ALIAS), (dict(scales=fake(5, 796)), ALIAS), (dict(T=0), OK), (dict(T=0, x=0, y=0), OK),
])
def test_norm_refusals(kw, status):
    assert norm(**kw) == status


def norm_back(r=None, rd=0, ldr=None, w=None, wd=0, dy=None, yd=0, ldy=None, dt=None, ldt=None, T=4, H=200, eps=1e-6, dx=None,
              ldd=None, dw=None, ws=None, wn=1 << 30):
    ld = lambda v: H if v is None else v  # noqa: E731
    return q.lib().moe_rms_norm_backward(p(r, 0), rd, ld(ldr), p(w, 1), wd, p(dy, 2), yd, ld(ldy), p(dt, 3), ld(ldt), T, H, eps,
                                         p(dx, 4), ld(ldd), p(dw, 5), p(ws, 6), wn, None)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), SHAPE), (dict(H=0), SHAPE), (dict(ldr=1), SHAPE), (dict(ldy=1), SHAPE), (dict(ldt=1), SHAPE),
    (dict(ldd=1), SHAPE), (dict(eps=-1.0), SHAPE), (dict(H=16385), UNSUP), (dict(rd=5), UNSUP), (dict(yd=5), UNSUP),
    (dict(wd=5), UNSUP), (dict(r=0), NULL), (dict(dy=0), NULL), (dict(dx=0), NULL), (dict(w=0), NULL), (dict(ws=0), WORK),
    # one byte less than the documented need, which is a row of sums a workgroup (here one, of 200 floats)
    (dict(wn=q.moe_rms_norm_backward_workspace_bytes(4, 200) - 1), WORK), (dict(wn=200 * 4 - 1), WORK), (dict(ws=fake(6, 128)), ALIGN), (dict(dx=fake(4, 1)), ALIGN), (dict(dw=fake(5, 1)), ALIGN),
    (dict(dt=fake(3, 1)), ALIGN), (dict(dx=fake(0)), ALIAS), (dict(dx=fake(3)), ALIAS), (dict(dw=fake(1)), ALIAS),
    (dict(ws=fake(2)), ALIAS), (dict(ws=fake(4)), ALIAS), (dict(dw=fake(6, 512)), ALIAS),
])
def test_norm_backward_refusals(kw, status):
    assert norm_back(**kw) == status


def quant(x=None, xd=0, ldx=None, T=4, K=200, rows=1, codes=None, ldc=None, scales=None):
    return q.lib().moe_quantize_fp8(p(x, 0), xd, K if ldx is None else ldx, T, K, rows, p(codes, 1), K if ldc is None else ldc,
                                    p(scales, 2), None)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), SHAPE), (dict(K=0), SHAPE), (dict(ldx=1), SHAPE), (dict(ldc=1), SHAPE), (dict(xd=3), UNSUP), (dict(rows=2), UNSUP),
    (dict(T=1 << 27, K=256), UNSUP), (dict(T=(1 << 30) + 1, K=1, rows=128), UNSUP), (dict(x=0), NULL), (dict(codes=0), NULL),
    (dict(scales=0), NULL), (dict(x=fake(0, 1)), ALIGN), (dict(scales=fake(2, 1)), ALIGN), (dict(codes=fake(0)), ALIAS),
    (dict(scales=fake(1)), ALIAS), (dict(scales=fake(0)), ALIAS), (dict(T=0), OK),
])
def test_quantize_refusals(kw, status):
    assert quant(**kw) == status


def fp8(x=None, ldx=None, sx=None, w=None, sw=None, bias=0, L=40, N=24, K=144, out=None, od=0, ldo=None, ws=None, wn=1 << 34):
    return q.lib().moe_linear_fp8_forward(p(x, 0), K if ldx is None else ldx, p(sx, 1), p(w, 2), p(sw, 3), bias, L, N, K, p(out, 5),
                                          od, N if ldo is None else ldo, p(ws, 6), wn, None)


@pytest.mark.parametrize("kw,status", [
    (dict(L=-1), SHAPE), (dict(N=0), SHAPE), (dict(K=0), SHAPE), (dict(ldx=128), SHAPE), (dict(ldo=23), SHAPE),
    (dict(K=136), UNSUP), (dict(L=q.MOE_Q4_LINEAR_MAX_L + 1), UNSUP), (dict(N=q.MOE_Q4_LINEAR_MAX_N + 1), UNSUP),
    (dict(L=1 << 19, N=1 << 22, ldo=1 << 22), UNSUP),
    (dict(K=q.MOE_Q4_LINEAR_MAX_K + 16), UNSUP), (dict(ldx=q.MOE_Q4_LINEAR_MAX_LDX + 16), UNSUP), (dict(od=3), UNSUP),
    (dict(x=0), NULL), (dict(sx=0), NULL), (dict(w=0), NULL), (dict(sw=0), NULL), (dict(out=0), NULL), (dict(x=fake(0, 8)), ALIGN),
    (dict(ldx=152), ALIGN), (dict(w=fake(2, 8)), ALIGN), (dict(sx=fake(1, 2)), ALIGN), (dict(sw=fake(3, 2)), ALIGN),
    (dict(bias=fake(4, 2)), ALIGN), (dict(out=fake(5, 1)), ALIGN), (dict(od=1, out=fake(5, 2)), ALIGN), (dict(out=fake(0)), ALIAS),
    (dict(out=fake(1)), ALIAS), (dict(out=fake(2)), ALIAS), (dict(out=fake(3)), ALIAS), (dict(out=fake(4), bias=fake(4)), ALIAS),
    (dict(L=0, x=0), OK),
])
def test_fp8_refusals(kw, status):
    assert fp8(**kw) == status


def test_fp8_workspace():
    L, N, K = 40, 100, 8192  # few tiles, long rows: K is split
    n = q.moe_linear_fp8_workspace_bytes(L, N, K)
    assert n > 0 and n % 256 == 0
    assert fp8(L=L, N=N, K=K, ws=0) == WORK and fp8(L=L, N=N, K=K, wn=255) == WORK
    assert fp8(L=L, N=N, K=K, ws=fake(6, 16)) == ALIGN and fp8(L=L, N=N, K=K, ws=fake(0)) == ALIAS
    assert fp8(L=L, N=N, K=K, ws=fake(5)) == ALIAS
    assert q.moe_linear_fp8_workspace_bytes(1, 6144, 6144) == 0 == q.moe_linear_fp8_workspace_bytes(40, 100, 8)
    for L in (33, 64, 300, 3000):
        for N in (1, 100, 5000):
            for K in (16, 2048, 14336):
                assert q.moe_linear_fp8_workspace_bytes(L, N, K) <= 16 * L * N * 4 + 256


def glu(dt=0, x=None, ldx=None, wg=None, wu=None, ldw=None, T=40, H=64, I=72, h=None, ldh=None, saved=0, ws=None, wn=1 << 34):
    return q.lib().moe_glu_forward(dt, p(x, 0), H if ldx is None else ldx, p(wg, 1), p(wu, 2), H if ldw is None else ldw, T, H, I,
                                   p(h, 3), I if ldh is None else ldh, saved, p(ws, 5), wn, None)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), SHAPE), (dict(H=0), SHAPE), (dict(I=0), SHAPE), (dict(ldx=56), SHAPE), (dict(ldw=56), SHAPE), (dict(ldh=71), SHAPE),
    (dict(H=60), UNSUP), (dict(I=70), UNSUP), (dict(dt=1), UNSUP), (dict(T=q.MOE_Q4_LINEAR_MAX_L + 1), UNSUP),
    (dict(ldx=q.MOE_Q4_GLU_MAX_LD + 8), UNSUP), (dict(ldw=q.MOE_Q4_GLU_MAX_LD + 8), UNSUP), (dict(x=0), NULL), (dict(wg=0), NULL),
    (dict(wu=0), NULL), (dict(h=0), NULL), (dict(x=fake(0, 8)), ALIGN), (dict(wg=fake(1, 8)), ALIGN), (dict(wu=fake(2, 2)), ALIGN),
    (dict(ldx=68), ALIGN), (dict(ldw=68), ALIGN), (dict(h=fake(3, 1)), ALIGN), (dict(saved=fake(4, 4)), ALIGN),
    (dict(h=fake(0)), ALIAS), (dict(h=fake(1)), ALIAS), (dict(saved=fake(2)), ALIAS), (dict(saved=fake(3)), ALIAS), (dict(T=0, x=0), OK),
])
def test_glu_refusals(kw, status):
    assert glu(**kw) == status


def glu_back(dt=0, x=None, ldx=None, wg=None, wu=None, ldw=None, dh=None, lddh=None, saved=0, T=40, H=64, I=72, dx=None, lddx=None,
             dwg=None, dwu=None, ws=None, wn=1 << 34):
    return q.lib().moe_glu_backward(dt, p(x, 0), H if ldx is None else ldx, p(wg, 1), p(wu, 2), H if ldw is None else ldw, p(dh, 3),
                                    I if lddh is None else lddh, saved, T, H, I, p(dx, 5), H if lddx is None else lddx, p(dwg, 6),
                                    p(dwu, 7), p(ws, 8), wn, None)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), SHAPE), (dict(lddh=71), SHAPE), (dict(lddx=63), SHAPE), (dict(H=60), UNSUP), (dict(dt=1), UNSUP), (dict(dh=0), NULL),
    (dict(x=0), NULL), (dict(dwg=0), NULL), (dict(dwu=0), NULL), (dict(ws=0), WORK), (dict(wn=1000), WORK),
    (dict(ws=fake(8, 16)), ALIGN), (dict(dwg=fake(6, 2)), ALIGN), (dict(dx=fake(5, 1)), ALIGN), (dict(dx=fake(3)), ALIAS),
    (dict(dwg=fake(7)), ALIAS), (dict(dwu=fake(1)), ALIAS), (dict(ws=fake(2)), ALIAS), (dict(saved=fake(4), ws=fake(4)), ALIAS),
    (dict(dx=0, dwg=0, dwu=0), OK),
])
def test_glu_backward_refusals(kw, status):
    assert glu_back(**kw) == status


def test_bindings_refuse_host_tensors_and_given_outputs():
    x, w = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(8, 64, dtype=torch.bfloat16)
    c, s = torch.zeros(4, 64).to(R.F8), torch.zeros(4, 1)
    for call in (lambda: q.moe_rms_norm(x), lambda: q.moe_rms_norm_fp8(x), lambda: q.moe_rms_norm_backward(x, None, x),
                 lambda: q.moe_quantize_fp8(x), lambda: q.moe_linear_fp8_forward(c, s, c, s[:1]), lambda: q.moe_glu(x, w, w),
                 lambda: q.moe_glu_backward(x, w, w, torch.zeros(4, 8, dtype=torch.bfloat16))):
        with pytest.raises(ValueError, match="device"):
            call()
    x.requires_grad_()
    with pytest.raises(RuntimeError, match="gradient"):
        q.moe_rms_norm(x, out=torch.zeros_like(x))
    with pytest.raises(RuntimeError, match="gradient"):
        q.moe_rms_norm(x, residual=x, total=torch.zeros_like(x))
    with pytest.raises(RuntimeError, match="gradient"):
        q.moe_glu(x, w, w, saved=torch.zeros(2, 4, 8))


# ---- the references themselves, against torch's own differentiation ----

def test_references_against_autograd():
    g = torch.Generator().manual_seed(1)
    rnd = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    x, wg, wu, dh = rnd(4, 16).half(), rnd(8, 16).half(), rnd(8, 16).half(), rnd(4, 8).half()
    a, b, c = (t.double().requires_grad_() for t in (x, wg, wu))
    (torch.nn.functional.silu(a @ b.T) * (c @ a.T).T).backward(dh.double())
    for ref, leaf in zip(R.glu_backward(x, wg, wu, dh)[0], (a, b, c)):
        assert (ref - leaf.grad).abs().max() < 1e-12
    r, w, dy, dt = rnd(3, 20), rnd(20), rnd(3, 20), rnd(3, 20)
    a, b = r.clone().requires_grad_(), w.clone().requires_grad_()
    ((R.norm(a, b, 1e-6)[0] * dy).sum() + (a * dt).sum()).backward()
    dx, _, dw, _ = R.norm_backward(r, w, dy, dt, 1e-6)
    assert (dx - a.grad).abs().max() < 1e-12 and (dw - b.grad).abs().max() < 1e-12


def test_code_reference_finds_a_wrong_code():
    y = torch.randn(5, 200, generator=torch.Generator().manual_seed(2))
    s = R.scales(y, 1).float()
    i, j = R.blocks_of(y, 1)
    codes = (y.double() / s.double()[i, j]).float().to(R.F8)
    R.check_codes(codes, s, y)
    wrong = codes.clone()
    k = y.abs().argmax()
    wrong.view(torch.uint8).view(-1)[k] -= 1
    with pytest.raises(AssertionError):
        R.check_codes(wrong, s, y)
