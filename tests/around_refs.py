"""Plain 64-bit references (torch, on the host) of the norm, the quantization,
the 8-bit block product and the gated block, with the error bounds that their
tests use.  A bound counts roundings: half a step of the result's type, and
2^-24 of the magnitudes that pass through fp32."""

import torch

HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}
U = 2.0 ** -24
F8 = torch.float8_e4m3fn


def total_of(x, residual):
    """x + residual as it is carried on: one rounding to the residual's type."""
    return x if residual is None else (x.float() + residual.float()).to(residual.dtype)


def norm(r, w, eps):
    """(y, bound of its fp32 error): a thread adds at most 32 squares, then 6
    lanes and 16 waves; the root halves what that and the mean leave."""
    r, w = r.double(), 1.0 if w is None else w.double()
    y = r * w / (r.square().mean(1, keepdim=True) + eps).sqrt()
    return y, 40 * U * y.abs()


def norm_backward(r, w, dy, dtotal, eps, rounds=1):
    """(dx, its fp32 bound, dw, its fp32 bound); a thread adds `rounds` rows."""
    r, dy = r.double(), dy.double()
    wd = torch.ones(r.shape[1], dtype=torch.float64) if w is None else w.double()
    v = 1 / (r.square().mean(1, keepdim=True) + eps).sqrt()
    n, a = r * v, dy * wd
    dx = v * (a - n * (a * n).mean(1, keepdim=True))
    # a, n and the product: a few roundings each; the mean's sum 54 and v's 30, of the magnitudes
    bound = 120 * U * v * (a.abs() + n.abs() * (a * n).abs().mean(1, keepdim=True))
    if dtotal is not None:
        dx = dx + dtotal.double()
        bound = bound + U * dtotal.double().abs() + U * dx.abs()
    dw = (dy * n).sum(0)
    return dx, bound, dw, (100 + rounds) * U * (dy * n).abs().sum(0)


def blocks_of(v, rows):
    """Index of each element's scale: (block row, block column)."""
    T, K = v.shape
    return torch.arange(T).unsqueeze(1) // rows, torch.arange(K).unsqueeze(0) // 128


def scales(y, rows):
    T, K = y.shape
    tb, kb = -(-T // rows), -(-K // 128)
    p = torch.zeros(tb * rows, kb * 128, dtype=torch.float64)
    p[:T, :K] = y.double().abs()
    return (p.view(tb, rows, kb, 128).amax((1, 3)) / 448).clamp(min=2.0 ** -126)


def check_codes(codes, got_scales, y, rows=1, slack=60 * U):
    """Scales within `slack`; codes within half a step of y / s (e4m3: 2^-4 of
    the value, 2^-10 near zero), s as the kernel has it."""
    assert codes.dtype == F8 and got_scales.dtype == torch.float32
    s = scales(y, rows)
    g = got_scales.double().cpu()
    assert g.shape == s.shape
    assert ((g - s).abs() <= slack * s).all()
    i, j = blocks_of(y, rows)
    v = y.double() / g[i, j]
    q = codes.cpu().float().double()
    assert ((q - v).abs() <= torch.maximum(v.abs() * 2.0 ** -4, torch.tensor(2.0 ** -10)) + slack * v.abs()).all()


def dequant(codes, s, rows):
    i, j = blocks_of(codes, rows)
    return codes.float().double() * s.double()[i, j]


def linear_fp8(x, sx, w, sw, bias, out=torch.float32):
    """(out, fp32 bound): 128 additions in a block, one a block of K, 24 where
    waves or splits are joined, and the scales' and the bias's roundings.
    16-bit results of more than 32 tokens: 8 neighbours' products each lose up
    to 2^-13 of the largest one's power of two, which is at most that product."""
    X, W = dequant(x, sx, 1), dequant(w, sw, 128)
    res, mag = X @ W.T, X.abs() @ W.abs().T
    if bias is not None:
        res, mag = res + bias.double(), mag + bias.double().abs()
    bound = (160 + x.shape[1] / 128) * U * mag
    if out != torch.float32 and x.shape[0] > 32:
        a, b = X.abs().float(), W.abs().float()
        cut = torch.zeros(a.shape[0], b.shape[0], device=a.device)
        for k in range(0, x.shape[1], 8):
            most = torch.zeros_like(cut)
            for c in range(k, k + 8):
                most = torch.maximum(most, a[:, c:c + 1] * b[:, c])
            cut += most
        bound = bound + 8 * 2.0 ** -13 * cut.double()
    return res, bound


def glu(x, wg, wu):
    """g, u, h and the fp32 bounds of the three."""
    x, wg, wu = x.double(), wg.double(), wu.double()
    H = x.shape[1]
    g, u = x @ wg.T, x @ wu.T
    bg, bu = (H + 24) * U * (x.abs() @ wg.abs().T), (H + 24) * U * (x.abs() @ wu.abs().T)
    s = torch.sigmoid(g)
    h = g * s * u
    # |silu'| <= 1.1; the exponential is off by 2^-24 (2 |g| + 4) of itself
    bh = 1.1 * bg * u.abs() + (g * s).abs() * bu + (2 * g.abs() + 10) * U * h.abs()
    return g, u, h, bg, bu, bh


def glu_backward(x, wg, wu, dh):
    """dx, dwg, dwu with their bounds; dg and du are rounded once to x's type."""
    half, tiny = HALF[x.dtype], TINY[x.dtype]
    g, u, h, bg, bu, _ = glu(x, wg, wu)
    x, wg, wu, dh = (t.double() for t in (x, wg, wu, dh))
    s = torch.sigmoid(g)
    slope = s * (1 + g * (1 - s))
    dg, du = dh * u * slope, dh * g * s
    e = (2 * g.abs() + 12) * U
    # |silu''| <= 0.5; slope's own sum is of numbers up to |g s| + s
    bdg = dh.abs() * (u.abs() * (0.5 * bg + e * (s + (g * s * (1 - s)).abs())) + slope.abs() * bu)
    bdu = dh.abs() * (1.1 * bg + e * (g * s).abs())
    bdg, bdu = bdg + half * (dg.abs() + bdg) + tiny, bdu + half * (du.abs() + bdu) + tiny
    T, I = g.shape
    dx = dg @ wg + du @ wu
    bdx = bdg @ wg.abs() + bdu @ wu.abs() + (2 * I + 24) * U * (dg.abs() @ wg.abs() + du.abs() @ wu.abs())
    dwg, dwu = dg.T @ x, du.T @ x
    bwg = bdg.T @ x.abs() + (T + 24) * U * (dg.abs().T @ x.abs())
    bwu = bdu.T @ x.abs() + (T + 24) * U * (du.abs().T @ x.abs())
    return (dx, dwg, dwu), (bdx, bwg, bwu)


def check(got, ref, bound, dtype=None):
    """got within the fp32 bound of ref, rounded once to its type."""
    dtype = dtype or got.dtype
    assert got.dtype == dtype and got.shape == ref.shape
    g = got.double().cpu()
    assert torch.isfinite(g).all()
    tol = bound + HALF[dtype] * (ref.abs() + bound) + TINY[dtype]
    bad = (g - ref).abs() > tol
    if bad.any():
        i = ((g - ref).abs() / tol).flatten().argmax()
        raise AssertionError(f"{int(bad.sum())} of {bad.numel()} off, worst at {int(i)}: {g.flatten()[i]} for "
                             f"{ref.flatten()[i]}, bound {tol.flatten()[i]}")
