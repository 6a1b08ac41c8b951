"""Cases of the operators around the expert layer: the root-mean-square norm
with the residual's addition and 8-bit output (`moe_rms_norm`,
`moe_rms_norm_fp8`, `moe_rms_norm_backward`), the quantization into 8 bits
(`moe_quantize_fp8`), the 8-bit product with scales for blocks of 128
(`moe_linear_fp8_forward`) and the gated feed-forward block (`moe_glu`,
`moe_glu_backward`).

Every operator is here twice: `run` computes it in its plain form (elementary
torch operations in 32 bits) or, with `own` set, through the package; `exact`
computes it again in 64 bits.

Formulas
  norm   r = x + residual, rounded to the residual's type (the stream that a model
         carries on); y = r w / sqrt(mean(r^2) + eps); 8 bits: for each token and
         128 channels s = max(max |y| / 448, 2^-126), q = e4m3(y / s);
         backward: with v = 1 / sqrt(mean(r^2) + eps), n = r v, a = w dy:
         dr = v (a - n mean(a n)) + dtotal, dw = sum over tokens of dy n
  quant  the same s and q of given values, for blocks of 1 x 128 or 128 x 128
  fp8    out[t, n] = sum over blocks b of sx[t, b] sw[n / 128, b] (sum over c in b of x[t, c] w[n, c]) + bias[n]
  glu    g = x Wg^T, u = x Wu^T, h = g sigmoid(g) u; backward: dg = dh u sigmoid(g) (1 + g (1 - sigmoid(g))),
         du = dh g sigmoid(g), dx = dg Wg + du Wu, dWg = dg^T x, dWu = du^T x
"""

import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}
F8 = torch.float8_e4m3fn
EPS = 1e-6
TINY = 2.0 ** -126

# the largest listed cases, which bound the drawn ones
MOST_NORM = 8192 * 6144
MOST_QUANT = 12288 * 6144
MOST_PRODUCT = 2 * 8192 * 12288 * 6144
MOST_WEIGHTS = 12288 * 8192
MOST_GLU = 12 * 8192 * 6144 * 2048


def listed():
    return [
        # the norm before a layer's experts while one token is decoded, straight into the 8-bit product's input
        dict(name="norm_decode_1", op="norm", x="bf16", res="bf16", w="bf16", T=1, H=6144, mode="fp8"),
        # a prefill's norm, residual stream in bf16
        dict(name="norm_prefill_8192", op="norm", x="bf16", res="bf16", w="bf16", T=8192, H=6144, mode="fp8"),
        # a training step's norm of odd sizes, forward and backward, residual stream in fp32
        dict(name="norm_train_5003", op="norm", x="bf16", res="f32", w="f32", T=5003, H=2050, mode="train"),
        # the input of an 8-bit projection that no norm precedes, a batch of decoding requests
        dict(name="quant_batch_96", op="quant", x="bf16", T=96, K=4112, rows=1),
        # a weight matrix on its way into 8 bits
        dict(name="quant_weight_12288", op="quant", x="f32", T=12288, K=6144, rows=128),
        # an attention output or dense layer's projection, one token
        dict(name="fp8_decode_1", op="fp8", L=1, N=6144, K=6144, out="bf16", bias=False),
        # a verify window over a ragged fused projection with a bias, inputs that end inside a block
        dict(name="fp8_verify_7", op="fp8", L=7, N=4099, K=4112, out="f16", bias=True),
        # a short prompt, or a batch of decoding requests, with fp32 results
        dict(name="fp8_batch_96", op="fp8", L=96, N=2050, K=4096, out="f32", bias=False),
        # a long prefill
        dict(name="fp8_prefill_8192", op="fp8", L=8192, N=12288, K=6144, out="bf16", bias=False),
        # a shared expert of a verify window
        dict(name="glu_verify_4", op="glu", x="bf16", T=4, H=6144, I=2048, back=False),
        # a small training batch of odd sizes in fp16
        dict(name="glu_train_1537", op="glu", x="f16", T=1537, H=2056, I=1416, back=True),
        # a training batch: forward and backward of a shared expert
        dict(name="glu_train_8192", op="glu", x="bf16", T=8192, H=6144, I=2048, back=True),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(("norm", "quant", "fp8", "fp8", "glu", "glu"))
    if op == "norm":
        x = rng.choice(("bf16", "bf16", "f16", "f32"))
        res = rng.choice((x, x, "f32", ""))
        w = rng.choice((x, "f32"))
        mode = rng.choice(("fp8", "y", "train"))
        while True:
            T, H = _log(rng, 1, 32768), _log(rng, 64, 16384)
            if T * H * (3 if mode == "train" else 1) * (SIZE[x] // 2) <= MOST_NORM:
                return dict(op=op, x=x, res=res, w=w, T=T, H=H, mode=mode)
    if op == "quant":
        x, rows = rng.choice(("bf16", "f16", "f32")), rng.choice((1, 1, 128))
        while True:
            T, K = _log(rng, 1, 32768), _log(rng, 64, 16384)
            if T * K <= MOST_QUANT:
                return dict(op=op, x=x, T=T, K=K, rows=rows)
    if op == "fp8":
        while True:
            L, N, K = _log(rng, 1, 8192), _log(rng, 64, 65536), 16 * _log(rng, 8, 1024)
            if 2 * L * N * K <= MOST_PRODUCT and N * K <= MOST_WEIGHTS:
                return dict(op=op, L=L, N=N, K=K, out=rng.choice(("bf16", "bf16", "f16", "f32")), bias=rng.random() < 0.4)
    back = rng.random() < 0.6
    while True:
        T, H, I = _log(rng, 1, 8192), 8 * _log(rng, 16, 1536), 8 * _log(rng, 8, 1024)
        if (12 if back else 4) * T * H * I <= MOST_GLU and H * I <= MOST_WEIGHTS // 2:
            return dict(op=op, x=rng.choice(("bf16", "bf16", "f16")), T=T, H=H, I=I, back=back)


# ---- inputs ----

def _hidden(g, T, H, kind, size=1.0):
    """Activations: normal values with a few loud channels."""
    x = torch.randn(T, H, generator=g, device=DEV)
    x *= size * (1 + 12 * (torch.rand(H, generator=g, device=DEV) < 0.004).float())
    return x.to(TYPES[kind])


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    if c["op"] == "norm":
        T, H = c["T"], c["H"]
        st = dict(c=c, x=_hidden(g, T, H, c["x"], 0.3), res=_hidden(g, T, H, c["res"]) if c["res"] else None)
        st["w"] = (1 + 0.2 * torch.randn(H, generator=g, device=DEV)).to(TYPES[c["w"]])
        if c["mode"] == "train":  # gradients as a loss scale leaves them in 16 bits
            st["dy"] = torch.randn(T, H, generator=g, device=DEV).to(TYPES[c["x"]])
            st["dtotal"] = torch.randn(T, H, generator=g, device=DEV).to(TYPES[c["res"]]) if c["res"] else None
        return st
    if c["op"] == "quant":
        T, K = c["T"], c["K"]
        return dict(c=c, x=_hidden(g, T, K, c["x"]) if c["rows"] == 1 else (torch.randn(T, K, generator=g, device=DEV) / math.sqrt(K)).to(TYPES[c["x"]]))
    if c["op"] == "fp8":
        L, N, K = c["L"], c["N"], c["K"]
        kb = -(-K // 128)
        # codes of normal values whose block's largest is near 448, scales that differ from token to token and block to block
        x = (140 * torch.randn(L, K, generator=g, device=DEV)).clamp_(-448, 448).to(F8)
        sx = torch.exp(0.5 * torch.randn(L, kb, generator=g, device=DEV)) / 140
        w = torch.randn(N, K, generator=g, device=DEV).mul_(105).clamp_(-448, 448).to(F8)
        sw = (1 + 0.2 * torch.rand(-(-N // 128), kb, generator=g, device=DEV)) / (105 * math.sqrt(K))
        return dict(c=c, x=x, sx=sx, w=w, sw=sw, bias=0.1 * torch.randn(N, generator=g, device=DEV) if c["bias"] else None)
    T, H, I = c["T"], c["H"], c["I"]
    kind = TYPES[c["x"]]
    st = dict(c=c, x=_hidden(g, T, H, c["x"]))
    st["wg"] = (torch.randn(I, H, generator=g, device=DEV) / math.sqrt(H)).to(kind)
    st["wu"] = (torch.randn(I, H, generator=g, device=DEV) / math.sqrt(H)).to(kind)
    if c["back"]:
        st["dh"] = torch.randn(T, I, generator=g, device=DEV).to(kind)
    return st


# ---- plain forms ----

def _blocks(v):
    """Rows in blocks of 128 columns, the last filled up with zeros: [T, blocks, 128]."""
    T, K = v.shape
    kb = -(-K // 128)
    return torch.nn.functional.pad(v, (0, kb * 128 - K)).view(T, kb, 128)


def _plain_fp8(v, rows=1):
    T, K = v.shape
    b = _blocks(v)
    most = b.abs().amax(-1)
    if rows > 1:
        tb = -(-T // rows)
        most = torch.nn.functional.pad(most, (0, 0, 0, tb * rows - T)).view(tb, rows, -1).amax(1)
    s = (most / 448).clamp(min=TINY)
    each = s if rows == 1 else s.repeat_interleave(rows, 0)[:T]
    q = (b / each.unsqueeze(-1)).view(T, -1)[:, :K].contiguous().to(F8)
    return q, s


def _plain_norm(st):
    c = st["c"]
    r = st["x"] if st["res"] is None else (st["x"].float() + st["res"].float()).to(st["res"].dtype)
    f, w = r.float(), st["w"].float()
    v = 1 / torch.sqrt((f * f).mean(-1, keepdim=True) + EPS)
    n = f * v
    y = n * w
    out = {} if st["res"] is None else {"total": r}
    if c["mode"] == "fp8":
        out["codes"], out["scales"] = _plain_fp8(y)
        return out
    out["y"] = y.to(st["x"].dtype)
    if c["mode"] == "train":
        dy = st["dy"].float()
        a = w * dy
        d = v * (a - n * (a * n).mean(-1, keepdim=True))
        if st["dtotal"] is not None:
            d = d + st["dtotal"].float()
        out["dx"], out["dw"] = d.to(r.dtype), (dy * n).sum(0).to(st["w"].dtype)
    return out


def _plain_product(st):
    c = st["c"]
    K = c["K"]
    x = (_blocks(st["x"].float()) * st["sx"].unsqueeze(-1)).view(c["L"], -1)[:, :K]
    w = (_blocks(st["w"].float()) * st["sw"].repeat_interleave(128, 0)[:c["N"]].unsqueeze(-1)).view(c["N"], -1)[:, :K]
    y = x @ w.t()
    if st["bias"] is not None:
        y = y + st["bias"]
    return y.to(TYPES[c["out"]])


def _plain_glu(st):
    x, wg, wu = st["x"].float(), st["wg"].float(), st["wu"].float()
    g, u = x @ wg.t(), x @ wu.t()
    sig = 1 / (1 + torch.exp(-g))
    silu = g * sig
    kind = st["x"].dtype
    out = {"h": (silu * u).to(kind)}
    if st["c"]["back"]:
        dh = st["dh"].float()
        dg, du = dh * u * (sig * (1 + g * (1 - sig))), dh * silu
        out["dx"] = (dg @ wg + du @ wu).to(kind)
        out["dwg"], out["dwu"] = (dg.t() @ x).to(kind), (du.t() @ x).to(kind)
    return out


# ---- the package's calls ----

def _own_norm(st):
    import quantized_expert_gather_amd as q
    c = st["c"]
    out = {}
    if c["mode"] == "fp8":
        got = q.moe_rms_norm_fp8(st["x"], st["w"], residual=st["res"], eps=EPS)
        out["codes"], out["scales"] = got[:2]
        if st["res"] is not None:
            out["total"] = got[2]
        return out
    got = q.moe_rms_norm(st["x"], st["w"], residual=st["res"], eps=EPS)
    out["y"], r = (got, st["x"]) if st["res"] is None else got
    if st["res"] is not None:
        out["total"] = r
    if c["mode"] == "train":
        out["dx"], out["dw"] = q.moe_rms_norm_backward(r, st["w"], st["dy"], dtotal=st["dtotal"], eps=EPS)
    return out


def _own_glu(st):
    import quantized_expert_gather_amd as q
    x, wg, wu = st["x"], st["wg"], st["wu"]
    if not st["c"]["back"]:
        return {"h": q.moe_glu(x, wg, wu)}
    saved = torch.empty(2, x.shape[0], wg.shape[0], dtype=torch.float32, device=x.device)
    h = q.moe_glu(x, wg, wu, saved=saved)
    dx, dwg, dwu = q.moe_glu_backward(x, wg, wu, st["dh"], saved=saved)
    return {"h": h, "dx": dx, "dwg": dwg, "dwu": dwu}


def run(state):
    op = state["c"]["op"]
    if own:
        import quantized_expert_gather_amd as q
        if op == "norm":
            return _own_norm(state)
        if op == "quant":
            codes, scales = q.moe_quantize_fp8(state["x"], block_rows=state["c"]["rows"])
            return {"codes": codes, "scales": scales}
        if op == "fp8":
            return q.moe_linear_fp8_forward(state["x"], state["sx"], state["w"], state["sw"], bias=state["bias"],
                                            out_dtype=TYPES[state["c"]["out"]])
        return _own_glu(state)
    if op == "norm":
        return _plain_norm(state)
    if op == "quant":
        codes, scales = _plain_fp8(state["x"].float(), state["c"]["rows"])
        return {"codes": codes, "scales": scales}
    return _plain_product(state) if op == "fp8" else _plain_glu(state)


# ---- what a pass cannot do without ----

def work(case):
    c = case
    if c["op"] == "norm":
        T, H = c["T"], c["H"]
        r = SIZE[c["res"]] if c["res"] else 0
        n = T * H * (SIZE[c["x"]] + 2 * r) + H * SIZE[c["w"]]
        if c["mode"] == "fp8":
            return {"bytes": n + T * H + 4 * T * (-(-H // 128)), "flops": 6 * T * H}
        n += T * H * SIZE[c["x"]]
        if c["mode"] == "y":
            return {"bytes": n, "flops": 4 * T * H}
        # dy and dtotal in, dx out; the sum is at hand from the forward
        n += T * H * (SIZE[c["x"]] + r + (r or SIZE[c["x"]])) + H * SIZE[c["w"]]
        return {"bytes": n, "flops": 14 * T * H}
    if c["op"] == "quant":
        T, K = c["T"], c["K"]
        return {"bytes": T * K * (SIZE[c["x"]] + 1) + 4 * (-(-T // c["rows"])) * (-(-K // 128)), "flops": 2 * T * K}
    if c["op"] == "fp8":
        L, N, K = c["L"], c["N"], c["K"]
        kb = -(-K // 128)
        n = L * K + N * K + 4 * L * kb + 4 * (-(-N // 128)) * kb + L * N * SIZE[c["out"]] + (4 * N if c["bias"] else 0)
        return {"bytes": n, "flops": 2 * L * N * K}
    T, H, I = c["T"], c["H"], c["I"]
    n = 2 * (T * H + 2 * I * H + T * I)
    if c["back"]:
        n += 2 * (T * I + T * H + 2 * I * H)
    return {"bytes": n, "flops": (12 if c["back"] else 4) * T * H * I}


# ---- the definitions in 64 bits ----

def _exact_codes(v, rows):
    """Scales of the blocks and the values over them, block column by block column."""
    T, K = v.shape
    scales, values = [], []
    for k in range(0, K, 128):
        part = v[:, k:k + 128]
        most = part.abs().max(dim=1).values
        if rows > 1:
            most = torch.stack([p.max() for p in most.split(rows)])
        s = torch.maximum(most / 448, torch.tensor(TINY, dtype=v.dtype, device=v.device))
        scales.append(s)
        values.append(part / torch.repeat_interleave(s, rows)[:T].unsqueeze(1))
    return torch.cat(values, 1), torch.stack(scales, 1)


def _exact_norm(st):
    x, w = st["x"].double(), st["w"].double()
    out = {}
    if st["res"] is not None:
        s = x + st["res"].double()
        out["total"] = s
        x = s.to(st["res"].dtype).double()  # the norm is that of the sum as it is carried on
    H = x.shape[1]
    v = torch.rsqrt(torch.linalg.vector_norm(x, dim=1, keepdim=True) ** 2 / H + EPS)
    y = x * v * w
    if st["c"]["mode"] == "fp8":
        out["codes"], out["scales"] = _exact_codes(y, 1)
        return out
    out["y"] = y
    if st["c"]["mode"] == "train":
        dy = st["dy"].double()
        dot = (dy * w * x).sum(1, keepdim=True)
        d = dy * w * v - x * v ** 3 * dot / H
        out["dx"] = d if st["dtotal"] is None else d + st["dtotal"].double()
        out["dw"] = torch.einsum("th,th,t->h", dy, x, v.squeeze(1))
    return out


def _exact_product(st):
    x, w = st["x"].double(), st["w"].double()
    L, N, K = x.shape[0], w.shape[0], x.shape[1]
    col = torch.arange(K, device=x.device) // 128
    x = x * st["sx"].double()[:, col]
    y = torch.empty(L, N, dtype=torch.float64, device=x.device)
    for n in range(0, N, 8192):
        rows = torch.arange(n, min(N, n + 8192), device=x.device) // 128
        part = w[n:n + 8192] * st["sw"].double()[rows][:, col]
        y[:, n:n + 8192] = torch.matmul(x, part.transpose(0, 1).contiguous())
    return y if st["bias"] is None else y + st["bias"].double()


def _exact_glu(st):
    x, wg, wu = st["x"].double(), st["wg"].double(), st["wu"].double()
    g = torch.matmul(x, wg.transpose(0, 1).contiguous())
    u = torch.matmul(x, wu.transpose(0, 1).contiguous())
    s = torch.sigmoid(g)
    out = {"h": g * s * u}
    if st["c"]["back"]:
        dh = st["dh"].double()
        dg, du = dh * u * (s + g * s * torch.sigmoid(-g)), dh * g * s
        out["dx"] = torch.matmul(dg, wg) + torch.matmul(du, wu)
        out["dwg"] = torch.matmul(dg.transpose(0, 1).contiguous(), x)
        out["dwu"] = torch.matmul(du.transpose(0, 1).contiguous(), x)
    return out


def exact(case, seed):
    st = prepare(case, seed)
    op = st["c"]["op"]
    if op == "norm":
        return _exact_norm(st)
    if op == "quant":
        codes, scales = _exact_codes(st["x"].double(), st["c"]["rows"])
        return {"codes": codes, "scales": scales}
    return _exact_product(st) if op == "fp8" else _exact_glu(st)
