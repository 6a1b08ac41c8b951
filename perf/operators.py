"""Cases of the operators beside the expert layer: the dense product with 4-bit
weights (`moe_linear_codec_forward`), the router's selection
(`moe_router_topk`, `moe_router_topk_backward`) and the balance loss
(`moe_balance_loss`, `moe_balance_loss_backward`).

Every operator is here twice: `run` computes it in its plain form (elementary
torch operations in 32 bits, or in 64 where an order of values is decided) or,
with `own` set, through the package; `exact` computes it again in 64 bits.

Formulas
  linear   out[t, n] = sum_c x[t, c] W[n, c] + bias[n];
           W = s q + b (4-bit affine, bf16 s and b per 64 or 32 inputs),
           W = 2^(e - 127) e2m1(q) (mxfp4, 32 inputs) or e4m3(s) e2m1(q) (nvfp4, 16 inputs);
           element c of a row is nibble c % 8 of its word c / 8
  route    p = softmax(z) or sigmoid(z); the k largest of p + select_bias, in
           falling order (ties: the lower expert); w = scale p / sum of the chosen p
           (or scale p); backward: dz from dw, the choice held fixed
  balance  per sequence of n unmasked tokens: counts_e = routes to e,
           P_e = mean of p (softmax, or sigmoid / its sum),
           loss = coef E / (k n) sum_e counts_e P_e; backward: dz, counts held fixed
"""

import math

import torch

own = False

DEV = "cuda"
CODECS = {"affine4_g64": 64, "affine4_g32": 32, "mxfp4": 32, "nvfp4": 16}
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
MAGNITUDES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)

# the largest product of the listed cases and the largest weight
MOST_FLOPS = 2 * 2048 * 6144 * 4096
MOST_WEIGHTS = 131072 * 4096
MOST_LOGITS = 32768 * 256


def listed():
    return [
        # the router's own projection while one token is decoded: 256 experts, fp32 logits
        dict(name="linear_router_1", op="linear", codec="affine4_g64", x="bf16", out="f32", L=1, N=256, K=6144, bias=False),
        # an attention output or dense layer's projection, one token
        dict(name="linear_decode_1", op="linear", codec="affine4_g64", x="bf16", out="bf16", L=1, N=6144, K=6144, bias=False),
        # a verify window over a ragged fused projection with a bias
        dict(name="linear_verify_7", op="linear", codec="affine4_g32", x="f16", out="f16", L=7, N=4099, K=4096, bias=True),
        # the vocabulary's logits of a verify window
        dict(name="linear_head_4", op="linear", codec="mxfp4", x="bf16", out="f32", L=4, N=131072, K=4096, bias=False),
        # a short prompt, or a batch of decoding requests
        dict(name="linear_batch_96", op="linear", codec="nvfp4", x="bf16", out="bf16", L=96, N=2050, K=4096, bias=False),
        # a prefill
        dict(name="linear_prefill_2048", op="linear", codec="affine4_g64", x="bf16", out="bf16", L=2048, N=6144, K=4096, bias=False),
        # the routes of a verify window: sigmoid scores and a selection bias
        dict(name="route_verify_4", op="route", z="f32", T=4, E=256, k=8, score="sigmoid", bias=True, norm=True, scale=2.5, back=False),
        # a training batch, with the gradient
        dict(name="route_train_16384", op="route", z="bf16", T=16384, E=256, k=8, score="softmax", bias=False, norm=True, scale=1.0, back=True),
        # odd sizes, weights left unnormalised (their gradient reaches every logit)
        dict(name="route_odd_5003", op="route", z="f32", T=5003, E=288, k=6, score="softmax", bias=False, norm=False, scale=1.0, back=True),
        # a small batch: loss and gradient of one sequence
        dict(name="balance_1000", op="balance", z="f32", S=1, T=1000, E=64, k=6, score="softmax", coef=0.01, mask=False),
        # a training batch
        dict(name="balance_train_32768", op="balance", z="bf16", S=1, T=32768, E=256, k=8, score="softmax", coef=0.001, mask=False),
        # padded sequences, a loss of its own for each
        dict(name="balance_padded_8", op="balance", z="f32", S=8, T=1500, E=288, k=8, score="sigmoid", coef=0.0001, mask=True),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(("linear", "linear", "route", "balance"))
    if op == "linear":
        codec, x = rng.choice(sorted(CODECS)), rng.choice(("bf16", "f16"))
        out = rng.choice((x, x, "f32"))
        while True:
            L, N = _log(rng, 1, 2048), _log(rng, 64, 131072)
            K = 64 * _log(rng, 2, 192)
            if 2 * L * N * K <= MOST_FLOPS and N * K <= MOST_WEIGHTS:
                return dict(op=op, codec=codec, x=x, out=out, L=L, N=N, K=K, bias=rng.random() < 0.4)
    z, score = rng.choice(("f32", "bf16", "f16")), rng.choice(("softmax", "sigmoid"))
    while True:
        E = _log(rng, 8, 512)
        k = rng.randint(1, min(E // 2, 16))  # with every expert chosen, or one alone made to sum to 1, the gradients vanish
        if op == "route":
            T = _log(rng, 1, 16384)
            if T * E <= 16384 * 256:
                return dict(op=op, z=z, T=T, E=E, k=k, score=score, bias=rng.random() < 0.4, norm=k > 1 and rng.random() < 0.6,
                            scale=rng.choice((1.0, 2.5)), back=rng.random() < 0.7)
        else:
            S, T = rng.choice((1, 1, 2, 5, 16)), _log(rng, 16, 32768)
            if S * T * E <= MOST_LOGITS:
                return dict(op=op, z=z, S=S, T=T, E=E, k=k, score=score, coef=rng.choice((0.01, 0.001)), mask=rng.random() < 0.5)


# ---- inputs ----

def _codes(g, codec, N, K):
    """Packed codes of normal weights, int32 [N, K/8], made in runs of rows."""
    packed = torch.empty(N, K // 8, dtype=torch.int32, device=DEV)
    edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=DEV)
    step = max(1, (1 << 26) // K)
    shifts = torch.arange(0, 32, 4, device=DEV, dtype=torch.int32)
    for r in range(0, N, step):
        v = torch.randn(min(step, N - r), K, generator=g, device=DEV)
        if codec.startswith("affine"):
            q = (7.5 + 3.2 * v).round_().clamp_(0, 15).to(torch.int32)
        else:
            v *= 2.1
            q = torch.bucketize(v.abs(), edges, out_int32=True) + 8 * (v < 0).to(torch.int32)
        packed[r:r + step] = (q.view(q.shape[0], K // 8, 8) << shifts).sum(-1, dtype=torch.int32)
    return packed


def _prepare_linear(c, g):
    L, N, K, codec = c["L"], c["N"], c["K"], c["codec"]
    groups = K // CODECS[codec]
    sigma = 1.0 / math.sqrt(K)
    w = _codes(g, codec, N, K)
    b = None
    if codec.startswith("affine"):
        s = sigma * 0.31 * (1 + 0.12 * torch.randn(N, groups, generator=g, device=DEV))
        b = (-7.5 * s * (1 + 0.05 * torch.randn(N, groups, generator=g, device=DEV))).to(torch.bfloat16)
        s = s.to(torch.bfloat16)
    elif codec == "mxfp4":
        e = torch.randint(-1, 2, (N, groups), generator=g, device=DEV) + int(math.floor(math.log2(sigma / 2)))
        s = (127 + e).to(torch.uint8)
    else:  # E4M3 bytes of positive normal numbers near 2^-6 .. 2^-4
        s = torch.randint(0x08, 0x20, (N, groups), generator=g, device=DEV).to(torch.uint8)
    x = torch.randn(L, K, generator=g, device=DEV)
    x *= 1 + 12 * (torch.rand(K, generator=g, device=DEV) < 0.004).float()  # a few loud channels
    bias = 0.1 * torch.randn(N, generator=g, device=DEV) if c["bias"] else None
    return dict(c=c, x=x.to(TYPES[c["x"]]), w=w, s=s, b=b, bias=bias)


def _logits(g, T, E, kind):
    """Router logits: experts differ in how popular they are, tokens in how sure the router is."""
    z = 1.3 * torch.randn(T, E, generator=g, device=DEV) + 0.7 * torch.randn(E, generator=g, device=DEV)
    z *= 0.5 + torch.rand(T, 1, generator=g, device=DEV)
    return z.to(TYPES[kind])


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    if c["op"] == "linear":
        return _prepare_linear(c, g)
    E, k = c["E"], c["k"]
    if c["op"] == "route":
        z = _logits(g, c["T"], E, c["z"])
        bias = 0.05 * torch.randn(E, generator=g, device=DEV) if c["bias"] else None
        dw = torch.randn(c["T"], k, generator=g, device=DEV) if c["back"] else None
        return dict(c=c, z=z, bias=bias, dw=dw)
    S, T = c["S"], c["T"]
    z = _logits(g, S * T, E, c["z"])
    ids = z.float().topk(k, dim=-1).indices.to(torch.int32)
    mask = None
    if c["mask"]:  # right-padded sequences of random lengths
        lens = torch.randint(0, T + 1, (S, 1), generator=g, device=DEV)
        mask = (torch.arange(T, device=DEV) < lens).reshape(S * T)
    # the gradient that reaches the losses: their mean's, and a loss scale where the gradients are fp16
    dloss = torch.full((S,), (65536.0 if c["z"] == "f16" else 1.0) / S, device=DEV)
    return dict(c=c, z=z, ids=ids, mask=mask, dloss=dloss)


# ---- plain forms ----

def _weights(codec, w, s, b):
    """W as fp32 [N, K]."""
    N = w.shape[0]
    shifts = torch.arange(0, 32, 4, device=w.device, dtype=torch.int32)
    q = ((w.unsqueeze(-1) >> shifts) & 15).view(N, s.shape[1], CODECS[codec])
    if codec.startswith("affine"):
        W = q.float() * s.float().unsqueeze(-1) + b.float().unsqueeze(-1)
    else:
        table = torch.tensor(MAGNITUDES + tuple(-m for m in MAGNITUDES), device=w.device)
        scale = torch.exp2(s.float() - 127) if codec == "mxfp4" else s.view(torch.float8_e4m3fn).float()
        W = table[q] * scale.unsqueeze(-1)
    return W.view(N, -1)


def _plain_linear(st):
    y = st["x"].float() @ _weights(st["c"]["codec"], st["w"], st["s"], st["b"]).t()
    if st["bias"] is not None:
        y = y + st["bias"]
    return y.to(TYPES[st["c"]["out"]])


def _softmax(z):
    e = torch.exp(z - z.amax(-1, keepdim=True))
    return e / e.sum(-1, keepdim=True)


def _sigmoid(z):
    return 1 / (1 + torch.exp(-z))


def _choice(z, bias, score, k):
    """The k experts of each token: in 64 bits where scores are added to a bias."""
    if bias is None:
        key = z.float()
    else:
        key = (_softmax if score == "softmax" else _sigmoid)(z.double()) + bias.double()
    return torch.sort(key, dim=-1, descending=True, stable=True).indices[:, :k]


def _plain_route(st):
    c, z = st["c"], st["z"].float()
    softmax, norm, scale = c["score"] == "softmax", c["norm"], c["scale"]
    ids = _choice(st["z"], st["bias"], c["score"], c["k"])
    p = (_softmax if softmax else _sigmoid)(z)
    chosen = p.gather(-1, ids)
    total = chosen.sum(-1, keepdim=True)
    w = scale * (chosen / total if norm else chosen)
    out = {"ids": ids.to(torch.int32), "weights": w}
    if c["back"]:
        g = st["dw"]
        if norm:
            dc = (scale * g - (w * g).sum(-1, keepdim=True)) / total
        else:
            dc = scale * g
        dp = torch.zeros_like(p).scatter_(-1, ids, dc)
        dz = p * (dp - (p * dp).sum(-1, keepdim=True)) if softmax else dp * p * (1 - p)
        out["dlogits"] = dz.to(st["z"].dtype)
    return out


def _plain_balance(st):
    c, z = st["c"], st["z"].float()
    S, T, E, k = c["S"], c["T"], c["E"], c["k"]
    if c["score"] == "softmax":
        p, s = _softmax(z), None
    else:
        s = _sigmoid(z)
        p = s / s.sum(-1, keepdim=True)
    live = torch.ones(S * T, device=z.device) if st["mask"] is None else st["mask"].float()
    n = live.view(S, T).sum(-1)
    hits = torch.zeros(S * T, E, device=z.device).scatter_(-1, st["ids"].long(), 1.0) * live.unsqueeze(-1)
    counts = hits.view(S, T, E).sum(1)
    total = (p * live.unsqueeze(-1)).view(S, T, E).sum(1)
    safe = n.clamp(min=1)
    loss = c["coef"] * E / (k * safe * safe) * (counts * total).sum(-1)
    a = (st["dloss"] * c["coef"] * E / (k * safe * safe)).unsqueeze(-1) * counts
    a = a.repeat_interleave(T, 0) * live.unsqueeze(-1)
    dz = p * (a - (p * a).sum(-1, keepdim=True))
    if s is not None:
        dz = dz * (1 - s)
    return {"loss": loss, "counts": counts.to(torch.int32), "tokens": n.to(torch.int32), "dlogits": dz.to(st["z"].dtype)}


# ---- the package's calls ----

def _own_linear(st):
    import quantized_expert_gather_amd as q
    c = st["c"]
    return q.moe_linear_codec_forward(c["codec"], st["x"], st["w"], st["s"], st["b"], bias=st["bias"],
                                      out_dtype=TYPES[c["out"]])


def _own_route(st):
    import quantized_expert_gather_amd as q
    c = st["c"]
    kw = dict(score=c["score"], renormalize=c["norm"], scale=c["scale"])
    ids, w = q.moe_router_topk(st["z"], c["k"], select_bias=st["bias"], **kw)
    out = {"ids": ids, "weights": w}
    if c["back"]:
        out["dlogits"] = q.moe_router_topk_backward(st["z"], ids, st["dw"], **kw)
    return out


def _own_balance(st):
    import quantized_expert_gather_amd as q
    c = st["c"]
    kw = dict(coef=c["coef"], score=c["score"], token_mask=st["mask"])
    loss, counts, tokens = q.moe_balance_loss(st["z"], st["ids"], seqs=c["S"], **kw)
    dz = q.moe_balance_loss_backward(st["z"], counts, tokens, st["dloss"], c["k"], **kw)
    return {"loss": loss, "counts": counts, "tokens": tokens, "dlogits": dz}


def run(state):
    op = state["c"]["op"]
    if own:
        return (_own_linear if op == "linear" else _own_route if op == "route" else _own_balance)(state)
    return (_plain_linear if op == "linear" else _plain_route if op == "route" else _plain_balance)(state)


# ---- what a pass cannot do without ----

def work(case):
    c = case
    size = {"bf16": 2, "f16": 2, "f32": 4}
    if c["op"] == "linear":
        L, N, K = c["L"], c["N"], c["K"]
        groups = K // CODECS[c["codec"]]
        side = N * groups * (4 if c["codec"].startswith("affine") else 1) + (4 * N if c["bias"] else 0)
        return {"bytes": N * K // 2 + side + L * K * 2 + L * N * size[c["out"]], "flops": 2 * L * N * K}
    z = size[c["z"]]
    if c["op"] == "route":
        T, E, k = c["T"], c["E"], c["k"]
        n = T * E * z + T * k * 8 + (4 * E if c["bias"] else 0)
        if c["back"]:
            n += T * k * 4 + T * E * z
        return {"bytes": n, "flops": T * E * (4 if c["back"] else 2)}
    T, E, k = c["S"] * c["T"], c["E"], c["k"]
    return {"bytes": 2 * T * E * z + T * k * 4 + (T if c["mask"] else 0) + c["S"] * (4 * E + 12), "flops": 8 * T * E}


# ---- the definitions in 64 bits ----

def _exact_linear(st):
    codec, w, s = st["c"]["codec"], st["w"], st["s"]
    N, K, gs = w.shape[0], w.shape[1] * 8, CODECS[st["c"]["codec"]]
    x = st["x"].double()
    y = torch.empty(x.shape[0], N, dtype=torch.float64, device=x.device)
    step = max(1, (1 << 27) // K)
    for r in range(0, N, step):
        raw = w[r:r + step].contiguous().view(torch.uint8)
        q = torch.stack((raw % 16, raw // 16), -1).view(raw.shape[0], K).double()
        if codec.startswith("affine"):
            v = q * s[r:r + step].double().repeat_interleave(gs, 1) + st["b"][r:r + step].double().repeat_interleave(gs, 1)
        else:
            sign, mag = 1 - 2 * torch.floor(q / 8), q % 8
            expo, mant = torch.floor(mag / 2), mag % 2
            v = sign * torch.where(expo == 0, mant / 2, (1 + mant / 2) * torch.exp2(expo - 1))
            sb = s[r:r + step].double()
            if codec == "mxfp4":
                sc = torch.pow(2.0, sb - 127)
            else:
                e4, m3 = torch.floor(sb / 8), sb % 8
                sc = torch.where(e4 == 0, m3 / 8 * 2.0 ** -6, (1 + m3 / 8) * torch.exp2(e4 - 7))
            v = v * sc.repeat_interleave(gs, 1)
        y[:, r:r + step] = torch.matmul(x, v.transpose(0, 1).contiguous())
    return y if st["bias"] is None else y + st["bias"].double()


def _exact_route(st):
    c, z, k = st["c"], st["z"].double(), st["c"]["k"]
    score = torch.softmax(z, -1) if c["score"] == "softmax" else torch.sigmoid(z)
    key = z if st["bias"] is None else score + st["bias"].double()
    order = torch.argsort(key, dim=-1, descending=True, stable=True)[:, :k]
    rows = torch.arange(z.shape[0], device=z.device).unsqueeze(-1)
    s = score[rows, order]
    S = s.sum(-1, keepdim=True) if c["norm"] else torch.ones_like(s[:, :1])
    w = c["scale"] * s / S
    out = {"ids": order.to(torch.int32), "weights": w}
    if c["back"]:
        g = st["dw"].double()
        dz = torch.zeros_like(z)
        dot = (w * g).sum(-1, keepdim=True)
        if c["score"] == "softmax":
            if c["norm"]:  # w depends on the chosen logits alone
                dz[rows, order] = w * (g - dot / c["scale"])
            else:
                dz = -score * dot
                dz[rows, order] += w * g
        else:
            dz[rows, order] = ((g - dot / c["scale"]) if c["norm"] else g) * w * (1 - s)
        out["dlogits"] = dz
    return out


def _exact_balance(st):
    c = st["c"]
    S, T, E, k = c["S"], c["T"], c["E"], c["k"]
    z = st["z"].double().view(S, T, E)
    if c["score"] == "softmax":
        p, damp = torch.softmax(z, -1), 1.0
    else:
        sg = torch.sigmoid(z)
        p, damp = sg / sg.sum(-1, keepdim=True), 1 - sg
    on = torch.ones(S, T, dtype=torch.float64, device=z.device) if st["mask"] is None else st["mask"].view(S, T).double()
    n = on.sum(1)
    counts = torch.zeros(S, E, dtype=torch.float64, device=z.device)
    counts.scatter_add_(1, st["ids"].long().view(S, T * k), on.repeat_interleave(k, 1))
    f = torch.where(n > 0, c["coef"] * E / (k * n.clamp(min=1)), torch.zeros_like(n)).unsqueeze(-1) * counts
    mean = (p * on.unsqueeze(-1)).sum(1) / n.clamp(min=1).unsqueeze(-1)
    a = st["dloss"].double().unsqueeze(-1) * f / n.clamp(min=1).unsqueeze(-1)
    inner = (a.unsqueeze(1) * p).sum(-1, keepdim=True)
    dz = damp * p * (a.unsqueeze(1) - inner) * on.unsqueeze(-1)
    return {"loss": (f * mean).sum(-1), "counts": counts.to(torch.int32), "tokens": n.to(torch.int32),
            "dlogits": dz.view(S * T, E)}


def exact(case, seed):
    st = prepare(case, seed)
    op = st["c"]["op"]
    return (_exact_linear if op == "linear" else _exact_route if op == "route" else _exact_balance)(st)
