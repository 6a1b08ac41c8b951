"""Plain 64-bit references (numpy) of the operators beside the expert layer,
and the error bounds their tests use."""

import numpy as np
import torch

import oracle
import synth

GROUPS = {"affine4_g64": 64, "affine4_g32": 32, "mxfp4": 32, "nvfp4": 16}
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
# half the spacing of the smallest numbers a type holds
HALF_TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}


def linear_weights(codec, N, K, seed):
    """(codes, scales, biases) of normal weights as the generators store them."""
    return synth.gen_matrix_q(codec, 1, N, K, ("dense", seed))


def linear_reference(codec, x, w, s, b, bias):
    """(out, bound) in 64 bits.  The kernel's products are exact and its sums
    fp32: an addend of the result is rounded at most 64 times inside a matrix
    product, twice per scale group of K and 16 times where waves or passes
    over K are joined, each time by 2^-24 of a partial sum that is at most the
    sum of the addends' magnitudes.  The addends are x (16 + q) s and
    x (b - 16 s) for the affine codecs, x W otherwise."""
    x64 = x.double().numpy()
    K = x64.shape[1]
    W = oracle.dequant_q(codec, w, s, b)[0]
    out = x64 @ W.T
    if codec.startswith("affine"):
        gs = GROUPS[codec]
        s64 = np.abs(s[0].double().numpy()).repeat(gs, 1)
        b64 = np.abs(b[0].double().numpy()).repeat(gs, 1)
        mag = np.abs(x64) @ (47 * s64 + b64).T
    else:
        mag = np.abs(x64) @ np.abs(W).T
    if bias is not None:
        out = out + bias.double().numpy()
        mag = mag + np.abs(bias.double().numpy())
    return out, (80 + K / 16) * 2.0 ** -24 * mag


def softmax(z):
    m = z.max(-1, keepdims=True)
    with np.errstate(invalid="ignore"):
        e = np.where(np.isneginf(m), 0.0, np.exp(z - m))
    t = e.sum(-1, keepdims=True)
    return np.divide(e, t, out=np.zeros_like(e), where=t != 0)


def sigmoid(z):
    with np.errstate(over="ignore"):
        return 1 / (1 + np.exp(-z))


def route(z, k, bias, score, norm, scale):
    """(ids, weights) of fp64 logits: numbers before NaN, larger first, lower expert first."""
    p = (softmax if score == "softmax" else sigmoid)(z)
    key = z if bias is None else p + bias
    nan = np.isnan(key)
    key = np.where(nan, -np.inf, key)
    ids = np.empty((z.shape[0], k), np.int64)
    for t in range(z.shape[0]):
        ids[t] = sorted(range(z.shape[1]), key=lambda e: (nan[t, e], -key[t, e], e))[:k]
    c = np.take_along_axis(p, ids, -1)
    if norm and score == "softmax":
        c = softmax(np.take_along_axis(z, ids, -1))
    elif norm:
        t = c.sum(-1, keepdims=True)
        c = np.divide(c, t, out=np.zeros_like(c), where=t != 0)
    return ids, scale * c


def route_weights(z, ids, score, norm, scale):
    """The weights of given ids (-1: left out), for differences."""
    live = ids >= 0
    at = np.where(live, ids, 0)
    p = (softmax if score == "softmax" else sigmoid)(z)
    c = np.take_along_axis(p, at, -1) * live
    if norm:
        t = c.sum(-1, keepdims=True)
        c = np.divide(c, t, out=np.zeros_like(c), where=t != 0)
    return scale * c


def route_backward(z, ids, g, score, norm, scale):
    w = route_weights(z, ids, score, norm, scale)
    live = ids >= 0
    dot = np.where(live, w * g, 0).sum(-1, keepdims=True)
    p = (softmax if score == "softmax" else sigmoid)(z)
    dz = np.zeros_like(z)
    if score == "softmax" and not norm:
        dz -= p * dot
    for t, j in zip(*np.nonzero(live)):
        e = ids[t, j]
        v = g[t, j] - (dot[t, 0] / scale if norm else 0.0)
        dz[t, e] += w[t, j] * v * (1 - p[t, e] if score == "sigmoid" else 1.0)
    return dz


def balance(z, ids, coef, score, seqs, mask):
    """(loss [S], counts [S, E], tokens [S])."""
    R, E = z.shape
    T, k = R // seqs, ids.shape[1]
    p = softmax(z) if score == "softmax" else sigmoid(z) / sigmoid(z).sum(-1, keepdims=True)
    live = np.ones(R, bool) if mask is None else np.asarray(mask).astype(bool)
    loss, counts, tokens = np.zeros(seqs), np.zeros((seqs, E), np.int64), np.zeros(seqs, np.int64)
    for s in range(seqs):
        rows = [t for t in range(s * T, (s + 1) * T) if live[t]]
        tokens[s] = n = len(rows)
        for t in rows:
            for e in ids[t]:
                if 0 <= e < E:
                    counts[s, e] += 1
        if n:
            loss[s] = coef * E / (k * n) * (counts[s] * p[rows].sum(0) / n).sum()
    return loss, counts, tokens


def balance_backward(z, counts, tokens, dloss, k, coef, score, mask):
    R, E = z.shape
    S = counts.shape[0]
    T = R // S
    sg = sigmoid(z)
    p = softmax(z) if score == "softmax" else sg / sg.sum(-1, keepdims=True)
    dz = np.zeros_like(z)
    for t in range(R):
        s = t // T
        if tokens[s] == 0 or (mask is not None and not mask[t]):
            continue
        a = dloss[s] * coef * E * counts[s] / (k * float(tokens[s]) ** 2)
        dz[t] = p[t] * (a - (a * p[t]).sum())
        if score == "sigmoid":
            dz[t] *= 1 - sg[t]
    return dz
