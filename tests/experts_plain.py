"""The mixture-of-experts operators' definitions in 64 bits (numpy), for the tests: the added norm, the choice of experts,
the gated and the summed products."""
import math

import numpy as np

import oracle

EPS = 1e-6
# a product is within this share of its row's L2 norm (the library's bound for every multiply)
PRODUCT = 1e-5


def act_of(wtype):
    return "q8_K" if wtype.endswith("_K") else "q8_0"


def add_norm(act, x, r, w, eps):
    """(y, h, the rows' bytes): every step in f32 but the sum of squares, taken in 64 bits and rounded once."""
    y = (x + r).astype(np.float32)
    ss = (y.astype(np.float64) ** 2).sum(-1, keepdims=True).astype(np.float32)
    s = np.float32(1) / np.sqrt((ss / np.float32(x.shape[-1])).astype(np.float32) + np.float32(eps))
    h = ((y * s.astype(np.float32)).astype(np.float32) * w).astype(np.float32)
    return y, h, oracle.quantize(act, h)


def route(logits, bias, k, score="softmax", groups=1, kept=1, top=1, renorm=True, scale=1.0):
    """(ids, weights in 64 bits) by sorting each token's open experts."""
    T, E = logits.shape
    each = E // groups
    ids, weights = np.full((T, k), -1, np.int32), np.zeros((T, k))
    most = float(np.finfo(np.float32).max)
    for t in range(T):
        live = {e: min(float(v), most) for e, v in enumerate(logits[t]) if v > -np.inf}
        if not live:
            continue
        m = max(live.values())
        if score == "softmax":
            total = math.fsum(math.exp(v - m) for v in live.values())
            s = {e: math.exp(v - m) / total for e, v in live.items()}
        else:
            s = {e: 1.0 / (1.0 + math.exp(-v)) if v > -700 else 0.0 for e, v in live.items()}
        if bias is None and (groups == 1 or top == 1):
            key = dict(live)
        else:
            key = {e: s[e] + (0.0 if bias is None else float(bias[e])) for e in live}
            key = {e: c for e, c in key.items() if c > -np.inf}
        if groups > 1:
            worth = []
            for g in range(groups):
                c = sorted((key[e] for e in key if e // each == g), reverse=True)
                if c:
                    worth.append((-sum(c[:top]), g))
            open_ = {g for _, g in sorted(worth)[:kept]}
            key = {e: c for e, c in key.items() if e // each in open_}
        chosen = [e for _, e in sorted((-c, e) for e, c in key.items())[:k]]
        w = np.array([s[e] for e in chosen])
        if renorm and w.sum() > 0:
            w = w / w.sum()
        ids[t, :len(chosen)], weights[t, :len(chosen)] = chosen, w * scale
    return ids, weights


def gate_of(kind, g):
    if kind == "silu":
        return g / (1 + np.exp(-np.clip(g, -700, None)))
    return 0.5 * g * (1 + np.tanh(math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3)))


def glu(wtype, Wg, Wu, xq, ids, kind, K):
    """(h, the error it may have) of byte arrays Wg, Wu [E][N][rb] and xq [T][rb]."""
    E, N = Wg.shape[:2]
    x = oracle.dequantize(act_of(wtype), xq, K)
    T, k = ids.shape
    h, off = np.zeros((T, k, N)), np.zeros((T, k, N))
    for e in np.unique(ids[(ids >= 0) & (ids < E)]):
        t, j = np.nonzero(ids == e)
        g = x[t] @ oracle.dequantize(wtype, Wg[e], K).T
        u = x[t] @ oracle.dequantize(wtype, Wu[e], K).T
        a = gate_of(kind, g)
        dg, du = (PRODUCT * np.linalg.norm(v, axis=-1, keepdims=True) for v in (g, u))
        h[t, j] = a * u
        # |gate'| is at most 1.13; the gate itself: the exponential's 2 units of 2^-23 and four roundings, on |g| at most,
        # and for gelu its argument's roundings (|z| e^-|z| |g| stays below |g|)
        off[t, j] = 1.13 * dg * np.abs(u) + np.abs(a) * du + 1.2 * dg * du + 2.0 ** -20 * np.abs(g * u)
    return h, off


def summed(wtype, W, h, ids, weights, residual, K):
    """(y, the error it may have): rows h f32 [T][k][K] quantized by the activations' rule."""
    E, N = W.shape[:2]
    T, k = ids.shape
    y, off, size = np.zeros((T, N)), np.zeros((T, N)), np.zeros((T, N))
    w = np.ones((T, k)) if weights is None else weights.astype(np.float64)
    for e in np.unique(ids[(ids >= 0) & (ids < E)]):
        t, j = np.nonzero(ids == e)
        x = oracle.dequantize(act_of(wtype), oracle.quantize(act_of(wtype), np.ascontiguousarray(h[t, j])), K)
        p = x @ oracle.dequantize(wtype, W[e], K).T
        np.add.at(y, t, p * w[t, j][:, None])
        np.add.at(size, t, np.abs(p * w[t, j][:, None]))
        np.add.at(off, t, np.abs(w[t, j])[:, None] * PRODUCT * np.linalg.norm(p, axis=-1, keepdims=True))
    if residual is not None:
        y, size = y + residual, size + np.abs(residual)
    return y, off + (k + 2) * 2.0 ** -24 * size
