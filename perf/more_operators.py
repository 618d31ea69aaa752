"""Measured cases of a mixture of experts around block-quantized weights: the residual's addition with the RMS norm and
its 8-bit rows, the routing of tokens to experts, the experts' gated products and the weighted sum of their last ones.

`run` computes a case in its plain form, from elementary torch operations, or, where `own` is true, through the library's
entry points (qmm_add_rmsnorm_quantize, qmm_route, qmm_experts_glu, qmm_experts_sum).

Weights are rows of blocks ([experts][N][row bytes]); activations meet them as 8-bit rows: 34-byte blocks of 32 values
with an f16 scale, or 292-byte blocks of 256 with an f32 scale, d = amax / 127, codes rne(x * (127 / amax)).
"""
import math
import random

import numpy as np
import torch

own = False

BLOCK = {"q4_0": (32, 18), "q8_0": (32, 34), "q4_1": (32, 20), "q5_0": (32, 22), "q5_1": (32, 24),
         "q4_K": (256, 144), "q5_K": (256, 176), "q6_K": (256, 210), "q2_K": (256, 84), "q8_K": (256, 292)}
WEIGHTS = ("q4_0", "q8_0", "q4_1", "q5_0", "q5_1", "q4_K", "q5_K", "q6_K", "q2_K")


def _row_bytes(t, K):
    values, size = BLOCK[t]
    return K // values * size


def _act(wtype):
    return "q8_K" if wtype.endswith("_K") else "q8_0"


# ---------------------------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # the norm between attention and the experts of one decoded token: latency only
        {"name": "norm_step", "kind": "norm", "tokens": 1, "K": 4096, "act": "q8_0", "normed": False},
        # the same for a 4096-token prompt, with the normed rows kept in f32 for a router of its own type
        {"name": "norm_prompt", "kind": "norm", "tokens": 4096, "K": 4096, "act": "q8_0", "normed": True},
        # an odd count of rows in the K-quants' activation format
        {"name": "norm_rows_K", "kind": "norm", "tokens": 1021, "K": 12288, "act": "q8_K", "normed": False},
        # the routing of a decode step of 4 sequences
        {"name": "route_step", "kind": "route", "tokens": 4, "experts": 64, "k": 8, "score": "softmax", "bias": False,
         "groups": 1, "kept": 1, "top": 1, "renorm": True, "scale": 1.0, "masked": False},
        # an 8192-token prompt: sigmoid scores, a bias for balance, 4 of 8 groups, some experts closed to some tokens
        {"name": "route_groups", "kind": "route", "tokens": 8192, "experts": 256, "k": 8, "score": "sigmoid", "bias": True,
         "groups": 8, "kept": 4, "top": 2, "renorm": True, "scale": 2.5, "masked": True},
        # one decoded token through 8 small experts
        {"name": "glu_token", "kind": "glu", "tokens": 1, "k": 8, "experts": 64, "N": 1024, "K": 2048, "type": "q4_K",
         "gate": "silu", "absent": False},
        # a serving batch over which most experts have a few tokens each
        {"name": "glu_batch", "kind": "glu", "tokens": 64, "k": 4, "experts": 32, "N": 1408, "K": 2048, "type": "q4_0",
         "gate": "silu", "absent": False},
        # odd sizes, tokens without some or all of their experts
        {"name": "glu_odd", "kind": "glu", "tokens": 333, "k": 3, "experts": 11, "N": 707, "K": 896, "type": "q5_1",
         "gate": "gelu", "absent": True},
        # a 2048-token prompt
        {"name": "glu_prompt", "kind": "glu", "tokens": 2048, "k": 8, "experts": 64, "N": 1024, "K": 2048, "type": "q4_K",
         "gate": "silu", "absent": False},
        # the last product of one decoded token
        {"name": "sum_token", "kind": "sum", "tokens": 1, "k": 8, "experts": 64, "N": 2048, "K": 1024, "type": "q6_K",
         "residual": True, "absent": False},
        # a batch with padding rows over few large experts
        {"name": "sum_batch", "kind": "sum", "tokens": 48, "k": 2, "experts": 8, "N": 4096, "K": 12288, "type": "q8_0",
         "residual": True, "absent": True},
        # a 2048-token prompt
        {"name": "sum_prompt", "kind": "sum", "tokens": 2048, "k": 8, "experts": 64, "N": 2048, "K": 1024, "type": "q6_K",
         "residual": True, "absent": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(("norm", "route", "glu", "glu", "sum", "sum"))
    if kind == "norm":
        act = rng.choice(("q8_0", "q8_K"))
        K = 256 * rng.randint(1, 48) if act == "q8_K" or rng.random() < 0.5 else 32 * rng.randint(1, 300)
        return {"kind": kind, "tokens": max(1, min(_log(rng, 1, 8000), (1 << 24) // K)), "K": K, "act": act,
                "normed": rng.random() < 0.5}
    if kind == "route":
        groups = rng.choice((1, 1, 2, 4, 8))
        experts = groups * rng.randint(4, max(5, 400 // groups))
        kept = rng.randint(1, groups)
        k = rng.randint(1, min(16, kept * (experts // groups)))
        return {"kind": kind, "tokens": max(1, min(_log(rng, 1, 8192), (1 << 21) // experts)), "experts": experts, "k": k,
                "score": rng.choice(("softmax", "sigmoid")), "bias": rng.random() < 0.5, "groups": groups, "kept": kept,
                "top": rng.choice((1, 2)), "renorm": rng.random() < 0.7, "scale": rng.choice((1.0, 2.5)),
                "masked": rng.random() < 0.3}
    typ = rng.choice(WEIGHTS)
    K = 256 * _log(rng, 1, 24) if _act(typ) == "q8_K" or rng.random() < 0.7 else 32 * rng.randint(2, 150)
    N, experts = _log(rng, 100, 4000), _log(rng, 1, 96)
    experts = max(1, min(experts, (1 << 28) // (N * K)))
    k = rng.randint(1, min(8, experts))
    tokens = max(1, min(_log(rng, 1, 2048), (1 << (35 if kind == "sum" else 34)) // (N * K * k)))
    case = {"kind": kind, "tokens": tokens, "k": k, "experts": experts, "N": N, "K": K, "type": typ,
            "absent": rng.random() < 0.3}
    if kind == "glu":
        case["gate"] = rng.choice(("silu", "silu", "gelu"))
    else:
        case["residual"] = rng.random() < 0.7
    return case


# --------------------------------------------------------------------------------------------------------------- inputs
def _half(x):
    return x.to(torch.float16).contiguous().view(torch.uint8).unflatten(-1, (-1, 2))


def _codes(gen, shape, mean, dev, lo, hi):
    x = torch.randn(shape, device="cuda", generator=gen).mul_(dev).add_(mean).round_().clamp_(lo, hi)
    return x.to(torch.int16) if lo < 0 and hi > 127 else x.to(torch.int8 if lo < 0 else torch.uint8)


def _whole(gen, shape, lo, hi):
    return torch.randint(lo, hi + 1, shape, device="cuda", generator=gen, dtype=torch.uint8)


def _nibbles(q):
    """Codes of the low nibbles' values and the high nibbles' into bytes."""
    return q[0] | (q[1] << 4)


def _weights(gen, typ, rows, K):
    """Rows of blocks as quantized weights have them: bell-shaped codes, scales that vary from block to block."""
    values, size = BLOCK[typ]
    n = rows * K // values
    w = torch.empty(n, size, dtype=torch.uint8, device="cuda")
    vary = torch.exp(0.3 * torch.randn(n, 1, device="cuda", generator=gen))
    if values == 32:
        top = 127 if typ == "q8_0" else 31 if typ[1] == "5" else 15
        d = vary * (0.06 / top)
        w[:, :2] = _half(d)[:, 0]
        if typ == "q8_0":
            w[:, 2:] = _codes(gen, (n, 32), 0.0, 40.0, -128, 127).view(torch.uint8)
            return w.view(rows, -1)
        at = 2
        if typ.endswith("1"):
            w[:, 2:4] = _half(d * (-0.5 * top))[:, 0]
            at = 4
        q = _codes(gen, (n, 32), 0.5 * top, 0.2 * top, 0, top)
        if typ[1] == "5":
            bits = (q >> 4).view(n, 4, 8) << torch.arange(8, device="cuda", dtype=torch.uint8)
            w[:, at: at + 4] = bits.sum(-1).to(torch.uint8)
            at += 4
            q = q & 15
        w[:, at:] = _nibbles((q[:, :16], q[:, 16:]))
        return w.view(rows, -1)
    if typ == "q6_K":
        q = _codes(gen, (n, 2, 4, 32), 32.0, 11.0, 0, 63)
        w[:, :128] = _nibbles((q[:, :, :2].flatten(2) & 15, q[:, :, 2:].flatten(2) & 15)).flatten(1)
        h = q >> 4
        w[:, 128:192] = (h[:, :, 0] | (h[:, :, 1] << 2) | (h[:, :, 2] << 4) | (h[:, :, 3] << 6)).flatten(1)
        w[:, 192:208] = _codes(gen, (n, 16), 0.0, 60.0, -128, 127).view(torch.uint8)
        w[:, 208:] = _half(vary * 2e-5)[:, 0]
        return w.view(rows, -1)
    if typ == "q2_K":
        sc, q = _whole(gen, (n, 16), 3, 15), _codes(gen, (n, 2, 4, 32), 1.5, 0.9, 0, 3)
        w[:, :16] = _nibbles((sc, sc))
        w[:, 16:80] = (q[:, :, 0] | (q[:, :, 1] << 2) | (q[:, :, 2] << 4) | (q[:, :, 3] << 6)).flatten(1)
        w[:, 80:82] = _half(vary * 2e-3)[:, 0]
        w[:, 82:] = _half(vary * 3e-3)[:, 0]
        return w.view(rows, -1)
    five = typ == "q5_K"
    top = 31 if five else 15
    sc, q = _whole(gen, (n, 8), 15, 63), _codes(gen, (n, 4, 2, 32), 0.5 * top, 0.2 * top, 0, top)
    mn = (sc.short() + _whole(gen, (n, 8), 0, 8).short() - 4).clamp_(0, 63).to(torch.uint8)
    w[:, :2] = _half(vary * (2e-3 / top))[:, 0]
    w[:, 2:4] = _half(vary * 1e-3)[:, 0]
    w[:, 4:8] = sc[:, :4] | ((sc[:, 4:] >> 4) << 6)
    w[:, 8:12] = mn[:, :4] | ((mn[:, 4:] >> 4) << 6)
    w[:, 12:16] = (sc[:, 4:] & 15) | ((mn[:, 4:] & 15) << 4)
    if five:
        shift = torch.arange(8, device="cuda", dtype=torch.uint8).view(4, 2, 1)
        w[:, 16:48] = ((q >> 4) << shift).sum((1, 2)).to(torch.uint8)
        q = q & 15
    w[:, size - 128:] = _nibbles((q[:, :, 0], q[:, :, 1])).flatten(1)
    return w.view(rows, -1)


def _rows(gen, n, K):
    """Activation rows: a few channels larger than the rest."""
    wide = 1.0 + 19.0 * (torch.rand(K, device="cuda", generator=gen) < 0.01).float()
    return torch.randn(n, K, device="cuda", generator=gen) * wide


def _picks(gen, rng, case):
    """The experts of each token (some experts are liked more than others), -1 where a token lacks one."""
    tokens, k, experts = case["tokens"], case["k"], case["experts"]
    like = torch.randn(tokens, experts, device="cuda", generator=gen) + 0.5 * torch.randn(experts, device="cuda", generator=gen)
    ids = like.topk(k, -1).indices.to(torch.int32)
    if case["absent"]:
        ids[torch.rand(tokens, k, device="cuda", generator=gen) < 0.1] = -1
        ids[rng.randrange(tokens)] = -1
    return ids.contiguous()


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    rng = random.Random(seed)
    kind, n, s = case["kind"], case["tokens"], {"case": case}
    if kind == "norm":
        K = case["K"]
        s["x"], s["r"] = _rows(gen, n, K), torch.randn(n, K, device="cuda", generator=gen)
        s["w"] = 1.0 + 0.2 * torch.randn(K, device="cuda", generator=gen)
        s["sum"], s["xq"] = torch.empty_like(s["x"]), torch.empty(n, _row_bytes(case["act"], K), dtype=torch.uint8, device="cuda")
        s["h"] = torch.empty_like(s["x"]) if case["normed"] else None
        s["all"], s["values"] = torch.arange(n, dtype=torch.int32, device="cuda"), torch.empty_like(s["x"])
        return s
    if kind == "route":
        s["logits"] = 1.5 * torch.randn(n, case["experts"], device="cuda", generator=gen)
        if case["masked"]:
            s["logits"][torch.rand(n, case["experts"], device="cuda", generator=gen) < 0.05] = -math.inf
            s["logits"][rng.randrange(n)] = -math.inf  # a padding token: no expert is open to it
        s["bias"] = 0.05 * torch.randn(case["experts"], device="cuda", generator=gen) if case["bias"] else None
        s["ids"] = torch.empty(n, case["k"], dtype=torch.int32, device="cuda")
        s["weights"] = torch.empty(n, case["k"], device="cuda")
        return s
    k, E, N, K = case["k"], case["experts"], case["N"], case["K"]
    s["ids"] = _picks(gen, rng, case)
    for name in ("gate", "up") if kind == "glu" else ("down",):
        s[name] = _weights(gen, case["type"], E * N, K).view(E, N, -1)
    if kind == "glu":
        s["xq"] = _quantize(_rows(gen, n, K), _act(case["type"]))
        s["h"] = torch.empty(n, k, N, device="cuda")
        return s
    s["h"] = _rows(gen, n * k, K).view(n, k, K)
    s["weights"] = torch.softmax(torch.randn(n, k, device="cuda", generator=gen), -1)
    s["residual"] = torch.randn(n, N, device="cuda", generator=gen) if case["residual"] else None
    s["y"] = torch.empty(n, N, device="cuda")
    return s


# --------------------------------------------------------------------------------------------------------- plain forms
def _quantize(x, act):
    """f32 rows into 8-bit rows, every step in f32.  Both quotients are of two tensors: a number as divisor or dividend
    would be turned into a product with a rounded reciprocal."""
    values, size = BLOCK[act]
    b = x.unflatten(-1, (-1, values))
    amax = b.abs().amax(-1, keepdim=True)
    most = torch.full_like(amax, 127.0)
    codes = torch.clamp(torch.round(b * torch.where(amax > 0, most / amax, torch.zeros_like(amax))), -128, 127).to(torch.int8)
    d = amax / most
    if act == "q8_0":
        parts = (d.to(torch.float16).view(torch.uint8), codes.view(torch.uint8))
    else:
        sums = codes.unflatten(-1, (16, 16)).sum(-1).to(torch.int16)
        parts = (d.view(torch.uint8), codes.view(torch.uint8), sums.view(torch.uint8))
    return torch.cat(parts, -1).flatten(-2)


def _values(xq, act):
    """The values that 8-bit rows stand for."""
    b = xq.unflatten(-1, (-1, BLOCK[act][1]))
    d = b[..., :2].contiguous().view(torch.float16).float() if act == "q8_0" else b[..., :4].contiguous().view(torch.float32)
    at = 2 if act == "q8_0" else 4
    return (b[..., at: at + BLOCK[act][0]].view(torch.int8).float() * d).flatten(-2)


def _dequantize(w, typ):
    """The values of rows of blocks, f32 [..., K]."""
    b = w.unflatten(-1, (-1, BLOCK[typ][1]))
    half = lambda at: b[..., at: at + 2].contiguous().view(torch.float16).float()  # noqa: E731
    if typ == "q8_0":
        return (b[..., 2:].view(torch.int8).float() * half(0)).flatten(-2)
    if typ == "q6_K":
        lo = b[..., :128].unflatten(-1, (2, 1, 64))
        q = torch.cat((lo & 15, lo >> 4), -2).unflatten(-1, (2, 32)).flatten(-3, -2)
        hi = (b[..., 128:192].unflatten(-1, (2, 1, 32)) >> torch.arange(0, 8, 2, device=w.device, dtype=torch.uint8).view(4, 1)) & 3
        sc = b[..., 192:208].view(torch.int8).float() * half(208)
        return ((q | (hi << 4)).float() - 32.0).flatten(-3).unflatten(-1, (16, 16)).mul(sc[..., None]).flatten(-3)
    if typ == "q2_K":
        q = (b[..., 16:80].unflatten(-1, (2, 1, 32)) >> torch.arange(0, 8, 2, device=w.device, dtype=torch.uint8).view(4, 1)) & 3
        sc = (b[..., :16] & 15).float() * half(80)
        mn = (b[..., :16] >> 4).float() * half(82)
        return (q.float().flatten(-3).unflatten(-1, (16, 16)) * sc[..., None] - mn[..., None]).flatten(-3)
    if typ in ("q4_K", "q5_K"):
        x, y, z = b[..., 4:8], b[..., 8:12], b[..., 12:16]
        sc = torch.cat((x & 63, (z & 15) | ((x >> 6) << 4)), -1).float() * half(0)
        mn = torch.cat((y & 63, (z >> 4) | ((y >> 6) << 4)), -1).float() * half(2)
        lo = b[..., -128:].unflatten(-1, (4, 1, 32))
        q = torch.cat((lo & 15, lo >> 4), -2).flatten(-3, -2)
        if typ == "q5_K":
            q = q | (((b[..., None, 16:48] >> torch.arange(8, device=w.device, dtype=torch.uint8).view(8, 1)) & 1) << 4)
        return (q.float() * sc[..., None] - mn[..., None]).flatten(-3)
    q = torch.cat((b[..., -16:] & 15, b[..., -16:] >> 4), -1)
    if typ[1] == "5":
        at = 4 if typ == "q5_1" else 2
        bits = (b[..., at: at + 4, None] >> torch.arange(8, device=w.device, dtype=torch.uint8)) & 1
        q = q | (bits.flatten(-2) << 4)
    if typ.endswith("1"):
        return (q.float() * half(0) + half(2)).flatten(-2)
    return ((q.float() - (16.0 if typ == "q5_0" else 8.0)) * half(0)).flatten(-2)


def _experts(ws, typ, x, ids):
    """x[slot] through each w[ids[slot]] of `ws`, f32 [slots][N] each, for slots whose id is not negative (others: zeros).
    Few slots take their experts' weights one by one; many are sorted into equal rooms, one for each expert."""
    E, slots = ws[0].shape[0], ids.numel()
    real = ids >= 0
    e = torch.where(real, ids, 0).long()
    if slots <= E:
        got = [torch.matmul(_dequantize(w[e], typ), x[:, :, None])[..., 0] for w in ws]
    else:
        e = torch.where(real, e, E)  # a room behind the last expert's
        order = torch.sort(e, stable=True).indices
        counts = torch.bincount(e, minlength=E + 1)
        place = torch.empty_like(order)
        place[order] = torch.arange(slots, device="cuda") - (torch.cumsum(counts, 0) - counts)[e[order]]
        rooms = torch.zeros(E + 1, int(counts.max()), x.shape[1], device="cuda")
        rooms[e, place] = x
        got = [torch.matmul(rooms[:E], _dequantize(w, typ).transpose(1, 2))[e.clamp(max=E - 1), place] for w in ws]
    return [torch.where(real[:, None], y, torch.zeros((), device="cuda")) for y in got]


def _plain_norm(s):
    case = s["case"]
    y = s["x"] + s["r"]
    K = torch.full((y.shape[0], 1), float(case["K"]), device="cuda")
    mean = y.double().square().sum(-1, keepdim=True).float() / K  # long sums, and values next to a code's border
    h = (y * (torch.ones_like(mean) / torch.sqrt(mean + 1e-5))) * s["w"]
    out = (y, _values(_quantize(h, case["act"]), case["act"]))
    return out + (h,) if case["normed"] else out


def _plain_route(s):
    case, x = s["case"], s["logits"].double()  # the choice: values next to a border
    present = x > -math.inf
    if case["score"] == "softmax":
        e = torch.where(present, torch.exp(x - x.amax(-1, keepdim=True)), 0.0)
        score = e / e.sum(-1, keepdim=True)
    else:
        score = 1.0 / (1.0 + torch.exp(-x))
    key = score if s["bias"] is None else score + s["bias"].double()
    key = torch.where(present, key, -math.inf)
    by = key.unflatten(-1, (case["groups"], -1))
    if case["groups"] > 1:
        best = torch.sort(by, dim=-1, descending=True).values[..., : case["top"]]
        worth = torch.where(best > -math.inf, best, 0.0).sum(-1)
        worth = torch.where(best[..., 0] > -math.inf, worth, -math.inf)
        keep = torch.sort(worth, dim=-1, descending=True, stable=True).indices[:, : case["kept"]]
        open_ = torch.zeros_like(worth, dtype=torch.bool).scatter_(1, keep, True)
        by = torch.where(open_[..., None], by, -math.inf)
    top = torch.sort(by.flatten(1), dim=-1, descending=True, stable=True)
    ids, there = top.indices[:, : case["k"]], top.values[:, : case["k"]] > -math.inf
    w = torch.where(there, score.gather(1, ids), 0.0)
    if case["renorm"]:
        total = w.sum(-1, keepdim=True)
        w = w / torch.where(total > 0, total, 1.0)
    return torch.where(there, ids, -1).to(torch.int32), (w * case["scale"]).float()


def _plain_glu(s):
    case, ids = s["case"], s["ids"].flatten()
    x = _values(s["xq"], _act(case["type"])).repeat_interleave(case["k"], 0)
    g, u = _experts((s["gate"], s["up"]), case["type"], x, ids)
    if case["gate"] == "silu":
        g = g / (1.0 + torch.exp(-g))
    else:
        g = 0.5 * g * (1.0 + torch.tanh(0.7978845608028654 * (g + 0.044715 * g * g * g)))
    return (g * u).view(case["tokens"], case["k"], -1)


def _plain_sum(s):
    case = s["case"]
    act = _act(case["type"])
    x = _values(_quantize(s["h"].flatten(0, 1), act), act)
    y = _experts((s["down"],), case["type"], x, s["ids"].flatten())[0].view(case["tokens"], case["k"], -1)
    y = (y * s["weights"][..., None]).sum(1)
    return y if s["residual"] is None else s["residual"] + y


# ------------------------------------------------------------------------------------------------- the library's calls
def _handles(s):
    """What a program sets up once and keeps: the workspace of the experts' calls."""
    import block_quantized_weight_q8_gb300 as qmm

    case, h = s["case"], {"qmm": qmm}
    if case["kind"] in ("glu", "sum"):
        h["bytes"] = qmm.qmm_experts_scratch_bytes(case["type"], case["tokens"], case["k"], case["experts"], case["N"], case["K"])
        h["scratch"] = torch.empty(h["bytes"], dtype=torch.uint8, device="cuda")
    return h


def _own(s):
    if "handles" not in s:
        s["handles"] = _handles(s)
    case, h = s["case"], s["handles"]
    qmm, kind = h["qmm"], case["kind"]
    if kind == "norm":
        qmm.qmm_add_rmsnorm_quantize(case["act"], s["x"], s["r"], s["w"], 1e-5, s["xq"], sum=s["sum"], h=s["h"])
        if case["act"] == "q8_0":
            qmm.qmm_get_rows("q8_0", s["xq"], s["all"], s["values"], case["tokens"], case["tokens"], case["K"])
            out = (s["sum"], s["values"])
        else:
            out = (s["sum"], _values(s["xq"], case["act"]))
        return out + (s["h"],) if case["normed"] else out
    if kind == "route":
        qmm.qmm_route(s["logits"], s["ids"], s["weights"], score=case["score"], bias=s["bias"], groups=case["groups"],
                      groups_kept=case["kept"], group_top=case["top"], renorm=case["renorm"], scale=case["scale"])
        return s["ids"], s["weights"]
    if kind == "glu":
        qmm.qmm_experts_glu(case["type"], s["gate"], s["up"], s["xq"], s["ids"], s["h"], h["scratch"], h["bytes"],
                            gate=case["gate"])
        return s["h"]
    qmm.qmm_experts_sum(case["type"], s["down"], s["h"], s["ids"], s["weights"], s["y"], h["scratch"], h["bytes"],
                        residual=s["residual"])
    return s["y"]


def run(state):
    if own:
        return _own(state)
    return {"norm": _plain_norm, "route": _plain_route, "glu": _plain_glu, "sum": _plain_sum}[state["case"]["kind"]](state)


# ---------------------------------------------------------------------------------------------------------- what it costs
def work(case):
    kind, n = case["kind"], case["tokens"]
    if kind == "norm":
        K = case["K"]
        return {"bytes": n * (12 * K + _row_bytes(case["act"], K) + (4 * K if case["normed"] else 0)) + 4 * K, "flops": 8 * n * K}
    if kind == "route":
        return {"bytes": n * (4 * case["experts"] + 8 * case["k"]), "flops": 10 * n * case["experts"]}
    k, E, N, K = case["k"], case["experts"], case["N"], case["K"]
    legs = 2 if kind == "glu" else 1
    used = E * (1.0 - (1.0 - k / E) ** n)  # experts that at least one token takes, where all are liked alike
    bytes_ = used * legs * N * _row_bytes(case["type"], K) + 4 * n * k
    if kind == "glu":
        bytes_ += n * _row_bytes(_act(case["type"]), K) + 4 * n * k * N
    else:
        bytes_ += 4 * n * k * (K + 1) + 4 * n * N * (2 if case["residual"] else 1)
    return {"bytes": bytes_, "flops": 2 * legs * n * k * N * K}


# ------------------------------------------------------------------------------------------- the definitions, in 64 bits
def _bits(word, at, count):
    return (word >> at) & ((1 << count) - 1)


def _exact_rows(raw, typ):
    """The values of rows of blocks in 64 bits, field by field: value j of a block from the bytes that hold it."""
    values, size = BLOCK[typ]
    b = raw.reshape(raw.shape[0], -1, size).long()
    f16 = lambda at: raw.reshape(raw.shape[0], -1, size)[:, :, at: at + 2].contiguous().view(torch.float16).double()  # noqa: E731
    out = torch.empty(b.shape[0], b.shape[1], values, dtype=torch.float64, device=raw.device)
    signed = lambda v: torch.where(v > 127, v - 256, v)  # noqa: E731
    if typ == "q8_0":
        return (signed(b[:, :, 2:]).double() * f16(0)).flatten(1)
    if values == 32:
        first = {"q4_0": 2, "q4_1": 4, "q5_0": 6, "q5_1": 8}[typ]
        for j in range(32):
            q = _bits(b[:, :, first + j % 16], 4 * (j // 16), 4)
            if typ[1] == "5":
                q = q + 16 * _bits(b[:, :, first - 4 + j // 8], j % 8, 1)
            off = {"q4_0": 8, "q5_0": 16}.get(typ, 0)
            out[:, :, j] = f16(0)[:, :, 0] * (q - off) + (f16(2)[:, :, 0] if typ.endswith("1") else 0.0)
        return out.flatten(1)
    for s in range(8):  # 32 values at a time
        at = slice(32 * s, 32 * s + 32)
        if typ == "q6_K":
            half, part = s // 4, s % 4
            lo = _bits(b[:, :, 64 * half + 32 * (part % 2): 64 * half + 32 * (part % 2) + 32], 4 * (part // 2), 4)
            q = lo + 16 * _bits(b[:, :, 128 + 32 * half: 160 + 32 * half], 2 * part, 2) - 32
            sc = signed(b[:, :, 192 + 2 * s: 194 + 2 * s]).double().repeat_interleave(16, -1)
            out[:, :, at] = f16(208) * sc * q
        elif typ == "q2_K":
            q = _bits(b[:, :, 16 + 32 * (s // 4): 48 + 32 * (s // 4)], 2 * (s % 4), 2)
            two = b[:, :, 2 * s: 2 * s + 2].repeat_interleave(16, -1)
            out[:, :, at] = f16(80) * (two & 15) * q - f16(82) * (two >> 4)
        else:
            q = _bits(b[:, :, size - 128 + 32 * (s // 2): size - 96 + 32 * (s // 2)], 4 * (s % 2), 4)
            if typ == "q5_K":
                q = q + 16 * _bits(b[:, :, 16:48], s, 1)
            if s < 4:
                sc, mn = b[:, :, 4 + s] & 63, b[:, :, 8 + s] & 63
            else:
                sc = (b[:, :, 8 + s] & 15) + 16 * (b[:, :, s] >> 6)
                mn = (b[:, :, 8 + s] >> 4) + 16 * (b[:, :, 4 + s] >> 6)
            out[:, :, at] = f16(0) * sc[..., None] * q - f16(2) * mn[..., None]
    return out.flatten(1)


def _exact_held(x, act):
    """The values that f32 rows have once they are held in 8 bits: the rule's rounding steps (numpy)."""
    b = x.reshape(x.shape[0], -1, BLOCK[act][0])
    amax = np.abs(b).max(-1, keepdims=True)
    with np.errstate(divide="ignore"):
        inv = np.where(amax > 0, np.float32(127) / amax, np.float32(0)).astype(np.float32)
    codes = np.clip(np.rint((b * inv).astype(np.float32)), -128, 127).astype(np.float64)
    d = (amax / np.float32(127)).astype(np.float32)
    if act == "q8_0":
        d = d.astype(np.float16)
    return (codes * d.astype(np.float64)).reshape(x.shape)


def _exact_route(s):
    case, logits = s["case"], s["logits"].cpu().numpy().astype(np.float64)
    bias = np.zeros(case["experts"]) if s["bias"] is None else s["bias"].cpu().numpy().astype(np.float64)
    each = case["experts"] // case["groups"]
    weights = np.zeros((case["tokens"], case["k"]))
    for t, x in enumerate(logits):
        live = [e for e in range(case["experts"]) if x[e] > -np.inf]
        if not live:
            continue
        if case["score"] == "softmax":
            top = max(x[e] for e in live)
            total = sum(math.exp(x[e] - top) for e in live)
            score = {e: math.exp(x[e] - top) / total for e in live}
        else:
            score = {e: 1.0 / (1.0 + math.exp(-x[e])) for e in live}
        if case["groups"] > 1:
            worth = []
            for g in range(case["groups"]):
                keys = sorted((score[e] + bias[e] for e in live if e // each == g), reverse=True)
                if keys:
                    worth.append((-sum(keys[: case["top"]]), g))
            kept = {g for _, g in sorted(worth)[: case["kept"]]}
            live = [e for e in live if e // each in kept]
        chosen = sorted((-(score[e] + bias[e]), e) for e in live)[: case["k"]]
        w = np.array([score[e] for _, e in chosen])
        weights[t, : len(w)] = (w / w.sum() if case["renorm"] and w.sum() > 0 else w) * case["scale"]
    return None, weights


def exact(case, seed):
    s = prepare(case, seed)
    if case["kind"] == "norm":
        y = (s["x"].cpu().numpy() + s["r"].cpu().numpy()).astype(np.float32)
        mean = (y.astype(np.float64) ** 2).sum(-1, keepdims=True).astype(np.float32) / np.float32(case["K"])
        scale = np.float32(1) / np.sqrt(mean + np.float32(1e-5))
        h = ((y * scale) * s["w"].cpu().numpy()).astype(np.float32)
        out = (s["x"].double() + s["r"].double(), _exact_held(h, case["act"]))
        if not case["normed"]:
            return out
        full = y.astype(np.float64)
        h = full / np.sqrt((full ** 2).mean(-1, keepdims=True) + 1e-5) * s["w"].cpu().numpy().astype(np.float64)
        return out + (h,)
    if case["kind"] == "route":
        return _exact_route(s) if case["tokens"] * case["experts"] <= 1 << 22 else None
    n, k, N, K = case["tokens"], case["k"], case["N"], case["K"]
    act, ids = _act(case["type"]), s["ids"].flatten().cpu().numpy()
    if case["kind"] == "glu":
        b = s["xq"].cpu().numpy().reshape(n, -1, BLOCK[act][1])
        at = 2 if act == "q8_0" else 4
        d = np.ascontiguousarray(b[:, :, :at]).view(np.float16 if at == 2 else np.float32).astype(np.float64)
        x = np.ascontiguousarray(b[:, :, at: at + BLOCK[act][0]]).view(np.int8).astype(np.float64) * d
        x = torch.from_numpy(x.reshape(n, K)).cuda()
        h = torch.zeros(n * k, N, dtype=torch.float64, device="cuda")
    else:
        x = torch.from_numpy(_exact_held(s["h"].flatten(0, 1).cpu().numpy(), act)).cuda()
        h = torch.zeros(n * k, N, dtype=torch.float64, device="cuda")
    for e in np.unique(ids[ids >= 0]):
        at = torch.from_numpy(np.flatnonzero(ids == e)).cuda()
        if case["kind"] == "glu":
            g = x[at // k] @ _exact_rows(s["gate"][e], case["type"]).T
            u = x[at // k] @ _exact_rows(s["up"][e], case["type"]).T
            if case["gate"] == "silu":
                g = g / (1.0 + torch.exp(-g))
            else:
                g = 0.5 * g * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (g + 0.044715 * g ** 3)))
            h[at] = g * u
        else:
            h[at] = x[at] @ _exact_rows(s["down"][e], case["type"]).T
    if case["kind"] == "glu":
        return h.view(n, k, N)
    y = (h.view(n, k, N) * s["weights"].double()[..., None]).sum(1)
    return y if s["residual"] is None else y + s["residual"].double()
