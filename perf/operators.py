"""Measured cases of the operators around a paged key-value cache: rotary positions, keys and values stored into pages
(and read back), and the attention of one new token over the pages.

`run` computes a case in its plain form, from elementary torch operations, or, where `own` is true, through the library's
entry points (qmm_rope, qmm_kv_store, qmm_kv_load, qmm_kv_attend).

A page holds `page` positions of every KV head: the codes of (head h, position o) at (h * page + o) * row bytes, and for
the 8-bit type the f32 scales behind all codes, at Hkv * page * hd + 4 * (h * page + o).  A sequence's position p lies in
page table[seq][p // page] at o = p % page.  8-bit rows: d = amax / 127, codes rne(x * (127 / amax)), every step in f32.
Rotary frequencies are turns per position as 64-bit fractions of a turn: the angle of position p and pair i is
2 pi * frac(p * F[i] / 2^64).
"""
import math
import random

import numpy as np
import torch

own = False

TURN = 2.0 ** 64


# ---------------------------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # the query heads of a decode step of 16 sequences, far into a context stretched by wavelength bands
        {"name": "rope_step", "kind": "rope", "tokens": 16, "heads": 32, "hd": 128, "n_rot": 128, "layout": "half",
         "scaling": "bands", "far": 131072, "inverse": False},
        # the query heads of a 4096-token prompt, neighbouring values paired
        {"name": "rope_prompt", "kind": "rope", "tokens": 4096, "heads": 32, "hd": 128, "n_rot": 128,
         "layout": "interleaved", "scaling": "plain", "far": 4096, "inverse": False},
        # the gradient of a rotation of part of each head, odd token count
        {"name": "rope_grad_part", "kind": "rope", "tokens": 2047, "heads": 28, "hd": 96, "n_rot": 64, "layout": "half",
         "scaling": "yarn", "far": 65536, "inverse": True},
        # one decode step of 64 sequences: queries and keys rotated, keys and values stored; what was stored read back
        {"name": "store_step", "kind": "store", "tokens": 64, "seqs": 64, "Hq": 32, "Hkv": 8, "hd": 128, "n_rot": 128,
         "layout": "half", "type": "q8", "page": 16, "far": 4096, "pad": 3},
        # an 8192-token prefill batch of three sequences, stored and read back
        {"name": "store_prompt", "kind": "store", "tokens": 8192, "seqs": 3, "Hq": 0, "Hkv": 8, "hd": 128, "n_rot": 128,
         "layout": "half", "type": "q8", "page": 16, "far": 8192, "pad": 0},
        # odd sizes: 5 heads of 80, half of each rotated, a 16-bit cache, padding tokens
        {"name": "store_f16_odd", "kind": "store", "tokens": 1021, "seqs": 7, "Hq": 20, "Hkv": 5, "hd": 80, "n_rot": 40,
         "layout": "interleaved", "type": "f16", "page": 32, "far": 2000, "pad": 13},
        # the cached prefix of one long sequence read back for a prefill that continues it
        {"name": "load_prefix", "kind": "load", "tokens": 32768, "seqs": 1, "Hkv": 8, "hd": 128, "type": "q8", "page": 16,
         "far": 32768, "pad": 0},
        # the first tokens of one small-model request: latency only
        {"name": "attend_first", "kind": "attend", "rows": 1, "longest": 33, "Hq": 14, "Hkv": 2, "hd": 64, "type": "q8",
         "page": 16, "window": 0},
        # one sequence at a 4096-position context
        {"name": "attend_4096", "kind": "attend", "rows": 1, "longest": 4096, "Hq": 32, "Hkv": 8, "hd": 128, "type": "q8",
         "page": 16, "window": 0},
        # a serving batch: 64 ragged sequences, one of them empty and one a padding row
        {"name": "attend_batch", "kind": "attend", "rows": 64, "longest": 8192, "Hq": 32, "Hkv": 8, "hd": 128,
         "type": "q8", "page": 16, "window": 0},
        # two long documents
        {"name": "attend_long", "kind": "attend", "rows": 2, "longest": 131072, "Hq": 64, "Hkv": 8, "hd": 128,
         "type": "q8", "page": 64, "window": 0},
        # a 16-bit cache with wide heads and a sliding window, no sharing of heads
        {"name": "attend_f16_window", "kind": "attend", "rows": 32, "longest": 20000, "Hq": 8, "Hkv": 8, "hd": 256,
         "type": "f16", "page": 32, "window": 1024},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(("rope", "store", "load", "attend", "attend"))
    hd = rng.choice((16, 48, 64, 80, 96, 112, 128, 128, 192, 256))
    if kind == "rope":
        n_rot = rng.choice((hd, hd, hd // 2, hd // 4))
        tokens, heads = _log(rng, 1, 6000), rng.randint(1, 40)
        tokens = max(1, min(tokens, (1 << 24) // (heads * hd)))
        return {"kind": kind, "tokens": tokens, "heads": heads, "hd": hd, "n_rot": n_rot,
                "layout": rng.choice(("half", "interleaved")), "scaling": rng.choice(("plain", "linear", "bands", "yarn")),
                "far": max(tokens, _log(rng, 100, 1000000)), "inverse": rng.random() < 0.5}
    hkv, typ, page = rng.randint(1, 10), rng.choice(("q8", "q8", "f16")), rng.choice((8, 16, 16, 32, 64, 128))
    if kind == "attend":
        rows, longest = _log(rng, 1, 100), _log(rng, 1, 100000)
        row = hkv * 2 * (hd + 4 if typ == "q8" else 2 * hd)
        longest = max(1, min(longest, 200000000 // (rows * row)))
        return {"kind": kind, "rows": rows, "longest": longest, "Hq": hkv * rng.randint(1, 8), "Hkv": hkv, "hd": hd,
                "type": typ, "page": page, "window": rng.choice((0, 0, _log(rng, 1, 4096)))}
    tokens = max(1, min(_log(rng, 1, 30000), (1 << 23) // (hkv * hd)))
    seqs = rng.randint(1, min(tokens, 50))
    case = {"kind": kind, "tokens": tokens, "seqs": seqs, "Hkv": hkv, "hd": hd, "type": typ, "page": page,
            "far": -(-tokens // seqs) + _log(rng, 1, 5000), "pad": min(tokens - 1, rng.choice((0, 1, 9)))}
    if kind == "store":
        case["n_rot"] = rng.choice((0, hd, hd, hd // 2))
        case["Hq"] = hkv * rng.randint(1, 4) if case["n_rot"] and rng.random() < 0.5 else 0
        case["layout"] = rng.choice(("half", "interleaved"))
    return case


# --------------------------------------------------------------------------------------------------------------- inputs
def _row_bytes(case):
    return case["hd"] + 4 if case["type"] == "q8" else 2 * case["hd"]


def _page_bytes(case):
    return case["page"] * case["Hkv"] * _row_bytes(case)


def _scaled(n_rot, scaling, base=10000.0):
    """The angles per position, in radians, of the n_rot / 2 pairs, in 64 bits."""
    i = np.arange(n_rot // 2, dtype=np.float64)
    f = base ** (-2.0 * i / n_rot)
    if scaling == "linear":        # every position divided by 4
        return f / 4.0
    if scaling == "bands":         # factor 8 below 1 turn in 8192 positions, none above 4, blended between
        keep = np.clip((8192.0 * f / (2 * math.pi) - 1.0) / (4.0 - 1.0), 0.0, 1.0)
        return (1 - keep) * f / 8.0 + keep * f
    if scaling == "yarn":          # factor 16 by pair index, between the pairs that turn 32 times and once in 4096
        at = lambda turns: n_rot * math.log(4096.0 / (turns * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
        lo, hi = max(math.floor(at(32.0)), 0), min(math.ceil(at(1.0)), n_rot - 1)
        keep = 1 - np.clip((i - lo) / max(hi - lo, 0.001), 0.0, 1.0)
        return (1 - keep) * f / 16.0 + keep * f
    return f


def _turns(n_rot, scaling):
    """The frequency table a program keeps: turns per position as 64-bit fractions."""
    whole = [int(t * TURN) % (1 << 64) for t in _scaled(n_rot, scaling) / (2 * math.pi)]
    return torch.tensor([w - (1 << 64) if w >> 63 else w for w in whole], dtype=torch.int64, device="cuda")


def _mscale(case):
    return float(np.float32(0.1 * math.log(16.0) + 1.0)) if case.get("scaling") == "yarn" else 1.0


def _lens(case):
    """The sequences' lengths: ragged, one empty and one padding row among many."""
    n, longest = case["rows"], case["longest"]
    lens = [max(1, int(longest * ((i + 1) / n) ** 2)) for i in range(n)]
    if n >= 8:
        lens[0], lens[1] = 0, -1
    return lens


def _key_rows(gen, n, hkv, hd):
    """Keys as they come: a few channels larger than the rest."""
    wide = 1.0 + 5.0 * (torch.rand(hkv, hd, device="cuda", generator=gen) < 0.03).float()
    return torch.randn(n, hkv, hd, device="cuda", generator=gen) * wide


def _quantize(x):
    """8-bit rows over the last dimension, every step in f32.  Both quotients are of two tensors: a number as divisor or
    dividend would be turned into a product with a rounded reciprocal."""
    amax = x.abs().amax(-1, keepdim=True)
    most = torch.full_like(amax, 127.0)
    inv = torch.where(amax > 0, most / amax, torch.zeros_like(amax))
    return torch.clamp(torch.round(x * inv), -128, 127).to(torch.int8), (amax / most).squeeze(-1)


def _planes(pool, case):
    """Views of a pool's pages: codes [pages][Hkv][page][hd] and, for the 8-bit type, scales [pages][Hkv][page]."""
    n, hkv, page, hd = pool.shape[0], case["Hkv"], case["page"], case["hd"]
    if case["type"] == "f16":
        return pool[:, : hkv * page * hd * 2].view(torch.float16).unflatten(1, (hkv, page, hd)), None
    cut = hkv * page * hd
    return (pool[:, :cut].view(torch.int8).unflatten(1, (hkv, page, hd)),
            pool[:, cut: cut + 4 * hkv * page].view(torch.float32).unflatten(1, (hkv, page)))


def _fill(pool, case, page, off, x):
    """Writes rows x [n][Hkv][hd] into (page, off) of a pool."""
    codes, scales = _planes(pool, case)
    if case["type"] == "f16":
        codes[page, :, off] = x.to(torch.float16)
    else:
        c, d = _quantize(x)
        codes[page, :, off] = c
        scales[page, :, off] = d


def _pools(case, gen, seqs, most):
    """Keys' and values' pools (the two halves of one buffer's pages) with a shuffled table of `most` positions per
    sequence.  What no position has been written to holds whatever was there: here bytes that read as NaN."""
    pages = -(-most // case["page"])
    total = seqs * pages + 3
    stride = -(-_page_bytes(case) // 16) * 16
    both = torch.full((total, 2, stride), 0xFF, dtype=torch.uint8, device="cuda")
    table = torch.randperm(total, device="cuda", generator=gen)[: seqs * pages].to(torch.int32).view(seqs, pages)
    return both[:, 0], both[:, 1], table.contiguous()


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    rng = random.Random(seed)
    kind, hd = case["kind"], case["hd"]
    s = {"case": case}
    if kind == "rope":
        s["x"] = torch.randn(case["tokens"], case["heads"], hd, device="cuda", generator=gen)
        s["pos"] = torch.randint(0, case["far"], (case["tokens"],), device="cuda", generator=gen).to(torch.int32)
        s["freqs"] = _turns(case["n_rot"], case["scaling"])
        s["out"] = torch.zeros_like(s["x"])
        return s
    hkv, page = case["Hkv"], case["page"]
    if kind == "attend":
        lens = _lens(case)
        rng.shuffle(lens)
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        s["longest"] = max(lens)
        s["k"], s["v"], s["table"] = _pools(case, gen, case["rows"], max(lens))
        for r, n in enumerate(lens):
            if n > 0:
                p = torch.arange(n, device="cuda")
                at = s["table"][r, p // page].long()
                _fill(s["k"], case, at, p % page, _key_rows(gen, n, hkv, hd))
                _fill(s["v"], case, at, p % page, torch.randn(n, hkv, hd, device="cuda", generator=gen))
        s["q"] = torch.randn(case["rows"], case["Hq"], hd, device="cuda", generator=gen)
        s["out"] = torch.zeros_like(s["q"])
        s["lse"] = torch.zeros(case["rows"], case["Hq"], device="cuda")
        return s
    # tokens of several sequences, each a run of neighbouring positions; the last `pad` tokens are padding
    n, seqs = case["tokens"] - case["pad"], case["seqs"]
    each = [n // seqs + (i < n % seqs) for i in range(seqs)]
    pos, seq = [], []
    for i, m in enumerate(each):
        first = rng.randint(0, case["far"] - m)
        pos += range(first, first + m)
        seq += [i] * m
    s["pos"] = torch.tensor(pos + [-1] * case["pad"], dtype=torch.int32, device="cuda")
    s["seq"] = torch.tensor(seq + [0] * case["pad"], dtype=torch.int32, device="cuda")
    s["k"], s["v"], s["table"] = _pools(case, gen, seqs, case["far"])
    s["k_out"] = torch.zeros(case["tokens"], hkv, hd, device="cuda")
    s["v_out"] = torch.zeros_like(s["k_out"])
    kx = _key_rows(gen, case["tokens"], hkv, hd)
    vx = torch.randn(case["tokens"], hkv, hd, device="cuda", generator=gen)
    if kind == "load":
        at, off = s["table"][s["seq"][:n].long(), s["pos"][:n].long() // page].long(), s["pos"][:n].long() % page
        _fill(s["k"], case, at, off, kx[:n])
        _fill(s["v"], case, at, off, vx[:n])
        return s
    s["kx"], s["vx"] = kx, vx
    if case["n_rot"]:
        s["freqs"] = _turns(case["n_rot"], "plain")
    if case["Hq"]:
        s["q"] = torch.randn(case["tokens"], case["Hq"], hd, device="cuda", generator=gen)
        s["q_out"] = torch.zeros_like(s["q"])
    return s


# --------------------------------------------------------------------------------------------------------- plain forms
def _rotate(x, pos, freqs, layout, mscale, inverse):
    """Rotates the first 2 * len(freqs) values of each head, in 64 bits (far positions' angles), rounded once."""
    half = freqs.numel()
    angle = (pos.long()[:, None] * freqs[None, :]).double() * (2 * math.pi / TURN)  # the product wraps by whole turns
    c, s = mscale * torch.cos(angle)[:, None], mscale * torch.sin(angle)[:, None]
    if inverse:
        s = -s
    part = x[..., : 2 * half].double()
    a, b = (part[..., :half], part[..., half:]) if layout == "half" else (part[..., 0::2], part[..., 1::2])
    y, z = a * c - b * s, a * s + b * c
    turned = torch.cat((y, z), -1) if layout == "half" else torch.stack((y, z), -1).flatten(-2)
    return torch.cat((turned.float(), x[..., 2 * half:]), -1)


def _rows(pool, case, at, off):
    """The values of rows (at, off) of a pool, f32 [..., Hkv, hd]."""
    codes, scales = _planes(pool, case)
    x = codes[at, :, off].float()
    return x if scales is None else x * scales[at, :, off][..., None]


def _plain_attend(s):
    case = s["case"]
    page, hkv = case["page"], case["Hkv"]
    group, lens = case["Hq"] // hkv, s["lens"].long()
    p = torch.arange(s["longest"], device="cuda")
    live = p[None, :] < lens[:, None]
    if case["window"]:
        live = live & (p[None, :] >= lens[:, None] - case["window"])
    at, off = s["table"][:, p // page].long(), (p % page).expand(lens.numel(), -1)
    zero = torch.zeros((), device="cuda")
    k = torch.where(live[..., None, None], _rows(s["k"], case, at, off), zero).permute(0, 2, 3, 1)
    q = s["q"].unflatten(1, (hkv, group))
    t = torch.where(live[:, None, None], torch.matmul(q, k) * (case["hd"] ** -0.5), -math.inf)
    del k
    top = t.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, zero, top)
    e = torch.exp(t - top)
    total = e.sum(-1, keepdim=True)
    v = torch.where(live[..., None, None], _rows(s["v"], case, at, off), zero).permute(0, 2, 1, 3)
    out = torch.matmul(e / torch.where(total > 0, total, zero + 1), v).flatten(1, 2)
    lse = (top + torch.log(total)).flatten(1)
    kept = lens >= 0  # a padding row stays as it was
    return (torch.where(kept[:, None, None], out, s["out"]), torch.where(kept[:, None], lse, s["lse"]))


def _plain_load(s):
    case, kept = s["case"], s["pos"] >= 0
    pos = torch.where(kept, s["pos"], 0).long()
    at, off = s["table"][s["seq"].long(), pos // case["page"]].long(), pos % case["page"]
    return tuple(torch.where(kept[:, None, None], _rows(s[w], case, at, off), s[w + "_out"]) for w in ("k", "v"))


def _plain_store(s):
    case = s["case"]
    n = case["tokens"] - case["pad"]  # the padding tokens are the last ones
    kx, q = s["kx"], s.get("q")
    if case["n_rot"]:
        kx = _rotate(kx, s["pos"], s["freqs"], case["layout"], 1.0, False)
    pos = s["pos"][:n].long()
    at, off = s["table"][s["seq"][:n].long(), pos // case["page"]].long(), pos % case["page"]
    _fill(s["k"], case, at, off, kx[:n])
    _fill(s["v"], case, at, off, s["vx"][:n])
    got = _plain_load(s)
    if q is None:
        return got
    turned = _rotate(q, s["pos"], s["freqs"], case["layout"], 1.0, False)
    return got + (torch.where((s["pos"] >= 0)[:, None, None], turned, s["q_out"]),)


# ------------------------------------------------------------------------------------------------- the library's calls
def _handles(s):
    """What a program sets up once and keeps: the cache's description, the rotation's, the attention's workspace."""
    import block_quantized_weight_q8_gb300 as qmm

    case, h = s["case"], {"qmm": qmm}
    if case["kind"] != "rope":
        h["pages"] = qmm.KvPages(case["type"], s["k"], s["v"], s["table"], case["page"], case["Hkv"], case["hd"])
    if "freqs" in s:
        h["rope"] = qmm.RopeSpec(s["freqs"], case["layout"], _mscale(case))
    if case["kind"] == "attend":
        h["bytes"] = qmm.qmm_kv_attend_scratch_bytes(case["Hq"], case["Hkv"], case["hd"])
        h["scratch"] = torch.empty(h["bytes"], dtype=torch.uint8, device="cuda")
    return h


def _own(s):
    if "handles" not in s:
        s["handles"] = _handles(s)
    case, h = s["case"], s["handles"]
    qmm, kind = h["qmm"], case["kind"]
    if kind == "rope":
        qmm.qmm_rope(h["rope"], s["x"], s["out"], s["pos"], inverse=case["inverse"])
        return s["out"]
    if kind == "attend":
        qmm.qmm_kv_attend(h["pages"], s["q"], s["lens"], s["out"], h["scratch"], h["bytes"], case["hd"] ** -0.5,
                          lse=s["lse"], window=case["window"])
        return s["out"], s["lse"]
    got = (s["k_out"], s["v_out"])
    if kind == "store":
        if case["Hq"]:
            qmm.qmm_kv_store(h["pages"], s["kx"], s["vx"], s["pos"], seq=s["seq"], rope=h["rope"], q=s["q"],
                             q_out=s["q_out"])
            got += (s["q_out"],)
        else:
            qmm.qmm_kv_store(h["pages"], s["kx"], s["vx"], s["pos"], seq=s["seq"], rope=h.get("rope"))
    qmm.qmm_kv_load(h["pages"], s["pos"], s["k_out"], s["v_out"], seq=s["seq"])
    return got


def run(state):
    if own:
        return _own(state)
    case = state["case"]
    if case["kind"] == "rope":
        return _rotate(state["x"], state["pos"], state["freqs"], case["layout"], _mscale(case), case["inverse"])
    if case["kind"] == "attend":
        return _plain_attend(state)
    return _plain_load(state) if case["kind"] == "load" else _plain_store(state)


# ---------------------------------------------------------------------------------------------------------- what it costs
def work(case):
    kind = case["kind"]
    if kind == "rope":
        n = case["tokens"] * case["heads"]
        return {"bytes": 8 * n * case["hd"] + 4 * case["tokens"] + 4 * case["n_rot"], "flops": 3 * n * case["n_rot"]}
    hkv, hd = case["Hkv"], case["hd"]
    if kind == "attend":
        lens = [max(n, 0) for n in _lens(case)]
        if case["window"]:
            lens = [min(n, case["window"]) for n in lens]
        seen = sum(lens)
        return {"bytes": 2 * seen * hkv * _row_bytes(case) + case["rows"] * case["Hq"] * (8 * hd + 4)
                + 4 * sum(-(-n // case["page"]) for n in lens), "flops": 4 * seen * case["Hq"] * hd}
    n = case["tokens"] - case["pad"]
    bytes_, flops = 2 * n * hkv * (4 * hd + _row_bytes(case)) + 8 * n, 2 * n * hkv * hd
    if kind == "store":
        bytes_ += 2 * n * hkv * (4 * hd + _row_bytes(case)) + 8 * n * case["Hq"] * hd
        flops += n * (3 * (case["Hq"] + hkv) * case["n_rot"] + 6 * hkv * hd)
    return {"bytes": bytes_, "flops": flops}


# ------------------------------------------------------------------------------- the definitions, in 64 bits, on the host
def _exact_turn(x, pos, freqs, layout, mscale, sign):
    """numpy, pair by pair; the fraction of a turn by whole-number arithmetic."""
    f = freqs.cpu().numpy().view(np.uint64)
    p = pos.cpu().numpy().astype(np.int64).view(np.uint64)
    x = x.cpu().numpy().astype(np.float64)
    y = x.copy()
    for i in range(f.size):
        a, b = (i, i + f.size) if layout == "half" else (2 * i, 2 * i + 1)
        t = (p * f[i]).astype(np.float64) / TURN * (2 * np.pi)
        c, s = (mscale * np.cos(t))[:, None], (sign * mscale * np.sin(t))[:, None]
        y[:, :, a] = c * x[:, :, a] - s * x[:, :, b]
        y[:, :, b] = s * x[:, :, a] + c * x[:, :, b]
    return y


def _exact_held(x, typ):
    """The values that rows x (f32) have once they are held: the type's rounding steps as the rule states them."""
    if typ == "f16":
        return x.astype(np.float16).astype(np.float64)
    amax = np.abs(x).max(-1, keepdims=True)
    with np.errstate(divide="ignore", invalid="ignore"):
        inv = np.where(amax > 0, np.float32(127) / amax, np.float32(0)).astype(np.float32)
    codes = np.rint((x * inv).astype(np.float32))
    return codes.astype(np.float64) * (amax / np.float32(127)).astype(np.float32).astype(np.float64)


def _exact_attend(s):
    case = s["case"]
    page, hkv, hd, group = case["page"], case["Hkv"], case["hd"], case["Hq"] // case["Hkv"]
    out, lse = s["out"].double(), s["lse"].double()
    for r, n in enumerate(s["lens"].tolist()):
        if n < 0:
            continue
        first = max(0, n - case["window"]) if case["window"] else 0
        if n == 0:
            lse[r] = -math.inf
            continue
        held = []
        for pool in (s["k"], s["v"]):
            mine = pool[s["table"][r, first // page: (n - 1) // page + 1].long()]
            if case["type"] == "q8":
                codes = mine[:, : hkv * page * hd].reshape(-1, hkv, page, hd).view(torch.int8).double()
                d = mine[:, hkv * page * hd: hkv * page * (hd + 4)].contiguous().view(torch.float32)
                rows = codes * d.reshape(-1, hkv, page, 1).double()
            else:
                rows = mine[:, : 2 * hkv * page * hd].contiguous().view(torch.float16).reshape(-1, hkv, page, hd).double()
            rows = rows.transpose(0, 1).reshape(hkv, -1, hd)
            skip = first - first // page * page
            held.append(rows[:, skip: skip + n - first])
        for h in range(case["Hq"]):
            t = (held[0][h // group] @ s["q"][r, h].double()) / math.sqrt(hd)
            e = torch.exp(t - t.max())
            out[r, h] = (e @ held[1][h // group]) / e.sum()
            lse[r, h] = t.max() + torch.log(e.sum())
    return out, lse


def exact(case, seed):
    s = prepare(case, seed)
    if case["kind"] == "rope":
        return _exact_turn(s["x"], s["pos"], s["freqs"], case["layout"], _mscale(case), -1.0 if case["inverse"] else 1.0)
    if case["kind"] == "attend":
        return _exact_attend(s)
    n = case["tokens"] - case["pad"]
    if case["kind"] == "load":
        got = []
        for w in ("k", "v"):
            flat = s[w].cpu().numpy()
            at = s["table"].cpu().numpy()[s["seq"][:n].cpu().numpy(), s["pos"][:n].cpu().numpy() // case["page"]]
            off = s["pos"][:n].cpu().numpy() % case["page"]
            rows = np.zeros((case["tokens"], case["Hkv"], case["hd"]))
            for h in range(case["Hkv"]):
                slot = h * case["page"] + off
                wide = 1 if case["type"] == "q8" else 2
                cols = slot[:, None] * (case["hd"] * wide) + np.arange(case["hd"] * wide)
                raw = np.ascontiguousarray(flat[at[:, None], cols])
                if case["type"] == "q8":
                    tail = case["Hkv"] * case["page"] * case["hd"] + slot[:, None] * 4 + np.arange(4)
                    d = np.ascontiguousarray(flat[at[:, None], tail]).view(np.float32)
                    rows[:n, h] = raw.view(np.int8).astype(np.float64) * d.astype(np.float64)
                else:
                    rows[:n, h] = raw.view(np.float16).astype(np.float64)
            got.append(rows)
        return tuple(got)
    kx, vx = s["kx"].cpu().numpy(), s["vx"].cpu().numpy()
    if case["n_rot"]:
        kx = _exact_turn(s["kx"], s["pos"], s["freqs"], case["layout"], 1.0, 1.0).astype(np.float32)
    got = []
    for x in (kx, vx):
        held = _exact_held(x, case["type"])
        held[n:] = 0.0
        got.append(held)
    if case["Hq"]:
        q = _exact_turn(s["q"], s["pos"], s["freqs"], case["layout"], 1.0, 1.0)
        q[n:] = 0.0
        got.append(q)
    return tuple(got)
