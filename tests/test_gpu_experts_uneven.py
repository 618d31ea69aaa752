"""Many choices of 32-value formats where a run of 256 values has one block of much larger scale than the others and that
block meets zeros: what is left of the products are the small blocks'.  Held against include/qmm.h's own words: within 1e-5
of the row's L2 norm where the largest scale is small enough, and else, beside that, scales off by 2^-32 of it (Q8_0 rows
beside Q4_1 and Q5_1: 2^-29)."""
import numpy as np
import pytest

import experts_plain as plain
import oracle
from test_gpu_experts import dev, gpu, host, picks, scratch_of, weights_of  # noqa: F401
from test_gpu_experts_many import FIELDS

torch = pytest.importorskip("torch")
import block_quantized_weight_q8_gb300 as qmm  # noqa: E402

pytestmark = pytest.mark.gpu
TYPES = ["q4_0", "q8_0", "q4_1", "q5_0", "q5_1"]
T, E, N, K = 3000, 2, 72, 1024
BIG = 3  # the large block of every eight
SPANS = [2.0 ** p for p in (8, 12, 14, 16, 18, 20, 22, 24)]


def f16(rng, size, shape):
    """Scales of all 11 bits between size and twice that."""
    return (size * rng.uniform(1, 1.999, shape)).astype(np.float16)


def weights(wtype, seed, big, small):
    """Random codes under these scales (and minimums of as much, either sign); big None: the large block is zero."""
    rng = np.random.default_rng(seed)
    at, mat, size = FIELDS[wtype]
    raw = weights_of(wtype, E, N, K, seed).reshape(E * N, -1, size).copy()
    for where in [at] if mat is None else [at, mat]:
        d = f16(rng, small, raw.shape[:2])
        if where == mat:
            d *= rng.choice([-2, 2], d.shape).astype(np.float16)
        d[:, BIG::8] = 0 if big is None else f16(rng, big, d[:, BIG::8].shape)
        raw[:, :, where:where + 2] = d.view(np.uint8).reshape(*d.shape, 2)
    return raw.reshape(E, N, -1)


def rows(seed, big, small):
    """f32 rows [T][K] whose blocks' largest value is 127 times such a scale; big None: the large block is zero."""
    rng = np.random.default_rng(seed)
    codes = rng.integers(-126, 127, (T, K // 32, 32)).astype(np.float32)
    codes[..., 5] = 127
    d = f16(rng, small, (T, K // 32)).astype(np.float32)
    d[:, BIG::8] = 0 if big is None else f16(rng, big, d[:, BIG::8].shape)
    return (codes * d[..., None]).reshape(T, K)


def parts(wtype, W):
    """|scale times code| and |minimum| of each value, apart."""
    _, mat, size = FIELDS[wtype]
    raw = W.reshape(E * N, -1, size)
    if mat is None:
        return np.abs(oracle.dequantize(wtype, raw.reshape(E * N, -1), K))
    out = 0
    for o in (0, mat):
        p = raw.copy()
        p[:, :, o:o + 2] = 0
        out = out + np.abs(oracle.dequantize(wtype, p.reshape(E * N, -1), K))
    return out


def lost(wtype, W, x, side, big, limit, share):
    """How far products may be off [T][E * N] by what scales lose."""
    top = 2 * big
    if top < limit:
        return 0.0
    if side == "rows":  # |code| of a row's value times the loss, times the weights' values
        q = np.full((1, K), 127.0)
    else:
        q = {"q8_0": 128.0, "q4_0": 8.0, "q4_1": 16.0, "q5_0": 16.0, "q5_1": 32.0}[wtype]
    small = np.ones(K // 32, bool)
    small[BIG::8] = False
    small = small.repeat(32)
    if side == "rows":
        return share * top * (q * small) @ parts(wtype, W).T
    return share * top * q * (np.abs(x) @ small)[:, None]


@pytest.mark.parametrize("wtype", TYPES)
@pytest.mark.parametrize("side", ["weights", "rows"])
@pytest.mark.parametrize("big", [14.0, 100.0, 30000.0])
def test_small_blocks_beside_a_large_one(wtype, side, big):
    minimums = wtype in ("q4_1", "q5_1")
    limit, share = (32.0, 2.0 ** -29) if minimums and side == "rows" else (256.0, 2.0 ** -32)
    assert qmm.qmm_experts_path(wtype, False, T, 1, E, N, K) == 1 and qmm.qmm_experts_path(wtype, True, T, 1, E, N, K) == 1
    ids = picks(T, 1, E, 5)
    at = ids[:, 0]
    for span in SPANS:
        small = max(big / span, 2.0 ** -20)
        other = min(max(1 / (small * 2000), 2.0 ** -10), 200.0)  # so that products are some units at most
        if side == "weights":
            W, x = weights(wtype, 1, big, small), rows(2, None, other)
            W2 = weights(wtype, 3, big, small)
        else:
            W, x = weights(wtype, 1, None, other), rows(2, big, small)
            W2 = weights(wtype, 3, None, other)
        xq = oracle.quantize("q8_0", x)
        xd = oracle.dequantize("q8_0", xq, K).astype(np.float64)

        y = torch.empty(T, N, device="cuda")
        scratch, n = scratch_of(wtype, T, 1, E, N, K)
        qmm.qmm_experts_sum(wtype, dev(W), dev(x.reshape(T, 1, K)), dev(ids), None, y, scratch, n)
        h = torch.empty(T, 1, N, device="cuda")
        qmm.qmm_experts_glu(wtype, dev(W), dev(W2), dev(xq), dev(ids), h, scratch, n)

        def product(V):
            p = xd @ oracle.dequantize(wtype, V.reshape(E * N, -1), K).astype(np.float64).T
            off = np.broadcast_to(lost(wtype, V, xd, side, big, limit, share), p.shape)
            pick = lambda a: a.reshape(T, E, N)[np.arange(T), at]  # noqa: E731
            p, off = pick(p), pick(np.ascontiguousarray(off))
            return p, off + plain.PRODUCT * np.linalg.norm(p, axis=-1, keepdims=True)

        g, dg = product(W)
        u, du = product(W2)
        off = np.abs(host(y) - g) / dg
        assert off.max() <= 1, ("sum", span, off.max())
        a = plain.gate_of("silu", g)
        dh = 1.13 * dg * np.abs(u) + np.abs(a) * du + 1.2 * dg * du + 2.0 ** -20 * np.abs(g * u)
        off = np.abs(host(h)[:, 0] - a * u) / dh
        assert off.max() <= 1, ("glu", span, off.max())
