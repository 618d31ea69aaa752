"""Many choices of K-quants whose scale d and minimums' scale m are far apart, with the larger part gone: codes of zero under
a large d, activations whose sums of 16 are zero under a large m.  Held against include/qmm.h's own words: 1e-5 of the row's
L2 norm, beside that 2^-25 |d| a minimum and, where |m| > 2^29 |d|, 2^-25 |m| a scale times code."""
import numpy as np
import pytest

import experts_plain as plain
import oracle
import workloads
from test_gpu_experts import dev, gpu, host, picks, scratch_of, weights_of  # noqa: F401
from test_gpu_experts_many import FIELDS

torch = pytest.importorskip("torch")
import block_quantized_weight_q8_gb300 as qmm  # noqa: E402

pytestmark = pytest.mark.gpu
T, E, N, K = 4500, 2, 72, 1024
CODES = {"q4_K": 16, "q5_K": 16, "q2_K": 16}  # where the codes begin (q5_K: their fifth bits; q2_K ends before its scales)


def blocks(wtype, seed, d, m):
    """Random scales, minimums and codes under these d and m, each block's times 1 to 2."""
    rng = np.random.default_rng(seed)
    at, mat, size = FIELDS[wtype]
    raw = weights_of(wtype, E, N, K, seed).reshape(E * N, -1, size).copy()
    raw[:, :, :16] = rng.integers(0, 256, raw[:, :, :16].shape)  # scales and minimums
    for where, v in ((at, d), (mat, m)):
        f = (v * rng.uniform(1, 1.99, raw.shape[:2])).astype(np.float16)
        raw[:, :, where:where + 2] = f.view(np.uint8).reshape(*f.shape, 2)
    return raw


def run(wtype, raw, x, off):
    """The summed products against the definition, off beside the share of the norm; the gated products of the same weights
    twice, silu(p) p."""
    W, ids = raw.reshape(E, N, -1), picks(T, 1, E, 5)
    assert qmm.qmm_experts_path(wtype, False, T, 1, E, N, K) == 1 and qmm.qmm_experts_path(wtype, True, T, 1, E, N, K) == 1
    xq = oracle.quantize("q8_K", x)
    p = oracle.dequantize("q8_K", xq, K).astype(np.float64) @ oracle.dequantize(wtype, raw.reshape(E * N, -1), K).astype(np.float64).T
    p, off = (np.broadcast_to(v, (T, E * N)).reshape(T, E, N)[np.arange(T), ids[:, 0]] for v in (p, off))
    off = off + plain.PRODUCT * np.linalg.norm(p, axis=-1, keepdims=True)
    y, h = torch.empty(T, N, device="cuda"), torch.empty(T, 1, N, device="cuda")
    scratch, n = scratch_of(wtype, T, 1, E, N, K)
    qmm.qmm_experts_sum(wtype, dev(W), dev(x.reshape(T, 1, K)), dev(ids), None, y, scratch, n)
    qmm.qmm_experts_glu(wtype, dev(W), dev(W), dev(xq), dev(ids), h, scratch, n)
    share = (np.abs(host(y) - p) / off).max()
    assert share <= 1, share
    a = plain.gate_of("silu", p)
    dh = 1.13 * off * np.abs(p) + np.abs(a) * off + 1.2 * off * off + 2.0 ** -20 * p * p
    share = (np.abs(host(h)[:, 0] - a * p) / (dh + 1e-42)).max()  # and the smallest f32
    assert share <= 1, share


@pytest.mark.parametrize("wtype", sorted(CODES))
@pytest.mark.parametrize("p", [-2, 3, 8, 12, 16, 20, 28])
def test_minimums_under_a_large_scale(wtype, p):
    d = 20.0
    raw = blocks(wtype, 1, d, d * 2.0 ** -p)
    end = 80 if wtype == "q2_K" else None
    raw[:, :, CODES[wtype]:end] = 0  # no codes: the minimums alone are left
    x = workloads.activations_f32(T, K, seed=4)
    xd = oracle.dequantize("q8_K", oracle.quantize("q8_K", x), K).astype(np.float64)
    sums = np.abs(xd.reshape(T, K // 16, 16).sum(-1)).sum(-1)
    run(wtype, raw, x, (2.0 ** -25 * 2 * d * sums)[:, None])


@pytest.mark.parametrize("wtype", sorted(CODES))
@pytest.mark.parametrize("p", [0, 8, 10, 14, 20, 26, 28, 30, 33, 36, 38])
def test_codes_under_large_minimums(wtype, p):
    m = 2.0 ** min(14, p - 12)
    d = m * 2.0 ** -p  # down to the smallest f16
    raw = blocks(wtype, 2, d, m)
    x = workloads.activations_f32(T, K, seed=5)
    x[:, 1::2] = -x[:, ::2]  # every sum of 16 is zero, and so is what the minimums add
    xd = oracle.dequantize("q8_K", oracle.quantize("q8_K", x), K).astype(np.float64)
    assert (xd.reshape(T, -1, 16).sum(-1) == 0).all()
    at, mat, _ = FIELDS[wtype]
    dd, mm = (np.abs(raw[:, :, o:o + 2].copy().view(np.float16).astype(np.float64)[..., 0]) for o in (at, mat))
    per = np.where(mm > 2.0 ** 29 * dd, 2.0 ** -25 * mm, 0.0).repeat(256, 1)  # of each value
    run(wtype, raw, x, np.abs(xd) @ per.T)
