"""What a weight far below its row's largest, or a value row far above the others, costs the attention's result.

The queries have one value only, so a score's terms are that value's alone, A_p = |scale q_0 k_p0|, and the bounds below
hold position by position (pages_plain.attend takes the largest A for all of them, and a wider floor for small weights)."""
import numpy as np
import pytest

import pages_plain as plain

torch = pytest.importorskip("torch")
import block_quantized_weight_q8_gb300 as qmm  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.fail("these tests need a CUDA GPU")
    qmm.build()
    qmm.load()
    qmm.qmm_device_status(clear=True)
    yield
    assert qmm.qmm_device_status(clear=True) == 0


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def definition(c, q0, n):
    """(out [Hq][hd], bound) in 64 bits for queries q0[h] e_0 and scale 1 over positions 0 .. n - 1 of sequence 0.

    A score is off by delta_p = A_p (2^-22 + (hd / 16) 2^-23 + 5 * 2^-24): the query's split, the matrix steps' cutting off,
    four f32 products and the softmax's argument.  A weight, in the numerator: delta_p, the exponential's 2^-22, its product
    with the value scale 2^-24, the split 2^-22, two matrix steps (2^-22 each) and one f32 addition per tile, the four
    warps and the joined parts (2^-24 each); in the denominator: delta_p, 2^-22 and the additions; the division and the
    last product 2^-24 each.  What is below 2^-12 of the largest of its tile is off by 2^-39 of that: of the largest weight
    times value scale for 8-bit rows, so 2^-39 of the largest weight times a row's largest value, of the largest weight in a
    tile of 32 (16) positions times the own value for f16 rows."""
    Hq, hd, G = len(q0), c.hd, len(q0) // c.Hkv
    k = np.stack([c.get(c.k, 0, p) for p in range(n)])
    v = np.stack([c.get(c.v, 0, p) for p in range(n)])
    out, bound = np.zeros((Hq, hd)), np.zeros((Hq, hd))
    adds = (n / 16 + 8) * 2.0 ** -24
    for h in range(Hq):
        t, x = float(q0[h]) * k[:, h // G, 0], v[:, h // G]
        w = np.exp(t - t.max())
        w /= w.sum()
        delta = np.abs(t) * (2.0 ** -22 + hd / 16 * 2.0 ** -23 + 5 * 2.0 ** -24)
        out[h] = w @ x
        bound[h] = (w * (delta + 4 * 2.0 ** -22 + 2.0 ** -24 + adds)) @ np.abs(x)
        bound[h] += np.abs(out[h]) * (w @ (delta + 2.0 ** -22) + adds + 2 * 2.0 ** -24) + 2.0 ** -120
        if c.typ == "q8":
            bound[h] += 2.0 ** -39 * n * (w * np.abs(x).max(-1)).max()
        else:
            tile = 32 if hd <= 64 else 16
            top = np.array([w[p - p % tile: p - p % tile + tile].max() for p in range(n)])
            bound[h] += 2.0 ** -39 * (top @ np.abs(x))
    return out, bound


def compare(c, q0, n, R):
    """R rows over the one sequence: each within the bound, all alike in bits where they share a partition."""
    Hq = len(q0)
    want, bound = definition(c, q0, n)
    q = np.zeros((R, Hq, c.hd), np.float32)
    q[:, :, 0] = q0
    pages = qmm.KvPages(c.typ, dev(c.k), dev(c.v), dev(c.table), c.page, c.Hkv, c.hd)
    m = qmm.qmm_kv_attend_scratch_bytes(Hq, c.Hkv, c.hd)
    scratch, out = torch.empty(m, dtype=torch.uint8, device="cuda"), torch.empty(R, Hq, c.hd, device="cuda")
    lens, seq = torch.full((R,), n, dtype=torch.int32, device="cuda"), torch.zeros(R, dtype=torch.int32, device="cuda")
    qmm.qmm_kv_attend(pages, dev(q), lens, out, scratch, m, 1.0, seq=seq)
    torch.cuda.synchronize()
    err = np.abs(out.cpu().numpy().astype(np.float64) - want)
    assert np.all(err <= bound), np.max(err / bound)


@pytest.mark.parametrize("Hkv,G,hd,n,R", [(1, 8, 128, 150, 1), (2, 3, 64, 300, 1), (1, 4, 256, 90, 1), (40, 2, 64, 320, 5),
                                          (40, 1, 80, 320, 4)])
@pytest.mark.parametrize("at", [1, 70])
@pytest.mark.parametrize("times", [13, 20, 30])
def test_a_large_value_row_without_weight(Hkv, G, hd, n, R, at, times):
    """One value row 2^13 to 2^30 times larger than the others, whose weight is e^-80: the others keep their low bits, in
    its own tile and in those after it; by CTAs and by single warps."""
    rng = np.random.default_rng(hd + times)
    c = plain.Cache("q8", Hkv, hd, 16, 1, n, seed=hd)
    for p in range(n):
        k, v = (rng.standard_normal((Hkv, hd)).astype(np.float32) for _ in range(2))
        k[:, 0] = -80.0 if p == at else rng.uniform(-1, 1, Hkv)
        c.put(c.k, 0, p, k)
        c.put(c.v, 0, p, v * np.float32(2.0 ** times) if p == at else v)
    compare(c, np.linspace(1.0, 1.5, Hkv * G).astype(np.float32), n, R)


@pytest.mark.parametrize("typ,Hkv,G,hd,n,R", [("f16", 40, 2, 64, 480, 5), ("f16", 40, 1, 128, 480, 5),
                                              ("q8", 40, 2, 64, 480, 5), ("f16", 1, 4, 64, 3000, 1)])
def test_large_values_of_small_weight(typ, Hkv, G, hd, n, R):
    """32 positions with nearly all weight and small values, 32 with weights of e^-20 and values that make up for it, in
    turn: the small weights are as exact as the large ones."""
    rng = np.random.default_rng(hd)
    c = plain.Cache(typ, Hkv, hd, 16, 1, n, seed=hd)
    for p in range(n):
        k, v = (rng.standard_normal((Hkv, hd)).astype(np.float32) for _ in range(2))
        far = p // 32 % 2
        k[:, 0] = -20.0 if far else 0.0
        if not far:
            k[:, 0] = rng.uniform(-0.5, 0.5, Hkv)
        c.put(c.k, 0, p, k)
        c.put(c.v, 0, p, np.clip(v, -2, 2) * np.float32(3e4 if far else 2.0 ** -14))
    compare(c, np.linspace(1.0, 1.25, Hkv * G).astype(np.float32), n, R)
