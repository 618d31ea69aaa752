"""Sums of squares a hair from the middle between two floats: the norm's bits are those of the exact sum."""
from fractions import Fraction

import numpy as np
import pytest

import oracle
from test_gpu_addnorm import gpu, run, same  # noqa: F401

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu
K = 65536
# equal values, 64 to a thread, whose errors all point one way, and the side of the middle that the exact sum is on
VALUES = [(1.6051366329193115, -1), (1.5320110321044922, 1), (1.7702089548110962, -1), (1.8043079376220703, 1),
          (1.0716485977172852, 1), (1.5126584768295288, 1), (1.3519327640533447, 1), (1.73167085647583, -1),
          (1.1583504676818848, -1), (1.9276889562606812, -1), (1.0077069997787476, 1), (1.5525082349777222, -1)]


def beside_a_middle(value, side):
    """(row, the exact sum's nearest float): K - 2 equal values and two that bring the sum 2^-42.6 beside a middle."""
    base = Fraction(value) ** 2 * (K - 2)
    step = Fraction(2) ** (int(base + 1).bit_length() - 24)
    below = int((base + 1) / step) * step
    want = (below + step / 2) * (1 + side * Fraction(1, 6 * 2 ** 40)) - base
    a = np.float32(np.sqrt(float(want)))
    while Fraction(float(a)) ** 2 > want:
        a = np.nextafter(a, np.float32(0))
    b = np.float32(np.sqrt(float(want - Fraction(float(a)) ** 2)))
    row = np.full(K, value, np.float32)
    row[:2] = a, b
    exact = base + Fraction(float(a)) ** 2 + Fraction(float(b)) ** 2
    off = (exact - below - step / 2) / exact
    assert 2.0 ** -43 < side * off < 2.0 ** -42
    return row, np.float32(float(below + (step if side > 0 else 0)))


@pytest.mark.parametrize("act", ["q8_0", "q8_K"])
def test_sums_beside_a_middle(act):
    rows, sums = zip(*(beside_a_middle(*v) for v in VALUES))
    y, ss = np.stack(rows), np.array(sums, np.float32)[:, None]
    s = np.float32(1) / np.sqrt((ss / np.float32(K)).astype(np.float32) + np.float32(1e-6))
    w = np.random.default_rng(1).uniform(0.5, 1.5, K).astype(np.float32)
    want = ((y * s.astype(np.float32)).astype(np.float32) * w).astype(np.float32)
    _, h, q = run(act, y, np.zeros_like(y), w, eps=1e-6)
    same(h, want)
    assert np.array_equal(q, oracle.quantize(act, want))
