"""Renormalised weights of scores that f32 cannot hold: experts chosen for their bias, or all far from 0."""
import numpy as np
import pytest

import experts_plain as plain
from test_gpu_route import dev, gpu  # noqa: F401

torch = pytest.importorskip("torch")
import block_quantized_weight_q8_gb300 as qmm  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("low", [-60.0, -90.0, -103.0, -300.0, -690.0])
def test_small_scores(score, low):
    """A weight is off by its f32 score's rounding where f32 holds them (as in tests/test_gpu_route.py), else by one rounding
    of 2^-24 and less than 2^-40 for binary64's."""
    rng = np.random.default_rng(3)
    T, E, k = 40, 32, 4
    logits = (low + rng.uniform(-3, 3, (T, E))).astype(np.float32)
    bias = np.zeros(E, np.float32)
    bias[::3] = 4.0 + np.arange(11, dtype=np.float32)  # these are chosen
    if score == "softmax":
        logits[:, 1] = 0.0  # and this has all of the score
    ids, w = torch.empty(T, k, dtype=torch.int32, device="cuda"), torch.empty(T, k, device="cuda")
    qmm.qmm_route(dev(logits), ids, w, score=score, bias=dev(bias))
    want_ids, want = plain.route(logits, bias, k, score=score)
    torch.cuda.synchronize()
    assert np.array_equal(ids.cpu().numpy(), want_ids)
    assert (np.abs(w.cpu().numpy() - want) <= 2.0 ** -24 * (2 * 90 + 2 * 36 + 16) * want).all()
    assert np.abs(want.sum(-1) - 1).max() < 1e-12
