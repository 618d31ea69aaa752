"""Many choices whose minimums' parts cancel: activations whose sums of 16 are +S and -S in every block of 32, under minimums of
2^p times the scale.  Held against include/qmm.h's own words: 1e-5 of the row's L2 norm and, of what the parts of a run add up
to in magnitude (the codes' products, and each sum of 16 times its minimum), 2^-18."""
import numpy as np
import pytest

import experts_plain as plain
import oracle
from test_gpu_experts import dev, gpu, host, picks, scratch_of, weights_of  # noqa: F401
from test_gpu_experts_many import FIELDS

torch = pytest.importorskip("torch")
import block_quantized_weight_q8_gb300 as qmm  # noqa: E402

pytestmark = pytest.mark.gpu
T, E, N, K = 4500, 2, 72, 1024


@pytest.mark.parametrize("wtype", ["q4_1", "q5_1", "q4_K", "q5_K"])
@pytest.mark.parametrize("p", [0, 6, 10, 14, 18])
def test_minimums_that_cancel(wtype, p):
    rng = np.random.default_rng(p)
    act = plain.act_of(wtype)
    at, mat, size = FIELDS[wtype]
    raw = weights_of(wtype, E, N, K, 1).reshape(E * N, -1, size).copy()
    for where, v in ((at, 2.0 ** -6), (mat, 2.0 ** (p - 6))):
        f = (v * rng.uniform(1, 1.99, raw.shape[:2])).astype(np.float16)
        raw[:, :, where:where + 2] = f.view(np.uint8).reshape(*f.shape, 2)
    x = rng.integers(-126, 127, (T, K // 32, 2, 16)).astype(np.float32)
    x[..., 0] = 127
    x[:, :, 1] = -x[:, :, 0, ::-1]
    x = x.reshape(T, K)
    xq = oracle.quantize(act, x)
    assert np.array_equal(oracle.dequantize(act, xq, K), x)  # scales of 1: exact

    def values(*drop):
        part = raw.copy()
        for o in drop:
            part[:, :, o:o + 2] = 0
        return oracle.dequantize(wtype, part.reshape(E * N, -1), K).astype(np.float64)

    ids = picks(T, 1, E, 5)
    want = x.astype(np.float64) @ values(mat).T  # the minimums' parts are zero
    codes = values(mat).reshape(E * N, -1, 32)
    codes = np.broadcast_to(np.abs(codes).max(-1, keepdims=True) * 2, codes.shape).reshape(E * N, K)  # centered or not
    parts = np.abs(x) @ codes.T + np.abs(x.reshape(T, -1, 16).sum(-1)) @ np.abs(values(at))[:, ::16].T
    want, parts = (v.reshape(T, E, N)[np.arange(T), ids[:, 0]] for v in (want, parts))
    off = plain.PRODUCT * np.linalg.norm(want, axis=-1, keepdims=True) + 2.0 ** -18 * parts
    assert qmm.qmm_experts_path(wtype, False, T, 1, E, N, K) == 1
    y = torch.empty(T, N, device="cuda")
    scratch, n = scratch_of(wtype, T, 1, E, N, K)
    qmm.qmm_experts_sum(wtype, dev(raw.reshape(E, N, -1)), dev(x.reshape(T, 1, K)), dev(ids), None, y, scratch, n)
    err = np.abs(host(y) - want)
    assert (err <= off).all(), (err / off).max()
