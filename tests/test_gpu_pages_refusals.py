"""Tensors of another number of dimensions are refused by the cache's binding with ValueError, as those of another type,
shape or device are."""
import numpy as np
import pytest

import pages_plain as plain

torch = pytest.importorskip("torch")
import block_quantized_weight_q8_gb300 as qmm  # noqa: E402

pytestmark = pytest.mark.gpu


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def test_numbers_of_dimensions():
    if not torch.cuda.is_available():
        pytest.fail("this test needs a CUDA GPU")
    qmm.build()
    c = plain.Cache("q8", 2, 64, 16, 2, 32)
    pages = qmm.KvPages("q8", dev(c.k), dev(c.v), dev(c.table), 16, 2, 64)
    rope = qmm.RopeSpec(dev(plain.turns(plain.freqs(64))))
    x, q = torch.zeros(2, 2, 64, device="cuda"), torch.zeros(2, 4, 64, device="cuda")
    pos = torch.zeros(2, dtype=torch.int32, device="cuda")
    n = qmm.qmm_kv_attend_scratch_bytes(4, 2, 64)
    scratch = torch.empty(n, dtype=torch.uint8, device="cuda")
    for bad in (x[0, 0, 0], x[0, 0], x[0], x[None]):
        with pytest.raises(ValueError):
            qmm.qmm_rope(rope, bad, bad, pos)
        with pytest.raises(ValueError):
            qmm.qmm_kv_store(pages, bad, x, pos)
        with pytest.raises(ValueError):
            qmm.qmm_kv_store(pages, x, bad, pos)
        with pytest.raises(ValueError):
            qmm.qmm_kv_load(pages, pos, bad, x)
    for bad in (q[0, 0, 0], q[0, 0], q[0], q[None]):
        with pytest.raises(ValueError):
            qmm.qmm_kv_store(pages, x, x, pos, rope=rope, q=bad, q_out=q)
        with pytest.raises(ValueError):
            qmm.qmm_kv_attend(pages, bad, pos, q, scratch, n, 0.1)
        with pytest.raises(ValueError):
            qmm.qmm_kv_attend(pages, q, pos, bad, scratch, n, 0.1)
    for bad in (pos[0], pos[None]):
        with pytest.raises(ValueError):
            qmm.qmm_kv_load(pages, bad, x, x)
        with pytest.raises(ValueError):
            qmm.qmm_kv_store(pages, x, x, bad)
        with pytest.raises(ValueError):
            qmm.qmm_kv_attend(pages, q, bad, q, scratch, n, 0.1)
    assert qmm.qmm_device_status(clear=True) == 0
