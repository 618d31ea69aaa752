"""How much room the page table has does not show in the attention's results."""
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


@pytest.mark.parametrize("typ,Hq,Hkv,hd,page,lens,window", [
    ("q8", 14, 2, 64, 16, [33], 0), ("q8", 8, 1, 128, 16, [1], 0), ("q8", 32, 8, 128, 16, [700, 0, -1, 16], 0),
    ("q8", 8, 1, 128, 8, [2000], 33), ("f16", 6, 2, 256, 4, [4, 90, 0], 0), ("f16", 3, 1, 80, 16, [513, 16], 17),
    ("q8", 40, 40, 32, 16, [16, 3, 0, 1, 9], 0), ("q8", 3, 3, 16, 16, [0, 0], 0)])
def test_the_rooms_of_the_table(typ, Hq, Hkv, hd, page, lens, window):
    """A table that the longest row fills to its last page, one with some room and one with far more: the same bits, from
    rows that are all empty to rows that are full, and the definition's values in the fullest."""
    rng = np.random.default_rng(hd)
    c = plain.Cache(typ, Hkv, hd, page, len(lens), max(max(lens), 1), seed=hd)
    for r, n in enumerate(lens):
        c.fill(r, max(n, 0), rng)
    q = rng.standard_normal((len(lens), Hq, hd)).astype(np.float32)
    want, _, bound, _ = plain.attend(c, q, lens, range(len(lens)), hd ** -0.5, window)
    k, v, full, n = dev(c.k), dev(c.v), c.table, qmm.qmm_kv_attend_scratch_bytes(Hq, Hkv, hd)
    scratch = torch.empty(n, dtype=torch.uint8, device="cuda")
    for some in (lens, [min(x, 1) for x in lens], [min(x, 0) for x in lens]):
        got = []
        for room in (full.shape[1], full.shape[1] + 3, 70000 // page):
            table = np.full((len(lens), room), 2 ** 30, np.int32)
            table[:, : full.shape[1]] = full
            pages = qmm.KvPages(typ, k, v, dev(table), page, Hkv, hd)
            out = torch.full(q.shape, 9.0, device="cuda")
            qmm.qmm_kv_attend(pages, dev(q), dev(np.array(some, np.int32)), out, scratch, n, hd ** -0.5, window=window)
            torch.cuda.synchronize()
            got.append(out.cpu().numpy())
        assert np.array_equal(got[0].view(np.int32), got[2].view(np.int32))
        assert np.array_equal(got[1].view(np.int32), got[2].view(np.int32))
        if some is lens:
            kept = np.array(lens) >= 0
            assert np.all(np.abs(got[0][kept] - want[kept]) <= bound[kept]) and np.all(got[0][~kept] == 9.0)
