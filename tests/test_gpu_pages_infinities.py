"""Infinities in the rows of a 16-bit cache, as values above 65504 leave them: the attention's results are the definition's."""
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


def attend(c, q, n, scale, R):
    pages = qmm.KvPages(c.typ, dev(c.k), dev(c.v), dev(c.table), c.page, c.Hkv, c.hd)
    m = qmm.qmm_kv_attend_scratch_bytes(q.shape[1], c.Hkv, c.hd)
    scratch, out = torch.empty(m, dtype=torch.uint8, device="cuda"), torch.empty(R, *q.shape[1:], device="cuda")
    lse = torch.empty(R, q.shape[1], device="cuda")
    lens, seq = torch.full((R,), n, dtype=torch.int32, device="cuda"), torch.zeros(R, dtype=torch.int32, device="cuda")
    qmm.qmm_kv_attend(pages, dev(np.repeat(q, R, 0)), lens, out, scratch, m, scale, lse=lse, seq=seq)
    torch.cuda.synchronize()
    return out.cpu().numpy(), lse.cpu().numpy()


SHAPES = [(4, 1, 64, 90, 1), (4, 2, 256, 50, 1), (3, 1, 80, 700, 1), (40, 40, 64, 120, 5), (40, 40, 128, 120, 5)]


@pytest.mark.parametrize("Hq,Hkv,hd,n,R", SHAPES)
def test_infinite_values_stay_in_their_column(Hq, Hkv, hd, n, R):
    """One value beyond f16 in column 3 (positive) and 5 (negative), both signs in column 7: an infinity, an infinity and a
    NaN there; the other columns within their bound."""
    rng = np.random.default_rng(hd)
    c = plain.Cache("f16", Hkv, hd, 16, 1, n, seed=1)
    c.fill(0, n, rng, loud=False)
    q = rng.standard_normal((1, Hq, hd)).astype(np.float32)
    want, _, bound, _ = plain.attend(c, q, [n], [0], 0.125)
    with np.errstate(over="ignore"):
        for p, column, x in ((20, 3, 1e5), (33, 5, -1e5), (40, 7, 1e5), (41, 7, -1e5)):
            v = c.get(c.v, 0, p).astype(np.float32)
            v[:, column] = x
            c.put(c.v, 0, p, v)
    got, lse = attend(c, q, n, 0.125, R)
    assert np.all(got[..., 3] == np.inf) and np.all(got[..., 5] == -np.inf) and np.all(np.isnan(got[..., 7]))
    rest = [d for d in range(hd) if d not in (3, 5, 7)]
    assert np.all(np.abs(got[..., rest] - want[..., rest]) <= bound[..., rest])
    assert np.all(np.isfinite(lse))


@pytest.mark.parametrize("Hq,Hkv,hd,n,R", SHAPES)
def test_infinite_scores(Hq, Hkv, hd, n, R):
    """A key below f16's range: where the query's value is positive the score is -inf and the position has no weight, where
    it is negative the score is +inf and the softmax has no value."""
    rng = np.random.default_rng(hd + 1)
    c = plain.Cache("f16", Hkv, hd, 16, 1, n, seed=1)
    c.fill(0, n, rng, loud=False)
    q = rng.standard_normal((1, Hq, hd)).astype(np.float32)
    q[0, :, 2] = np.where(np.arange(Hq) % 2 == 0, 0.7, -0.7)
    gone = (17, n - 1)
    left = plain.Cache("f16", Hkv, hd, 16, 1, n, seed=1)
    at = [p for p in range(n) if p not in gone]
    for i, p in enumerate(at):
        for x, y in ((c.k, left.k), (c.v, left.v)):
            left.put(y, 0, i, c.get(x, 0, p).astype(np.float32))
    want, wlse, bound, lbound = plain.attend(left, q, [len(at)], [0], 0.125)
    with np.errstate(over="ignore"):
        for p in gone:
            k = c.get(c.k, 0, p).astype(np.float32)
            k[:, 2] = -1e6
            c.put(c.k, 0, p, k)
    got, lse = attend(c, q, n, 0.125, R)
    assert np.all(np.abs(got[:, 0::2] - want[:, 0::2]) <= bound[:, 0::2])
    assert np.all(np.abs(lse[:, 0::2] - wlse[:, 0::2]) <= lbound[:, 0::2])
    assert np.all(np.isnan(got[:, 1::2]))
