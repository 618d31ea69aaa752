"""The residual's addition with the norm and its 8-bit rows on the GPU, bit for bit against the definition."""
import numpy as np
import pytest

import experts_plain as plain

torch = pytest.importorskip("torch")
import block_quantized_weight_q8_gb300 as qmm  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.fail("these tests need a CUDA GPU")
    qmm.build()
    qmm.load()
    yield
    assert qmm.qmm_device_status(clear=True) == 0


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def rows(M, K, seed):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((M, K)).astype(np.float32) * np.where(rng.random(K) < 0.01, 20, 1).astype(np.float32)
    return x, rng.standard_normal((M, K)).astype(np.float32), (1 + 0.2 * rng.standard_normal(K)).astype(np.float32)


def run(act, x, r, w, eps=plain.EPS, want_sum=True, want_h=True, want_q=True):
    M, K = x.shape
    s = torch.full((M, K), float("nan"), device="cuda") if want_sum else None
    h = torch.full((M, K), float("nan"), device="cuda") if want_h else None
    q = torch.full((M, qmm.qmm_row_bytes(act, K)), 0xEE, dtype=torch.uint8, device="cuda") if want_q else None
    qmm.qmm_add_rmsnorm_quantize(act, dev(x), dev(r), dev(w), eps, q, sum=s, h=h)
    torch.cuda.synchronize()
    return [None if t is None else t.cpu().numpy() for t in (s, h, q)]


def same(a, b):
    assert np.array_equal(a.view(np.uint32), b.view(np.uint32))


@pytest.mark.parametrize("act,K", [("q8_0", 32), ("q8_0", 96), ("q8_0", 896), ("q8_0", 4096), ("q8_0", 4128), ("q8_0", 12288),
                                   ("q8_0", 16384), ("q8_0", 16416), ("q8_0", 65536), ("q8_K", 256), ("q8_K", 2816),
                                   ("q8_K", 8192), ("q8_K", 8448), ("q8_K", 16384), ("q8_K", 16640), ("q8_K", 65536)])
@pytest.mark.parametrize("M", [1, 7])
def test_bits(act, K, M):
    """The sum of squares is the exact one's nearest f32 (but within 2^-20 or so of a tie), so every output's bits are the
    definition's."""
    x, r, w = rows(M, K, K + M)
    y, h, q = plain.add_norm(act, x, r, w, plain.EPS)
    gs, gh, gq = run(act, x, r, w)
    same(gs, y)
    same(gh, h)
    assert np.array_equal(gq, q)


@pytest.mark.parametrize("act,M,K", [("q8_K", 3000, 256), ("q8_0", 700, 4096), ("q8_K", 650, 4096), ("q8_0", 2000, 160)])
def test_many_rows(act, M, K):
    x, r, w = rows(M, K, 1)
    y, h, q = plain.add_norm(act, x, r, w, plain.EPS)
    gs, gh, gq = run(act, x, r, w)
    same(gs, y)
    same(gh, h)
    assert np.array_equal(gq, q)


@pytest.mark.parametrize("K", [512, 20480])
def test_outputs_that_are_left_out(K):
    x, r, w = rows(5, K, 2)
    full = run("q8_0", x, r, w)
    for a in (dict(want_sum=False), dict(want_h=False), dict(want_q=False), dict(want_sum=False, want_h=False),
              dict(want_sum=False, want_q=False)):
        for got, all_ in zip(run("q8_0", x, r, w, **a), full):
            assert got is None or np.array_equal(got.view(np.uint8), all_.view(np.uint8))


@pytest.mark.parametrize("K", [512, 20480])
@pytest.mark.parametrize("into", ["x", "r"])
def test_the_sum_in_place(K, into):
    x, r, w = rows(9, K, 3)
    y, h, q = plain.add_norm("q8_K", x, r, w, plain.EPS)
    t = {"x": dev(x), "r": dev(r)}
    gq = torch.empty(9, qmm.qmm_row_bytes("q8_K", K), dtype=torch.uint8, device="cuda")
    qmm.qmm_add_rmsnorm_quantize("q8_K", t["x"], t["r"], dev(w), plain.EPS, gq, sum=t[into])
    torch.cuda.synchronize()
    same(t[into].cpu().numpy(), y)
    assert np.array_equal(gq.cpu().numpy(), q)


def test_extremes():
    """Rows of zeros, of one large value, of values whose squares overflow (the sum is infinite and its inverse root 0)."""
    x, r, w = rows(6, 256, 4)
    x[0], r[0] = 0, 0
    x[1], r[1] = 0, 0
    x[1, 17] = 3e4
    x[2] *= 1e-12
    r[2] *= 1e-12
    x[3] *= np.float32(1e25)
    r[4] = -x[4]
    for eps in (1e-5, 1.0):
        with np.errstate(over="ignore", under="ignore"):
            y, h, q = plain.add_norm("q8_0", x, r, w, eps)
        gs, gh, gq = run("q8_0", x, r, w, eps)
        same(gs, y)
        same(gh, h)
        assert np.array_equal(gq, q)
    assert (gh[3] == 0).all()


def test_rows_do_not_meet():
    """A row with infinities or NaN leaves the others as they are."""
    x, r, w = rows(8, 512, 5)
    clean = run("q8_0", x, r, w)
    x[2, 7], x[5, 100] = np.inf, np.nan
    got = run("q8_0", x, r, w)
    keep = [0, 1, 3, 4, 6, 7]
    for a, b in zip(got, clean):
        assert np.array_equal(a[keep].view(np.uint8), b[keep].view(np.uint8))
    assert np.isnan(got[1][5]).all()


def test_refusals_of_the_binding():
    x, w = torch.zeros(4, 512, device="cuda"), torch.zeros(512, device="cuda")
    q = torch.zeros(4, qmm.qmm_row_bytes("q8_0", 512), dtype=torch.uint8, device="cuda")
    for a in ((x.half(), x, w, q), (x[0], x, w, q), (x, x[:3], w, q), (x, x, w[:500], q), (x, x, w, q[:3]), (x, x, w, q[:, :-2]),
              (x, x, w, q.int()), (x.cpu(), x, w, q), (x[:, ::2], x, w, q)):
        with pytest.raises(ValueError):
            qmm.qmm_add_rmsnorm_quantize("q8_0", a[0], a[1], a[2], 1e-5, a[3])
    for over in (dict(sum=x[:3]), dict(h=x.double())):
        with pytest.raises(ValueError):
            qmm.qmm_add_rmsnorm_quantize("q8_0", x, x, w, 1e-5, q, **over)
    with pytest.raises(qmm.QmmError):
        qmm.qmm_add_rmsnorm_quantize("q8_0", x, x, w, 1e-5)
