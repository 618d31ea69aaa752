"""The experts' gated and summed products on the GPU against their definitions in 64 bits (tests/experts_plain.py)."""
import numpy as np
import pytest

import experts_plain as plain
import oracle
import workloads

torch = pytest.importorskip("torch")
import block_quantized_weight_q8_gb300 as qmm  # noqa: E402

pytestmark = pytest.mark.gpu
TYPES = qmm.WEIGHT_TYPES


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.fail("these tests need a CUDA GPU")
    qmm.build()
    qmm.load()
    yield
    assert qmm.qmm_device_status(clear=True) == 0


def dev(a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()


def host(t):
    torch.cuda.synchronize()
    return t.cpu().numpy()


def weights_of(wtype, E, N, K, seed):
    w = workloads.weights_f32(E * N, K, seed=seed, row_jitter=True)
    return oracle.quantize(wtype, w).reshape(E, N, -1)


def picks(T, k, E, seed, absent=0.0):
    rng = np.random.default_rng(seed)
    ids = np.stack([rng.choice(E, k, replace=k > E) for _ in range(T)]).astype(np.int32)
    ids[rng.random((T, k)) < absent] = -1
    return ids


def scratch_of(wtype, T, k, E, N, K):
    n = qmm.qmm_experts_scratch_bytes(wtype, T, k, E, N, K)
    assert n > 0
    return torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda"), n  # bytes that read as NaN


def run_glu(wtype, T, k, E, N, K, kind="silu", absent=0.0, ids=None, seed=1):
    Wg, Wu = weights_of(wtype, E, N, K, seed), weights_of(wtype, E, N, K, seed + 1)
    xq = oracle.quantize(plain.act_of(wtype), workloads.activations_f32(T, K, seed=seed + 2))
    ids = picks(T, k, E, seed + 3, absent) if ids is None else ids
    h = torch.full((T, k, N), float("nan"), device="cuda")
    scratch, n = scratch_of(wtype, T, k, E, N, K)
    qmm.qmm_experts_glu(wtype, dev(Wg), dev(Wu), dev(xq), dev(ids), h, scratch, n, gate=kind)
    want, off = plain.glu(wtype, Wg, Wu, xq, ids, kind, K)
    got = host(h).astype(np.float64)
    bad = ~(np.abs(got - want) <= off)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4].tolist(), np.nanmax(np.abs(got - want) / (off + 1e-30)))
    return got


def run_sum(wtype, T, k, E, N, K, absent=0.0, weighted=True, residual=True, ids=None, seed=11):
    rng = np.random.default_rng(seed)
    W = weights_of(wtype, E, N, K, seed)
    h = workloads.activations_f32(T * k, K, seed=seed + 1).reshape(T, k, K)
    ids = picks(T, k, E, seed + 3, absent) if ids is None else ids
    h[(ids < 0) | (ids >= E)] = np.nan  # without effect
    w = rng.random((T, k)).astype(np.float32) if weighted else None
    r = rng.standard_normal((T, N)).astype(np.float32) if residual else None
    y = torch.full((T, N), float("nan"), device="cuda")
    scratch, n = scratch_of(wtype, T, k, E, N, K)
    qmm.qmm_experts_sum(wtype, dev(W), dev(h), dev(ids), dev(w), y, scratch, n, residual=dev(r))
    want, off = plain.summed(wtype, W, h, ids, w, r, K)
    got = host(y).astype(np.float64)
    bad = ~(np.abs(got - want) <= off)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4].tolist(), np.nanmax(np.abs(got - want) / (off + 1e-30)))


def K_of(wtype, K):
    return -(-K // 256) * 256 if wtype.endswith("_K") else K


# one token, a few, many; rows that end inside every tile; rows of every alignment that blocks can have
SHAPES = [(1, 8, 9, 100, 512), (1, 1, 1, 1, 256), (3, 2, 5, 77, 896), (40, 3, 4, 129, 768), (150, 2, 3, 65, 1024),
          (97, 4, 13, 33, 1280), (300, 1, 2, 40, 288)]


@pytest.mark.parametrize("wtype", TYPES)
@pytest.mark.parametrize("T,k,E,N,K", SHAPES)
def test_glu(wtype, T, k, E, N, K):
    run_glu(wtype, T, k, E, N, K_of(wtype, K), kind="gelu" if T % 2 else "silu")


@pytest.mark.parametrize("wtype", TYPES)
@pytest.mark.parametrize("T,k,E,N,K", SHAPES)
def test_sum(wtype, T, k, E, N, K):
    run_sum(wtype, T, k, E, N, K_of(wtype, K), weighted=T != 3, residual=T != 40)


@pytest.mark.parametrize("T", [1, 5, 64, 200])
def test_choices_that_are_not_there(T):
    ids = picks(T, 4, 6, 5, absent=0.4)
    ids[T // 2] = -1  # a token without any
    got = run_glu("q4_K", T, 4, 6, 50, 512, ids=ids)
    assert (got[ids < 0] == 0).all()
    run_sum("q6_K", T, 4, 6, 50, 512, ids=ids)
    run_sum("q6_K", T, 4, 6, 50, 512, ids=ids, residual=False)
    run_glu("q8_0", T, 4, 6, 50, 512, ids=np.full_like(ids, -1))
    run_sum("q8_0", T, 4, 6, 50, 512, ids=np.full_like(ids, -7))


@pytest.mark.parametrize("T", [2, 90])
def test_an_index_beyond_the_experts(T):
    ids = picks(T, 2, 5, 5)
    ids[0, 1], ids[T - 1, 0] = 5, 1 << 30
    assert qmm.qmm_device_status(clear=True) == 0
    got = run_glu("q4_0", T, 2, 5, 40, 512, ids=ids)
    assert (got[0, 1] == 0).all()
    assert qmm.qmm_device_status(clear=True) == 2
    run_sum("q4_0", T, 2, 5, 40, 512, ids=ids)
    assert qmm.qmm_device_status(clear=True) == 2


@pytest.mark.parametrize("T", [1, 30, 260])
def test_the_same_expert_more_than_once(T):
    ids = np.full((T, 3), 2, np.int32)
    run_glu("q5_K", T, 3, 4, 70, 768, ids=ids)
    run_sum("q5_K", T, 3, 4, 70, 768, ids=ids)


@pytest.mark.parametrize("wtype,T,k,E,N,K", [("q4_0", 700, 2, 1, 200, 512), ("q4_K", 1100, 4, 20, 150, 768),
                                             ("q8_0", 513, 8, 300, 64, 256), ("q2_K", 64, 64, 70, 30, 256),
                                             ("q6_K", 2, 64, 1024, 16, 256)])
def test_many(wtype, T, k, E, N, K):
    run_glu(wtype, T, k, E, N, K)
    run_sum(wtype, T, k, E, N, K)


@pytest.mark.parametrize("wtype,K", [("q8_0", 12288), ("q4_K", 14336), ("q2_K", 8192), ("q5_1", 4864)])
@pytest.mark.parametrize("T", [1, 33])
def test_long_rows(wtype, K, T):
    run_glu(wtype, T, 2, 3, 24, K)
    run_sum(wtype, T, 2, 3, 24, K)


def test_rows_too_long_for_one_cta():
    """8 rows of 65536 values do not fit beside the weights."""
    run_sum("q4_0", 1, 8, 2, 5, 65536)


def test_many_rows_of_weights():
    """More output rows than one CTA keeps sums of."""
    run_glu("q4_0", 3, 1, 1, 40000, 32)
    run_sum("q4_0", 3, 2, 1, 40000, 32)


@pytest.mark.parametrize("T", [1, 50])
def test_in_place_and_the_same_every_time(T):
    E, k, N, K = 6, 3, 256, 512
    W = dev(weights_of("q6_K", E, N, K, 1))
    h = dev(workloads.activations_f32(T * k, K, seed=2).reshape(T, k, K))
    ids, w = dev(picks(T, k, E, 3)), torch.rand(T, k, device="cuda")
    r = torch.randn(T, N, device="cuda")
    scratch, n = scratch_of("q6_K", T, k, E, N, K)
    first = torch.empty_like(r)
    qmm.qmm_experts_sum("q6_K", W, h, ids, w, first, scratch, n, residual=r)
    for _ in range(3):
        y = r.clone()
        qmm.qmm_experts_sum("q6_K", W, h, ids, w, y, scratch, n, residual=y)
        assert torch.equal(y, first)


@pytest.mark.parametrize("T", [1, 64])
def test_captured_with_other_ids(T):
    """A captured call serves ids that are written after the capture, on the stream of the capture."""
    E, k, N, K = 7, 2, 96, 512
    Wg, Wu = weights_of("q4_K", E, N, K, 1), weights_of("q4_K", E, N, K, 2)
    xq = oracle.quantize("q8_K", workloads.activations_f32(T, K, seed=3))
    g, u, x = dev(Wg), dev(Wu), dev(xq)
    ids, h = dev(picks(T, k, E, 4)), torch.empty(T, k, N, device="cuda")
    scratch, n = scratch_of("q4_K", T, k, E, N, K)
    qmm.qmm_experts_glu("q4_K", g, u, x, ids, h, scratch, n)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        qmm.qmm_experts_glu("q4_K", g, u, x, ids, h, scratch, n)
    for seed in (8, 9):
        new = picks(T, k, E, seed, absent=0.3)
        ids.copy_(dev(new))
        h.fill_(float("nan"))
        graph.replay()
        want, off = plain.glu("q4_K", Wg, Wu, xq, new, "silu", K)
        assert (np.abs(host(h) - want) <= off).all()


def test_refusals_of_the_binding():
    E, k, N, K, T = 4, 2, 64, 512, 3
    W = torch.zeros(E, N, qmm.qmm_row_bytes("q4_K", K), dtype=torch.uint8, device="cuda")
    x = torch.zeros(T, qmm.qmm_row_bytes("q8_K", K), dtype=torch.uint8, device="cuda")
    ids, h = torch.zeros(T, k, dtype=torch.int32, device="cuda"), torch.zeros(T, k, N, device="cuda")
    scratch, n = scratch_of("q4_K", T, k, E, N, K)
    good = dict(Wg=W, Wu=W, xq=x, ids=ids, h=h, scratch=scratch)
    for name, bad in (("Wg", W[0]), ("Wg", W[:, :, :100]), ("Wu", W[:, :32]), ("Wu", W.int()), ("xq", x[:2]), ("xq", x[:, :-4]),
                      ("ids", ids.long()), ("ids", ids[:, :1]), ("ids", ids.t()), ("h", h[:, :1]), ("h", h.double()),
                      ("h", h[..., :32]), ("scratch", scratch[:-1]), ("ids", ids.cpu()), ("h", h[0])):
        a = dict(good, **{name: bad})
        with pytest.raises(ValueError):
            qmm.qmm_experts_glu("q4_K", a["Wg"], a["Wu"], a["xq"], a["ids"], a["h"], a["scratch"], n)
    D = torch.zeros(E, K, qmm.qmm_row_bytes("q4_K", 256), dtype=torch.uint8, device="cuda")
    hh, y, w = torch.zeros(T, k, 256, device="cuda"), torch.zeros(T, K, device="cuda"), torch.zeros(T, k, device="cuda")
    scratch, n = scratch_of("q4_K", T, k, E, K, 256)
    good = dict(W=D, h=hh, ids=ids, weights=w, y=y, scratch=scratch, residual=y)
    for name, bad in (("W", D[0]), ("W", D[..., :-1]), ("h", hh[0]), ("h", hh[:2]), ("ids", ids[0]), ("weights", w[0]),
                      ("weights", w.half()), ("y", y[:, :-1]), ("y", y.half()), ("residual", y[:1]), ("scratch", scratch[:-1])):
        a = dict(good, **{name: bad})
        with pytest.raises(ValueError):
            qmm.qmm_experts_sum("q4_K", a["W"], a["h"], a["ids"], a["weights"], a["y"], a["scratch"], n, residual=a["residual"])
