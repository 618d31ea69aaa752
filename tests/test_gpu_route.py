"""The choice of experts on the GPU against sorting in 64 bits (tests/experts_plain.py): ids equal, weights f32."""
import numpy as np
import pytest

import experts_plain as plain

torch = pytest.importorskip("torch")
import block_quantized_weight_q8_gb300 as qmm  # noqa: E402

pytestmark = pytest.mark.gpu
INF = float("inf")


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


def check(logits, k, bias=None, score="softmax", groups=1, kept=1, top=1, renorm=True, scale=1.0, tensor=None):
    T, E = logits.shape
    ids = torch.full((T, k), 77, dtype=torch.int32, device="cuda")
    w = torch.full((T, k), float("nan"), device="cuda")
    qmm.qmm_route(dev(logits) if tensor is None else tensor, ids, w, score=score, bias=dev(bias), groups=groups,
                  groups_kept=kept, group_top=top, renorm=renorm, scale=scale)
    want, weights = plain.route(logits, bias, k, score, groups, kept, top, renorm, scale)
    torch.cuda.synchronize()
    assert np.array_equal(ids.cpu().numpy(), want)
    # a score: an exponential (2 units of 2^-23, its argument's rounding times its size, at most 90) over a sum of up to
    # 1024 (36 roundings), the quotients and the scale; and what falls below the normal range
    got = w.cpu().numpy().astype(np.float64)
    assert (np.abs(got - weights) <= 2.0 ** -24 * (2 * 90 + 2 * 36 + 16) * weights + 2e-37 * abs(scale)).all()
    return want, got


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("T,E,k,groups,kept,top", [
    (1, 1, 1, 1, 1, 1), (1, 8, 2, 1, 1, 1), (3, 33, 32, 1, 1, 1), (65, 64, 8, 1, 1, 1), (200, 100, 6, 5, 2, 1),
    (130, 256, 8, 8, 4, 2), (70, 160, 6, 8, 3, 2), (50, 64, 3, 64, 5, 2), (41, 1024, 8, 16, 3, 2), (1500, 40, 4, 40, 4, 1),
    (20, 510, 10, 3, 1, 2), (9, 1000, 32, 1, 1, 1)])
def test_against_sorting(score, biased, T, E, k, groups, kept, top):
    rng = np.random.default_rng(T * 1000 + E)
    logits = (1.5 * rng.standard_normal((T, E))).astype(np.float32)
    bias = (0.1 * rng.standard_normal(E)).astype(np.float32) if biased else None
    check(logits, k, bias, score, groups, kept, top, renorm=T % 2 == 1, scale=2.5 if biased else 1.0)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups,kept,top", [(1, 1, 1), (6, 2, 2), (6, 2, 1)])
def test_equal_keys_go_to_the_lower_index(score, groups, kept, top):
    rng = np.random.default_rng(3)
    logits = rng.integers(-2, 3, (120, 48)).astype(np.float32)
    logits[0] = 0.0
    logits[1, ::2] = -0.0
    for bias in (None, np.zeros(48, np.float32), rng.integers(0, 2, 48).astype(np.float32)):
        check(logits, 7, bias, score, groups, kept, top)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_keys_a_rounding_apart(score):
    """Keys that differ by less than f32 scores can tell: the choice is that of 64 bits."""
    rng = np.random.default_rng(4)
    base = rng.standard_normal((300, 1)).astype(np.float32)
    steps = rng.integers(0, 6, (300, 96)).astype(np.float32)
    logits = (base + steps * 2.0 ** -22).astype(np.float32)
    bias = (rng.integers(0, 3, 96) * 2.0 ** -23).astype(np.float32)
    check(logits, 8, bias, score)
    check(logits, 8, bias, score, groups=8, kept=3, top=2)
    check(logits, 8, None, score, groups=8, kept=3, top=2)
    big = (1000.0 * rng.standard_normal(96)).astype(np.float32)
    check(logits, 8, big, score, groups=8, kept=3, top=2)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups,kept,top", [(1, 1, 1), (4, 2, 2), (4, 2, 1)])
@pytest.mark.parametrize("biased", [False, True])
def test_closed_experts_and_empty_rows(score, groups, kept, top, biased):
    rng = np.random.default_rng(5)
    logits = rng.standard_normal((60, 64)).astype(np.float32)
    logits[rng.random((60, 64)) < 0.5] = -INF
    logits[7] = -INF                       # a token without any
    logits[8, 3:] = -INF                   # fewer than k
    logits[9] = np.where(np.arange(64) % 16 == 5, logits[9], -INF)  # one in each group
    logits[10, ::3] = np.nan
    logits[11] = np.nan
    logits[12, 20] = INF
    logits[13, [4, 40]] = INF
    logits[14] = np.finfo(np.float32).min
    logits[15, :32] = np.finfo(np.float32).min
    bias = (0.1 * rng.standard_normal(64)).astype(np.float32) if biased else None
    ids, w = check(logits, 6, bias, score, groups, kept, top, renorm=True)
    assert (ids[7] == -1).all() and (w[7] == 0).all() and (ids[8] >= 0).sum() == np.isfinite(logits[8]).sum()
    check(logits, 6, bias, score, groups, kept, top, renorm=False)
    if biased:
        bias[::5] = -INF
        bias[3] = np.nan
        check(logits, 6, bias, score, groups, kept, top)


def test_strided_logits_and_streams():
    rng = np.random.default_rng(6)
    wide = rng.standard_normal((90, 150)).astype(np.float32)
    t = dev(wide)
    check(wide[:, 20:84], 4, tensor=t[:, 20:84])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        check(wide[:, 1:66], 4, tensor=t[:, 1:66])
    torch.cuda.current_stream().wait_stream(s)


def test_many_tokens():
    rng = np.random.default_rng(7)
    logits = rng.standard_normal((20000, 16)).astype(np.float32)
    check(logits, 2, score="sigmoid", bias=(0.1 * rng.standard_normal(16)).astype(np.float32))


def test_refusals_of_the_binding():
    x = torch.zeros(5, 16, device="cuda")
    ids, w = torch.zeros(5, 2, dtype=torch.int32, device="cuda"), torch.zeros(5, 2, device="cuda")
    for a in ((x.half(), ids, w), (x[0], ids, w), (x.t(), ids, w), (x, ids[0], w), (x, ids.long(), w), (x, ids, w[:, :1]),
              (x, ids, w.double()), (x.cpu(), ids, w), (x, ids[:4], w)):
        with pytest.raises(ValueError):
            qmm.qmm_route(*a)
    with pytest.raises(ValueError):
        qmm.qmm_route(x, ids, w, bias=torch.zeros(15, device="cuda"))
    with pytest.raises(qmm.QmmError):
        qmm.qmm_route(x, ids, w, groups=3)
