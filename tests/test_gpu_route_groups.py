"""Groups whose worth is the sum of two keys that nearly cancel: f32 sums of such keys are off by more than their distance to
the groups that are open and closed, wherever the group stands, and the choice has to be that of 64 bits."""
import numpy as np
import pytest

from test_gpu_route import check, gpu  # noqa: F401

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


def near_groups(T, groups, each, size, step, score, seed):
    """(logits, bias): in every token the groups' worths are some permutation of steps of `step` apart; the first two experts
    of every other group have biases +size and -size, further experts lie far below."""
    rng = np.random.default_rng(seed)
    bias = np.zeros((groups, each), np.float32)
    bias[::2, 0], bias[::2, 1] = size, -size
    bias[:, 2:] = -3 * size - 10
    worth = np.stack([rng.permutation(groups) for _ in range(T)]) * step + 0.7
    first = rng.uniform(0.3, 0.4, (T, groups))
    p = np.full((T, groups, each), 0.05)
    p[..., 0], p[..., 1] = first, worth - first
    p = p.reshape(T, -1)
    logits = np.log(p / (1 - p)) if score == "sigmoid" else np.log(p)
    return logits.astype(np.float32), bias.reshape(-1)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups,each,kept", [(3, 2, 1), (4, 2, 2), (5, 3, 3), (8, 32, 4), (8, 4, 7), (40, 3, 5), (64, 2, 20)])
@pytest.mark.parametrize("size,step", [(1000.0, 1e-5), (30.0, 1.2e-6), (5000.0, 1e-4), (1e-3, 1e-5)])
def test_worths_of_cancelling_keys(score, groups, each, kept, size, step):
    """Softmax scores are a share of their sum, and so are the distances."""
    logits, bias = near_groups(300, groups, each, size, step, score, groups + kept)
    check(logits, min(2 * kept, 4), bias, score, groups, kept, top=2)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_a_group_below_the_cut(score):
    """The first group's f32 worth falls below two others that lie 2e-5 apart, between which f32 is sure."""
    rng = np.random.default_rng(5)
    T = 3000
    bias = np.array([1000, -1000, -0.0076, 0, 0.0134, 0], np.float32)
    p = np.full((T, 6), 0.3)
    p[:, 0] += rng.uniform(-0.05, 0.05, T)
    base = p[:, 0] + p[:, 1]
    p[:, 3] = base - 1e-5 - p[:, 2] + 0.0076
    p[:, 5] = base - 3e-5 - p[:, 4] - 0.0134
    logits = np.log(p / (1 - p)) if score == "sigmoid" else np.log(p / p.sum(1, keepdims=True))
    check(logits.astype(np.float32), 2, bias, score, 3, 1, top=2)


def test_infinite_and_overflowing_worths():
    """Biases of +inf, and of the largest f32 (whose sums of two are finite in 64 bits alone)."""
    rng = np.random.default_rng(6)
    logits = rng.standard_normal((50, 32)).astype(np.float32)
    most = np.finfo(np.float32).max
    for values in ((np.inf, 0.0), (most, -most), (most, most), (-most, -most), (np.inf, -most), (0.0, -most)):
        bias = (0.1 * rng.standard_normal(32)).astype(np.float32)
        bias[[0, 1]] = values
        bias[[20, 22]] = values
        for kept in (1, 2, 3):
            check(logits, 4, bias, "sigmoid", 4, kept, top=2)
