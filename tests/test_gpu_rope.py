"""Rotary positions on the GPU against their definition in 64 bits.

Tolerance: a result is the exact value rounded once (2^-24 of it) but for the angle's and products' pairs, 2^-42 of
m (|a| + |b|), and the reference's own binary64 angle (2^-53 of a turn, far below)."""
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


def host(t):
    torch.cuda.synchronize()
    return t.cpu().numpy()


def close(got, want, size):
    err = np.abs(got.astype(np.float64) - want)
    tol = 2.0 ** -24 * np.abs(want) + 2.0 ** -42 * size + 2.0 ** -149
    assert np.all(err <= tol), (np.max(err / np.maximum(tol, 1e-300)), np.argwhere(err > tol)[:4].tolist())


@pytest.mark.parametrize("scaling,kw", [("plain", {}), ("linear", dict(factor=4.0)),
                                        ("bands", dict(factor=8.0, orig_len=8192.0, lo=1.0, hi=4.0)),
                                        ("yarn", dict(factor=16.0, orig_len=4096.0, lo=1.0, hi=32.0))])
@pytest.mark.parametrize("n_rot,base", [(2, 10000.0), (20, 10000.0), (128, 500000.0), (256, 1e7)])
def test_freqs(scaling, kw, n_rot, base):
    """pow, the blend and 1 / 2 pi: under 16 roundings of 2^-53; the table's unit 2^-64 and the reading of it as a
    double 2^-53."""
    t = torch.zeros(n_rot // 2, dtype=torch.int64, device="cuda")
    qmm.qmm_rope_freqs(t, base, scaling, **kw)
    got = host(t).view(np.uint64).astype(np.float64) / 2.0 ** 64
    want = plain.freqs(n_rot, base, scaling, **kw) / (2 * np.pi)
    assert np.all(np.abs(got - want) <= 16 * 2.0 ** -53 * want + 2.0 ** -63), np.max(np.abs(got - want) / want)


CASES = [(1, 1, 16, 16, "half"), (1, 32, 128, 128, "half"), (3, 14, 64, 64, "interleaved"), (7, 5, 80, 20, "half"),
         (7, 5, 80, 20, "interleaved"), (5, 3, 48, 12, "half"), (33, 2, 96, 64, "half"), (2, 40, 256, 256, "interleaved"),
         (2, 40, 256, 256, "half"), (130, 1, 32, 2, "half"), (130, 1, 32, 30, "interleaved"), (513, 4, 112, 28, "half")]


@pytest.mark.parametrize("T,H,hd,n_rot,layout", CASES)
@pytest.mark.parametrize("inverse", [False, True])
def test_rotation(T, H, hd, n_rot, layout, inverse):
    rng = np.random.default_rng(T * 7 + hd)
    x = rng.standard_normal((T, H, hd)).astype(np.float32)
    pos = rng.integers(-1000, 1 << 20, size=T).astype(np.int32)
    pos[0] = 0
    if T > 2:
        pos[1], pos[2] = 2 ** 31 - 1, -(2 ** 31)
    table = plain.turns(plain.freqs(n_rot))
    m = float(np.float32(1.2772589))
    want, size = plain.rotate(x, pos, table, layout, m, inverse)
    rope = qmm.RopeSpec(dev(table), layout, m)
    y = torch.full((T, H, hd), float("nan"), device="cuda")
    qmm.qmm_rope(rope, dev(x), y, dev(pos), inverse=inverse)
    got = host(y)
    close(got, want, size)
    assert np.array_equal(got[..., n_rot:], x[..., n_rot:])
    z = dev(x)  # in place
    qmm.qmm_rope(rope, z, z, dev(pos), inverse=inverse)
    assert np.array_equal(host(z).view(np.int32), got.view(np.int32))


def test_position_zero_copies_and_results_are_the_nearest():
    """Angle 0 gives x itself; elsewhere the f32 nearest to the 64-bit value, but for what lies within 2^-42 of a border
    (about one value in 2^16 at most)."""
    rng = np.random.default_rng(3)
    x = rng.standard_normal((400, 8, 128)).astype(np.float32)
    table = plain.turns(plain.freqs(128))
    rope = qmm.RopeSpec(dev(table))
    y = torch.empty(x.shape, device="cuda")
    qmm.qmm_rope(rope, dev(x), y, torch.zeros(400, dtype=torch.int32, device="cuda"))
    assert np.array_equal(host(y), x)
    pos = rng.integers(0, 1 << 17, size=400).astype(np.int32)
    qmm.qmm_rope(rope, dev(x), y, dev(pos))
    want, _ = plain.rotate(x, pos, table)
    off = np.mean(host(y) != want.astype(np.float32))
    assert off <= 2.0 ** -13, off


def test_quarter_turns_are_exact():
    """Table entries of whole quarters of a turn: 0 and +-1 are exact, so values only move and change sign."""
    table = np.array([1 << 62, 1 << 61], dtype=np.int64)  # a quarter and an eighth per position
    x = np.random.default_rng(1).standard_normal((4, 2, 16)).astype(np.float32)
    y = torch.empty(x.shape, device="cuda")
    qmm.qmm_rope(qmm.RopeSpec(dev(table)), dev(x), y, dev(np.array([0, 2, 4, 6], dtype=np.int32)))
    got = host(y)
    for t, turn in enumerate((0, 2, 4, 6)):
        for i, quarters in ((0, turn % 4), (1, turn // 2 % 4)):
            a, b = x[t, :, i], x[t, :, i + 2]
            want = [(a, b), (-b, a), (-a, -b), (b, -a)][quarters]
            assert np.array_equal(got[t, :, i], want[0]) and np.array_equal(got[t, :, i + 2], want[1])


def test_infinities_and_nan_stay_with_their_pair():
    x = np.random.default_rng(2).standard_normal((2, 2, 32)).astype(np.float32)
    ref = x.copy()
    x[0, 0, 3], x[0, 1, 5], x[1, 0, 2] = np.inf, np.nan, 3e38
    table = plain.turns(plain.freqs(16))
    y = torch.empty(x.shape, device="cuda")
    qmm.qmm_rope(qmm.RopeSpec(dev(table)), dev(x), y, dev(np.array([5, 9], dtype=np.int32)))
    got = host(y)
    want, size = plain.rotate(ref, [5, 9], table)
    assert np.isinf(got[0, 0, 3]) and np.isinf(got[0, 0, 11])
    assert np.isnan(got[0, 1, 5]) and np.isnan(got[0, 1, 13])
    big, _ = plain.rotate(x, [5, 9], table)
    assert np.allclose(got[1, 0, [2, 10]], big[1, 0, [2, 10]], rtol=1e-6)
    for h, i in ((0, 3), (0, 11), (1, 5), (1, 13)):
        got[0, h, i] = want[0, h, i]
    got[1, 0, [2, 10]] = want[1, 0, [2, 10]]
    close(got, want, size)


def test_strided_rows_of_a_fused_projection():
    T, Hq, Hkv, hd = 9, 6, 2, 64
    rng = np.random.default_rng(4)
    buf = rng.standard_normal((T, Hq + 2 * Hkv, hd)).astype(np.float32)
    pos = rng.integers(0, 5000, size=T).astype(np.int32)
    table = plain.turns(plain.freqs(hd))
    t = dev(buf)
    qmm.qmm_rope(qmm.RopeSpec(dev(table)), t[:, Hq: Hq + Hkv], t[:, Hq: Hq + Hkv], dev(pos))
    got = host(t)
    want, size = plain.rotate(buf[:, Hq: Hq + Hkv], pos, table)
    close(got[:, Hq: Hq + Hkv], want, size)
    assert np.array_equal(got[:, :Hq], buf[:, :Hq]) and np.array_equal(got[:, Hq + Hkv:], buf[:, Hq + Hkv:])


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_gradient(layout):
    """The gradient of sum(g * rope(x)) is rope(g, inverse): against differences (the map is linear, so a central
    difference of any step is exact but for the outputs' roundings, 2^-24 of each term) and as an inner product."""
    T, H, hd, n_rot = 5, 3, 48, 32
    rng = np.random.default_rng(6)
    x, g = (rng.standard_normal((T, H, hd)).astype(np.float32) for _ in range(2))
    pos = dev(rng.integers(0, 70000, size=T).astype(np.int32))
    rope = qmm.RopeSpec(dev(plain.turns(plain.freqs(n_rot))), layout, 1.25)

    def run(a, inverse=False):
        y = torch.empty(T, H, hd, device="cuda")
        qmm.qmm_rope(rope, dev(a), y, pos, inverse=inverse)
        return host(y).astype(np.float64)
    grad = run(g, inverse=True)
    for t, h, d in ((0, 0, 0), (1, 2, 17), (4, 1, 31), (2, 0, 40)):
        e = np.zeros_like(x)
        e[t, h, d] = 1.0
        up, down = run(x + e), run(x - e)
        diff = np.sum(g * (up - down)) / 2
        tol = 2.0 ** -24 * (np.sum(np.abs(g) * (np.abs(up) + np.abs(down))[:]) + 4 * np.abs(grad[t, h, d]) + 4)
        assert abs(diff - grad[t, h, d]) <= tol
    left, right = np.sum(run(x) * g), np.sum(x * grad)
    assert abs(left - right) <= 2.0 ** -23 * np.sum(np.abs(run(x) * g) + np.abs(x * grad))


def test_captured_and_on_another_stream():
    T, H, hd = 4, 8, 128
    rng = np.random.default_rng(8)
    table = plain.turns(plain.freqs(hd))
    rope, x, pos = qmm.RopeSpec(dev(table)), dev(np.zeros((T, H, hd), np.float32)), dev(np.zeros(T, np.int32))
    y = torch.empty_like(x)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        qmm.qmm_rope(rope, x, y, pos)
    for k in range(2):
        xh, ph = rng.standard_normal((T, H, hd)).astype(np.float32), rng.integers(0, 9999, size=T).astype(np.int32)
        x.copy_(dev(xh))
        pos.copy_(dev(ph))
        graph.replay()
        close(host(y), *plain.rotate(xh, ph, table))


def test_binding_refuses():
    x, pos = torch.zeros(2, 2, 32, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda")
    rope = qmm.RopeSpec(dev(plain.turns(plain.freqs(32))))
    for bad in ((x.half(), x, pos), (x, x.cpu(), pos), (x, torch.zeros(2, 3, 32, device="cuda"), pos),
                (x, x, pos.long()), (x, x, pos[:1]), (x.transpose(1, 2), x, pos)):
        with pytest.raises(ValueError):
            qmm.qmm_rope(rope, *bad)
