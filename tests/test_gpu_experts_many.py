"""The experts' products at so many rows that they go to the tensor cores: odd sizes, absent and repeated choices, weights
of extreme scales, streams, captured calls; and a layer's operators in a row."""
import numpy as np
import pytest

import experts_plain as plain
import oracle
import workloads
from test_gpu_experts import K_of, TYPES, dev, gpu, host, picks, run_glu, run_sum, scratch_of, weights_of  # noqa: F401

torch = pytest.importorskip("torch")
import block_quantized_weight_q8_gb300 as qmm  # noqa: E402

pytestmark = pytest.mark.gpu

# whole chunks; part of one alone (one block, nine); five and a part, 41 blocks, where tiles end inside
SHAPES = [(1000, 2, 3, 129, 1024), (2000, 1, 2, 77, 288), (4000, 1, 1, 130, 32), (400, 4, 13, 100, 1312)]


@pytest.mark.parametrize("wtype", TYPES)
@pytest.mark.parametrize("T,k,E,N,K", SHAPES)
def test_glu(wtype, T, k, E, N, K):
    run_glu(wtype, T, k, E, N, K_of(wtype, K), kind="gelu" if T == 400 else "silu")


@pytest.mark.parametrize("wtype", TYPES)
@pytest.mark.parametrize("T,k,E,N,K", SHAPES)
def test_sum(wtype, T, k, E, N, K):
    run_sum(wtype, T, k, E, N, K_of(wtype, K), weighted=T != 400, residual=T != 2000)


@pytest.mark.parametrize("wtype", ["q4_0", "q5_1", "q4_K", "q6_K"])
def test_choices_that_are_not_there(wtype):
    T, k, E, N, K = 1100, 3, 6, 70, 1024
    ids = picks(T, k, E, 5, absent=0.4)
    ids[ids == 4] = -1  # an expert without rows
    ids[T // 2] = -1    # a token without experts
    got = run_glu(wtype, T, k, E, N, K, ids=ids)
    assert (got[ids < 0] == 0).all()
    run_sum(wtype, T, k, E, N, K, ids=ids)
    run_sum(wtype, T, k, E, N, K, ids=ids, residual=False)
    none = np.full_like(ids, -3)
    assert (run_glu(wtype, T, k, E, N, K, ids=none) == 0).all()
    run_sum(wtype, T, k, E, N, K, ids=none)


def test_an_index_beyond_the_experts():
    T, k, E, N, K = 1200, 2, 5, 90, 1024
    ids = picks(T, k, E, 5)
    ids[7, 1], ids[T - 1, 0] = E, 1 << 30
    assert qmm.qmm_device_status(clear=True) == 0
    got = run_glu("q4_0", T, k, E, N, K, ids=ids)
    assert (got[7, 1] == 0).all() and (got[T - 1, 0] == 0).all()
    assert qmm.qmm_device_status(clear=True) == 2
    run_sum("q4_0", T, k, E, N, K, ids=ids)
    assert qmm.qmm_device_status(clear=True) == 2


@pytest.mark.parametrize("wtype", ["q8_0", "q4_1", "q5_K", "q6_K"])
def test_the_same_expert_more_than_once(wtype):
    ids = np.full((700, 3), 2, np.int32)
    run_glu(wtype, 700, 3, 4, 70, 1024, ids=ids)
    run_sum(wtype, 700, 3, 4, 70, 1024, ids=ids)


# (offset of d, of the minimums' scale, block bytes)
FIELDS = {"q4_0": (0, None, 18), "q8_0": (0, None, 34), "q4_1": (0, 2, 20), "q5_0": (0, None, 22), "q5_1": (0, 2, 24),
          "q4_K": (0, 2, 144), "q5_K": (0, 2, 176), "q6_K": (208, None, 210), "q2_K": (80, 82, 84)}


def extreme_weights(wtype, E, N, K, seed):
    """(bytes, each row's values, what a value's error is measured by: the largest |scale part| + |minimum| of its 256)."""
    rng = np.random.default_rng(seed)
    at, mat, size = FIELDS[wtype]
    raw = weights_of(wtype, E, N, K, seed).reshape(E * N, -1, size).copy()
    rows, blocks = raw.shape[:2]

    def put(where, values):
        raw[:, :, where:where + 2] = values.astype(np.float16).view(np.uint8).reshape(rows, blocks, 2)

    # by the row: all alike, signs, single large blocks, zeros, subnormals, the largest
    d = np.exp(rng.uniform(-8, 2, (rows, blocks)))
    for r in range(rows):
        d[r] = (d[r], -d[r], np.where(rng.random(blocks) < 0.1, 60000.0, 1e-3), np.where(rng.random(blocks) < 0.5, 0.0, d[r]),
                np.full(blocks, 6e-8), np.full(blocks, 65504.0), np.zeros(blocks), -np.full(blocks, 3e-6))[r % 8]
    put(at, d)
    if mat is not None:
        m = np.exp(rng.uniform(-8, 2, (rows, blocks)))
        for r in range(rows):
            m[r] = (m[r], -m[r], np.zeros(blocks), np.full(blocks, 65504.0), np.full(blocks, 6e-8))[r % 5]
        put(mat, m)
        if wtype.endswith("_K"):  # every third row: minimums of zero under whatever scale
            none = raw[::3]
            if wtype == "q2_K":
                none[:, :, :16] &= 0x0F
            else:
                none[:, :, 8:12] = 0
                none[:, :, 12:16] &= 0x0F

    def values(drop):
        part = raw.copy()
        for o in drop:
            part[:, :, o:o + 2] = 0
        return oracle.dequantize(wtype, part.reshape(rows, -1), K)

    part = np.abs(values([] if mat is None else [mat]))
    if mat is not None:
        part = part + np.abs(values([at]))
    pad = -K % 256
    part = np.pad(part, ((0, 0), (0, pad))).reshape(rows, -1, 256).max(-1, keepdims=True).repeat(256, -1).reshape(rows, -1)[:, :K]
    return raw.reshape(E, N, -1), values([]).reshape(E, N, K), part.reshape(E, N, K)


@pytest.mark.parametrize("wtype", TYPES)
def test_extreme_scales(wtype):
    """An output's error against 1e-5 of the sum of its values' shares: the operands' 2^-21 each and at most 57 steps
    truncated to 2^-23 of what the sum has grown to are 2^-20 + 57 2^-23 = 7.8e-6."""
    T, k, E, N, K = 1500, 1, 2, 120, 1024
    W, values, part = extreme_weights(wtype, E, N, K, 3)
    h = workloads.activations_f32(T, K, seed=4).reshape(T, 1, K)
    ids = picks(T, 1, E, 5)
    y = torch.empty(T, N, device="cuda")
    scratch, n = scratch_of(wtype, T, 1, E, N, K)
    qmm.qmm_experts_sum(wtype, dev(W), dev(h), dev(ids), None, y, scratch, n)
    got = host(y).astype(np.float64)
    act = plain.act_of(wtype)
    x = oracle.dequantize(act, oracle.quantize(act, h[:, 0]), K).astype(np.float64)
    for e in range(E):
        t = ids[:, 0] == e
        want, off = x[t] @ values[e].T.astype(np.float64), 1e-5 * (np.abs(x[t]) @ part[e].T.astype(np.float64))
        bad = ~(np.abs(got[t] - want) <= off + 1e-30)
        assert not bad.any(), (e, int(bad.sum()), np.argwhere(bad)[:4].tolist())


@pytest.mark.parametrize("wtype", ["q8_0", "q5_1", "q4_K", "q6_K"])
def test_infinities_stay_in_their_rows(wtype):
    """A choice's row with infinities or NaN, in the middle of a tile, and weights with an infinite scale: every other
    product is what it is without them."""
    T, k, E, N, K = 1300, 1, 2, 100, 1024
    at, _, size = FIELDS[wtype]
    W = weights_of(wtype, E, N, K, 3)
    h = workloads.activations_f32(T, K, seed=4).reshape(T, 1, K)
    ids = dev(picks(T, 1, E, 5))
    scratch, n = scratch_of(wtype, T, 1, E, N, K)
    clean, y = torch.empty(T, N, device="cuda"), torch.empty(T, N, device="cuda")
    qmm.qmm_experts_sum(wtype, dev(W), dev(h), ids, None, clean, scratch, n)
    h[77, 0, 3], h[600, 0, 1000] = np.inf, np.nan
    W.reshape(E, N, -1, size)[:, 50, 1, at:at + 2] = np.array([np.inf], np.float16).view(np.uint8)
    qmm.qmm_experts_sum(wtype, dev(W), dev(h), ids, None, y, scratch, n)
    got, want = host(y), host(clean)
    assert not np.isfinite(got[:, 50]).any()
    keep = np.ones(T, bool)
    keep[[77, 600]] = False
    cols = np.arange(N) != 50
    assert np.array_equal(got[keep][:, cols], want[keep][:, cols])


def test_two_streams_with_a_workspace_each():
    T, k, E, N, K = 1200, 2, 6, 130, 1024
    W = dev(weights_of("q6_K", E, N, K, 1))
    h = dev(workloads.activations_f32(T * k, K, seed=2).reshape(T, k, K))
    ids = [dev(picks(T, k, E, s)) for s in (3, 4)]
    w = torch.rand(T, k, device="cuda")
    ws = [scratch_of("q6_K", T, k, E, N, K) for _ in ids]
    want = [torch.empty(T, N, device="cuda") for _ in ids]
    for i in range(2):
        qmm.qmm_experts_sum("q6_K", W, h, ids[i], w, want[i], ws[i][0], ws[i][1])
    got = [torch.zeros(T, N, device="cuda") for _ in ids]
    streams = [torch.cuda.Stream() for _ in ids]
    torch.cuda.synchronize()
    for _ in range(5):
        for i in range(2):
            qmm.qmm_experts_sum("q6_K", W, h, ids[i], w, got[i], ws[i][0], ws[i][1], stream=streams[i])
    torch.cuda.synchronize()
    for i in range(2):
        assert torch.equal(got[i], want[i])


def test_two_captured_graphs_share_a_workspace():
    """Replayed in turn on one stream, as two layers of a model would be."""
    T, k, E, N, K = 1100, 2, 5, 96, 1024
    W = [dev(weights_of("q4_K", E, N, K, s)) for s in (1, 2)]
    xq = dev(oracle.quantize("q8_K", workloads.activations_f32(T, K, seed=3)))
    ids = dev(picks(T, k, E, 4))
    scratch, n = scratch_of("q4_K", T, k, E, N, K)
    want = [torch.empty(T, k, N, device="cuda") for _ in W]
    got = [torch.empty(T, k, N, device="cuda") for _ in W]
    for i in range(2):
        qmm.qmm_experts_glu("q4_K", W[i], W[1 - i], xq, ids, want[i], scratch, n)
    torch.cuda.synchronize()
    graphs = []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            qmm.qmm_experts_glu("q4_K", W[i], W[1 - i], xq, ids, got[i], scratch, n)
        graphs.append(g)
    for _ in range(3):
        for t in got:
            t.fill_(float("nan"))
        graphs[0].replay()
        graphs[1].replay()
        torch.cuda.synchronize()
        for i in range(2):
            assert torch.equal(got[i], want[i])


def test_rows_and_bytes_around_stay_as_they_are():
    """A call for the first T tokens of larger buffers writes no more than those, and of the workspace what it asked for."""
    T, k, E, N, K = 1000, 2, 3, 131, 1024
    W = dev(weights_of("q5_0", E, N, K, 1))
    h = dev(workloads.activations_f32((T + 9) * k, K, seed=2).reshape(T + 9, k, K))
    ids = dev(picks(T + 9, k, E, 3))
    y = torch.full((T + 9, N), 7.0, device="cuda")
    n = qmm.qmm_experts_scratch_bytes("q5_0", T, k, E, N, K)
    scratch = torch.full((n + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
    qmm.qmm_experts_sum("q5_0", W, h[:T], ids[:T], None, y[:T], scratch, n)
    torch.cuda.synchronize()
    assert (y[T:] == 7.0).all() and (scratch[n:] == 0xA5).all() and not (y[:T] == 7.0).all()


@pytest.mark.parametrize("T", [2, 6000])
def test_weights_beyond_32_bits_of_bytes(T):
    """1024 experts of 4096 x 1024 Q8_0, 4.6 GB: the last expert's rows, by few and by many choices."""
    E, N, K = 1024, 4096, 1024
    W = torch.zeros(E, N, qmm.qmm_row_bytes("q8_0", K), dtype=torch.uint8, device="cuda")
    last = weights_of("q8_0", 1, N, K, 3)
    W[-1].copy_(dev(last[0]))
    h = workloads.activations_f32(T, K, seed=4).reshape(T, 1, K)
    ids = np.zeros((T, 1), np.int32)
    ids[::2] = E - 1
    y = torch.full((T, N), float("nan"), device="cuda")
    scratch, n = scratch_of("q8_0", T, 1, E, N, K)
    qmm.qmm_experts_sum("q8_0", W, dev(h), dev(ids), None, y, scratch, n)
    got = host(y).astype(np.float64)
    want, off = plain.summed("q8_0", last, h[:40:2], np.zeros((len(h[:40:2]), 1), np.int32), None, None, K)
    assert (np.abs(got[:40:2] - want) <= off).all() and (got[1::2] == 0).all()


def test_outputs_beyond_32_bits_of_bytes():
    """300000 choices of 4096 outputs, 4.9 GB; the last tokens' are looked at."""
    T, k, E, N, K = 150000, 2, 2, 4096, 256
    Wg, Wu = weights_of("q4_K", E, N, K, 1), weights_of("q4_K", E, N, K, 2)
    x = workloads.activations_f32(1000, K, seed=3)
    xq = oracle.quantize("q8_K", x)
    ids = picks(T, k, E, 4)
    h = torch.empty(T, k, N, device="cuda")
    scratch, n = scratch_of("q4_K", T, k, E, N, K)
    qmm.qmm_experts_glu("q4_K", dev(Wg), dev(Wu), dev(np.tile(xq, (T // 1000, 1))), dev(ids), h, scratch, n)
    for t in (0, T - 30):
        want, off = plain.glu("q4_K", Wg, Wu, xq[t % 1000:t % 1000 + 30], ids[t:t + 30], "silu", K)
        assert (np.abs(host(h[t:t + 30]) - want) <= off).all()


@pytest.mark.parametrize("wtype,T", [("q4_K", 1), ("q4_K", 900), ("q8_0", 3), ("q5_1", 700)])
def test_a_layer(wtype, T):
    """The added norm, a router's product, the choice, the gated and the summed products in a row on one stream, captured;
    each step against its definition on what the step before it gave."""
    K, N, E, k = 512, 768, 16, 4
    act = plain.act_of(wtype)
    x, r = workloads.activations_f32(T, K, seed=1), workloads.activations_f32(T, K, seed=2)
    w = np.random.default_rng(3).uniform(0.5, 1.5, K).astype(np.float32)
    R = oracle.quantize("q8_0", workloads.weights_f32(E, K, seed=4))
    Wg, Wu, Wd = weights_of(wtype, E, N, K, 5), weights_of(wtype, E, N, K, 6), weights_of(wtype, E, K, N, 7)
    gx, gr, gw, gR, gg, gu, gd = (dev(a) for a in (x, r, w, R, Wg, Wu, Wd))
    y, hn = torch.empty(T, K, device="cuda"), torch.empty(T, K, device="cuda")
    xq = torch.empty(T, qmm.qmm_row_bytes(act, K), dtype=torch.uint8, device="cuda")
    rq = torch.empty(T, qmm.qmm_row_bytes("q8_0", K), dtype=torch.uint8, device="cuda")
    logits = torch.empty(T, E, device="cuda")
    ids, weights = torch.empty(T, k, dtype=torch.int32, device="cuda"), torch.empty(T, k, device="cuda")
    h, out = torch.empty(T, k, N, device="cuda"), torch.empty(T, K, device="cuda")
    n = max(qmm.qmm_experts_scratch_bytes(wtype, T, k, E, N, K), qmm.qmm_experts_scratch_bytes(wtype, T, k, E, K, N))
    scratch = torch.empty(n, dtype=torch.uint8, device="cuda")

    def layer():
        qmm.qmm_add_rmsnorm_quantize(act, gx, gr, gw, plain.EPS, xq=xq, sum=y, h=hn)
        qmm.quantize("q8_0", hn, rq, T, K)
        qmm.matmul("q8_0", gR, rq, logits, T, E, K)
        qmm.qmm_route(logits, ids, weights)
        qmm.qmm_experts_glu(wtype, gg, gu, xq, ids, h, scratch, n)
        qmm.qmm_experts_sum(wtype, gd, h, ids, weights, out, scratch, n, residual=y)

    layer()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer()
    for t in (y, hn, logits, weights, h, out):
        t.fill_(float("nan"))
    graph.replay()
    sy, sh, sq = plain.add_norm(act, x, r, w, plain.EPS)
    assert np.array_equal(host(y), sy) and np.array_equal(host(hn), sh) and np.array_equal(host(xq), sq.reshape(T, -1))
    lg = host(logits)
    want = oracle.dequantize("q8_0", oracle.quantize("q8_0", sh), K) @ oracle.dequantize("q8_0", R, K).T
    assert (np.abs(lg - want) <= 1e-5 * np.linalg.norm(want, axis=-1, keepdims=True)).all()
    wi, ww = plain.route(lg, None, k)
    assert np.array_equal(host(ids), wi) and (np.abs(host(weights) - ww) <= 2.0 ** -24 * (2 * 90 + 2 * 36 + 16) * ww).all()
    wh, off = plain.glu(wtype, Wg, Wu, sq.reshape(T, -1), wi, "silu", K)
    assert (np.abs(host(h) - wh) <= off).all()
    wo, off = plain.summed(wtype, Wd, host(h), wi, host(weights), sy, N)
    assert (np.abs(host(out) - wo) <= off).all()
