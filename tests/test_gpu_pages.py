"""The paged cache on the GPU: rows stored bit for bit, read back exactly, and the attention over them within the bound
derived in pages_plain.attend; padding rows, pages without a place, far offsets, streams and captured graphs."""
import numpy as np
import pytest

import oracle
import pages_plain as plain
import workloads

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


def on_gpu(c):
    """(KvPages, k pool, v pool, table) of a host cache."""
    k, v, table = dev(c.k), dev(c.v), dev(c.table)
    return qmm.KvPages(c.typ, k, v, table, c.page, c.Hkv, c.hd), k, v, table


def scratch_for(Hq, c):
    n = qmm.qmm_kv_attend_scratch_bytes(Hq, c.Hkv, c.hd)
    return torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda"), n


def tokens(rng, seqs, most, T, pad):
    """Distinct places for T tokens; `pad` of them padding, anywhere in the list."""
    all_places = [(s, p) for s in range(seqs) for p in range(most)]
    pick = rng.permutation(len(all_places))[:T]
    seq = np.array([all_places[i][0] for i in pick], dtype=np.int32)
    pos = np.array([all_places[i][1] for i in pick], dtype=np.int32)
    pos[rng.permutation(T)[:pad]] = -1
    return seq, pos


STORE = [("q8", 1, 16, 16, 1, 0, 0, None), ("q8", 8, 128, 16, 40, 3, 32, "half"), ("q8", 2, 64, 8, 17, 1, 14, "interleaved"),
         ("q8", 3, 48, 1, 20, 2, 0, "half"), ("f16", 5, 80, 32, 33, 4, 20, "interleaved"), ("f16", 4, 128, 64, 30, 0, 0, None),
         ("q8", 2, 256, 128, 9, 1, 4, "half"), ("f16", 1, 256, 2, 9, 1, 6, "half"), ("q8", 4, 80, 16, 21, 2, 8, "half20"),
         ("f16", 3, 96, 4, 12, 0, 3, "half20"), ("q8", 40, 64, 16, 3, 0, 160, "half"), ("f16", 2, 192, 16, 5, 1, 2, "half")]


@pytest.mark.parametrize("typ,Hkv,hd,page,T,pad,Hq,layout", STORE)
def test_store_and_load(typ, Hkv, hd, page, T, pad, Hq, layout):
    rng = np.random.default_rng(hd * 31 + T)
    seqs, most = 3, max(20, page + 3)
    c = plain.Cache(typ, Hkv, hd, page, seqs, most, seed=T, fill=0xA5)
    pages, k, v, _ = on_gpu(c)
    seq, pos = tokens(rng, seqs, most, T, pad)
    kx, vx = (rng.standard_normal((T, Hkv, hd)).astype(np.float32) for _ in range(2))
    vx[0] = 0.0  # an all-zero row
    q = rng.standard_normal((T, Hq, hd)).astype(np.float32) if Hq else None
    rope, kr = None, kx
    if layout:
        n_rot = 20 if layout == "half20" else hd
        layout = "half" if layout == "half20" else layout
        table = plain.turns(plain.freqs(n_rot))
        rope = qmm.RopeSpec(dev(table), layout)
        kr = plain.rotate(kx, pos, table, layout)[0].astype(np.float32)
    q_out = torch.full((T, Hq, hd), 7.0, device="cuda") if Hq else None
    qmm.qmm_kv_store(pages, dev(kx), dev(vx), dev(pos), seq=dev(seq), rope=rope, q=dev(q) if Hq else None, q_out=q_out)
    for t in range(T):
        if pos[t] >= 0:
            c.put(c.k, seq[t], pos[t], kr[t])
            c.put(c.v, seq[t], pos[t], vx[t])
    # every byte of both pools: rows, scales, and what no token names left as it was
    assert np.array_equal(host(k), c.k) and np.array_equal(host(v), c.v)
    if Hq:
        y = torch.empty(T, Hq, hd, device="cuda")
        qmm.qmm_rope(rope, dev(q), y, dev(pos))
        want = host(y)
        want[pos < 0] = 7.0
        assert np.array_equal(host(q_out).view(np.int32), want.view(np.int32))
    ko, vo = (torch.full((T, Hkv, hd), 5.0, device="cuda") for _ in range(2))
    qmm.qmm_kv_load(pages, dev(pos), ko, vo, seq=dev(seq))
    want = np.full((2, T, Hkv, hd), 5.0, dtype=np.float32)
    for t in range(T):
        if pos[t] >= 0:
            want[0, t], want[1, t] = c.get(c.k, seq[t], pos[t]), c.get(c.v, seq[t], pos[t])
    assert np.array_equal(host(ko), want[0]) and np.array_equal(host(vo), want[1])
    only = torch.full((T, Hkv, hd), 5.0, device="cuda")
    qmm.qmm_kv_load(pages, dev(pos), None, only, seq=dev(seq))
    assert np.array_equal(host(only), want[1])
    only.fill_(5.0)
    qmm.qmm_kv_load(pages, dev(pos), only, None, seq=dev(seq))
    assert np.array_equal(host(only), want[0])


def test_rows_are_those_of_kv_quantize():
    rng = np.random.default_rng(5)
    Hkv, hd, page, T = 4, 64, 16, 11
    c = plain.Cache("q8", Hkv, hd, page, T, page, seed=1, fill=0)
    pages, k, _, _ = on_gpu(c)
    x = workloads.activations_f32(T * Hkv, hd, seed=9).reshape(T, Hkv, hd)
    qmm.qmm_kv_store(pages, dev(x), dev(x), dev(np.full(T, 3, np.int32)))  # no seq: token t in sequence t
    rows = torch.empty(T * Hkv * qmm.qmm_kv_row_bytes(hd), dtype=torch.uint8, device="cuda")
    qmm.qmm_kv_quantize(dev(x), rows, T * Hkv, hd)
    rows, pool = host(rows).reshape(T, Hkv, 4 + hd), host(k)
    for t in range(T):
        p, o = c.place(t, 3)
        for h in range(Hkv):
            slot = h * page + o
            assert np.array_equal(pool[p, slot * hd: (slot + 1) * hd], rows[t, h, 4:])
            at = Hkv * page * hd + 4 * slot
            assert np.array_equal(pool[p, at: at + 4], rows[t, h, :4])


def test_special_rows_are_those_of_kv_quantize():
    """Rows of subnormal values (127 / amax overflows), infinities, NaN and ties: the same codes and scales."""
    Hkv, hd, page, T = 2, 32, 16, 6
    c = plain.Cache("q8", Hkv, hd, page, T, page, seed=1, fill=0)
    pages, k, v, _ = on_gpu(c)
    x = workloads.activations_f32(T * Hkv, hd, seed=19).reshape(T, Hkv, hd)
    x[0] *= np.float32(1e-41)
    x[1, 0, 3], x[1, 1, 5] = np.inf, -np.inf
    x[2, 0, 4] = np.nan
    x[3, 0], x[3, 1] = np.float32(3e38), 0.0
    x[4, 0, 0], x[4, 0, 1], x[4, 0, 2], x[4, 0, 3:] = 127.0, 2.5, -3.5, 0.5
    rows = torch.empty(T * Hkv * qmm.qmm_kv_row_bytes(hd), dtype=torch.uint8, device="cuda")
    qmm.qmm_kv_quantize(dev(x), rows, T * Hkv, hd)
    for layout in (None, "half", "interleaved"):  # at position 0 a rotation copies
        pos = np.zeros(T, np.int32)
        rope = qmm.RopeSpec(dev(plain.turns(plain.freqs(hd))), layout) if layout else None
        qmm.qmm_kv_store(pages, dev(x), dev(x), dev(pos), rope=rope)
        want = host(rows).reshape(T, Hkv, 4 + hd)
        # an infinity or NaN, and what overflows, reaches its pair through the rotation's products: keys 1 .. 3 then
        # hold other rows
        for which, pool in (("k", host(k)), ("v", host(v))):
            for t in range(T):
                if layout and which == "k" and t in (1, 2, 3):
                    continue
                p, o = c.place(t, 0)
                for h in range(Hkv):
                    at, sc = (h * page + o) * hd, Hkv * page * hd + 4 * (h * page + o)
                    assert np.array_equal(pool[p, at: at + hd], want[t, h, 4:]), (layout, which, t, h)
                    assert np.array_equal(pool[p, sc: sc + 4], want[t, h, :4]), (layout, which, t, h)


ATTEND = [  # type, Hq, Hkv, hd, page, lens, window
    ("q8", 1, 1, 16, 16, [1], 0), ("q8", 14, 2, 64, 16, [33], 0), ("q8", 32, 8, 128, 16, [1, 31, 32, 33, 0, -1, 129, 700], 0),
    ("q8", 8, 8, 128, 64, [257, 5], 0), ("q8", 3, 1, 48, 1, [40, 2, 300], 0), ("q8", 10, 5, 80, 8, [77, 513], 0),
    ("q8", 12, 1, 128, 32, [200, 65], 0), ("q8", 64, 1, 64, 16, [100, -1, 17], 0), ("q8", 6, 2, 256, 16, [150, 16, 15], 0),
    ("q8", 7, 1, 192, 128, [300, 128], 0), ("q8", 2, 2, 112, 4, [1000], 0), ("q8", 16, 2, 96, 512, [600, 3], 0),
    ("f16", 32, 8, 128, 16, [1, 15, 16, 17, 0, -1, 200], 0), ("f16", 4, 4, 256, 32, [300, 31], 0),
    ("f16", 14, 2, 64, 8, [65, 640], 0), ("f16", 5, 1, 80, 2, [90], 0), ("f16", 9, 1, 16, 16, [50, 1], 0),
    ("q8", 8, 2, 128, 16, [500, 3, 40, 41, 0], 1), ("q8", 8, 2, 128, 16, [500, 3, 40, 41, 0], 37),
    ("q8", 8, 2, 128, 16, [500, 3, 40, 41, 0], 4000), ("f16", 2, 2, 256, 32, [500, 3, 33], 100),
    ("q8", 4, 1, 64, 16, [2500], 0), ("f16", 8, 8, 64, 64, [2000, 1], 0), ("q8", 1, 1, 128, 16, [-1, 0], 0)]


@pytest.mark.parametrize("typ,Hq,Hkv,hd,page,lens,window", ATTEND)
def test_attend(typ, Hq, Hkv, hd, page, lens, window):
    rng = np.random.default_rng(hd * 7 + len(lens) + window)
    c = plain.Cache(typ, Hkv, hd, page, len(lens), max(max(lens), 1), seed=hd)
    for r, n in enumerate(lens):
        if n > 0:
            c.fill(r, n, rng)
            c.table[r, -(-n // page):] = 2 ** 30  # behind the last position: not read
    q = rng.standard_normal((len(lens), Hq, hd)).astype(np.float32)
    scale = hd ** -0.5
    want, wlse, bound, lbound = plain.attend(c, q, lens, range(len(lens)), scale, window)
    pages = on_gpu(c)[0]
    scratch, n = scratch_for(Hq, c)
    out, lse = torch.full(q.shape, 9.0, device="cuda"), torch.full(q.shape[:2], 9.0, device="cuda")
    qmm.qmm_kv_attend(pages, dev(q), dev(np.array(lens, np.int32)), out, scratch, n, scale, lse=lse, window=window)
    got, glse = host(out), host(lse)
    kept = np.array(lens) >= 0
    assert np.all(got[~kept] == 9.0) and np.all(glse[~kept] == 9.0)  # padding rows are left alone
    err = np.abs(got.astype(np.float64) - want)[kept]
    assert np.all(err <= bound[kept]), (np.max(err), np.max(err / np.maximum(bound[kept], 1e-300)))
    empty = np.array(lens) == 0
    assert np.all(got[empty] == 0) and np.all(np.isneginf(glse[empty]))
    some = np.array(lens) > 0
    assert np.all(np.abs(glse[some].astype(np.float64) - wlse[some]) <= lbound[some])
    again = torch.full(q.shape, 9.0, device="cuda")  # without lse, and bit for bit the same
    qmm.qmm_kv_attend(pages, dev(q), dev(np.array(lens, np.int32)), again, scratch, n, scale, window=window)
    assert np.array_equal(host(again).view(np.int32), got.view(np.int32))


def test_many_rows_and_shared_sequences():
    """More rows than a CTA has threads, several of them reading one sequence at lengths of their own."""
    rng = np.random.default_rng(12)
    Hq, Hkv, hd, page, seqs, R = 4, 2, 64, 16, 5, 300
    c = plain.Cache("q8", Hkv, hd, page, seqs, 90, seed=3)
    for s in range(seqs):
        c.fill(s, 90, rng)
    lens, seq = rng.integers(-1, 91, size=R).astype(np.int32), rng.integers(0, seqs, size=R).astype(np.int32)
    q = rng.standard_normal((R, Hq, hd)).astype(np.float32)
    want, _, bound, _ = plain.attend(c, q, lens, seq, 0.125)
    scratch, n = scratch_for(Hq, c)
    out = torch.zeros(q.shape, device="cuda")
    qmm.qmm_kv_attend(on_gpu(c)[0], dev(q), dev(lens), out, scratch, n, 0.125, seq=dev(seq))
    kept = lens >= 0
    err = np.abs(host(out).astype(np.float64) - want)[kept]
    assert np.all(err <= bound[kept])


@pytest.mark.parametrize("typ,Hq,Hkv,hd,page,lens,window", [
    ("q8", 40, 40, 64, 16, [1, 33, 0, -1, 40, 32, 7, 64, 5, 31, 2, 50, 17, 48, 3, 65], 0),
    ("q8", 120, 40, 128, 16, [700, 3, 0, 250, 64, 1, 300, 20, 9, 33, 128, 5, 77, 600, -1, 31, 450], 0),
    ("q8", 80, 40, 256, 8, [90, 1, 15, 16, 17, 60, 0, 33, 5, 40, 2, 80, 64, 100, 9, 3], 0),
    ("f16", 41, 41, 80, 32, [90, 1, 15, 16, 17, 60, 0, 33, 5, 40, 2, 80, 64, 100, 9, -1], 20),
    ("f16", 160, 40, 128, 1, [70, 1, 15, 16, 17, 60, 0, 33, 5, 40, 2, 80, 64, 100, 9, 3], 0),
    ("f16", 40, 40, 256, 16, [90, 1, 15, 16, 17, 60, 0, 33, 5, 40, 2, 80, 64, 100, 9, 3], 0),
    ("q8", 50, 1, 48, 16, [20 + i % 40 for i in range(90)], 0)])
def test_many_units(typ, Hq, Hkv, hd, page, lens, window):
    """More units (KV heads, or eights of their query heads, of a row) than get a CTA each: a warp takes them alone."""
    test_attend(typ, Hq, Hkv, hd, page, lens, window)


@pytest.mark.parametrize("typ", ["q8", "f16"])
def test_extreme_values(typ):
    """Very large and very small rows, zero rows, a zero query, a query whose scores dwarf the others."""
    rng = np.random.default_rng(21)
    Hq, Hkv, hd, page, n = 4, 1, 64, 16, 70
    c = plain.Cache(typ, Hkv, hd, page, 1, n, seed=5)
    for p in range(n):
        big = 1e4 if p % 7 == 0 else (1e-6 if p % 5 == 0 else 1.0)
        k = rng.standard_normal((Hkv, hd)).astype(np.float32)
        c.put(c.k, 0, p, k * 0 if p % 11 == 0 else k)
        c.put(c.v, 0, p, k * 0 if p % 13 == 0 else (rng.standard_normal((Hkv, hd)) * big).astype(np.float32))
    q = rng.standard_normal((1, Hq, hd)).astype(np.float32)
    q[0, 1], q[0, 2], q[0, 3] = 0.0, q[0, 2] * 30, q[0, 3] * 1e-20
    want, wlse, bound, lbound = plain.attend(c, q, [n], [0], 0.125)
    scratch, m = scratch_for(Hq, c)
    out, lse = torch.empty(q.shape, device="cuda"), torch.empty(1, Hq, device="cuda")
    qmm.qmm_kv_attend(on_gpu(c)[0], dev(q), dev(np.array([n], np.int32)), out, scratch, m, 0.125, lse=lse)
    err = np.abs(host(out).astype(np.float64) - want)
    assert np.all(err <= bound), np.max(err / bound)
    assert np.all(np.abs(host(lse) - wlse) <= lbound)


@pytest.mark.parametrize("typ,Hq,Hkv,hd,window,R", [("q8", 16, 2, 64, 0, 5000), ("f16", 3, 3, 32, 19, 700), ("q8", 9, 1, 128, 7, 129)])
def test_thousands_of_rows(typ, Hq, Hkv, hd, window, R):
    """Rows of every length, empty and padding ones among them, with one set of queries: a result per sequence and length."""
    rng = np.random.default_rng(R)
    c = plain.Cache(typ, Hkv, hd, 8, 3, 44, seed=3)
    for s in range(3):
        c.fill(s, 44, rng)
    lens, seq = rng.integers(-1, 45, size=R).astype(np.int32), rng.integers(0, 3, size=R).astype(np.int32)
    lens[R // 2: R // 2 + R // 7] = 0  # long runs of rows without work
    lens[-R // 9:] = -1
    q = np.repeat(rng.standard_normal((1, Hq, hd)).astype(np.float32), 135, axis=0)
    at, of = np.tile(np.arange(45), 3), np.repeat(np.arange(3), 45)
    want, wlse, bound, lbound = plain.attend(c, q, at, of, 0.2, window)
    scratch, n = scratch_for(Hq, c)
    out, lse = torch.full((R, Hq, hd), 9.0, device="cuda"), torch.full((R, Hq), 9.0, device="cuda")
    qs = dev(q[:1]).expand(R, Hq, hd).contiguous()
    qmm.qmm_kv_attend(on_gpu(c)[0], qs, dev(lens), out, scratch, n, 0.2, lse=lse, seq=dev(seq), window=window)
    got, glse = host(out), host(lse)
    kept, some, which = lens >= 0, lens > 0, seq * 45 + lens
    assert np.all(got[~kept] == 9.0) and np.all(glse[~kept] == 9.0)
    assert np.all(np.abs(got[kept].astype(np.float64) - want[which[kept]]) <= bound[which[kept]])
    assert np.all(np.abs(glse[some].astype(np.float64) - wlse[which[some]]) <= lbound[which[some]])
    assert np.all(np.isneginf(glse[lens == 0]))


@pytest.mark.parametrize("scale", [0.0, -0.3, 3.0])
def test_scales(scale):
    """No scale (the mean of the values), a negative one (the softmax prefers the smallest products), a large one."""
    rng = np.random.default_rng(23)
    c = plain.Cache("q8", 2, 64, 16, 2, 90, seed=5)
    c.fill(0, 90, rng, loud=False)
    c.fill(1, 33, rng, loud=False)
    q = rng.standard_normal((2, 6, 64)).astype(np.float32)
    want, wlse, bound, lbound = plain.attend(c, q, [90, 33], [0, 1], scale)
    scratch, m = scratch_for(6, c)
    out, lse = torch.empty(q.shape, device="cuda"), torch.empty(2, 6, device="cuda")
    qmm.qmm_kv_attend(on_gpu(c)[0], dev(q), dev(np.array([90, 33], np.int32)), out, scratch, m, scale, lse=lse)
    assert np.all(np.abs(host(out) - want) <= bound)
    assert np.all(np.abs(host(lse) - wlse) <= lbound)


def test_store_of_a_fused_projection_rotates_in_place():
    """Queries, keys and values as columns of one row buffer, the queries rotated where they stand."""
    rng = np.random.default_rng(24)
    T, Hq, Hkv, hd = 21, 6, 2, 96
    c = plain.Cache("q8", Hkv, hd, 16, 1, 64, seed=6, fill=0)
    pages, k, v, _ = on_gpu(c)
    buf = rng.standard_normal((T, Hq + 2 * Hkv, hd)).astype(np.float32)
    t = dev(buf)
    pos, seq = np.arange(5, 5 + T, dtype=np.int32), np.zeros(T, np.int32)
    table = plain.turns(plain.freqs(64))
    rope = qmm.RopeSpec(dev(table))
    q = t[:, :Hq]
    qmm.qmm_kv_store(pages, t[:, Hq: Hq + Hkv], t[:, Hq + Hkv:], dev(pos), seq=dev(seq), rope=rope, q=q, q_out=q)
    kr = plain.rotate(buf[:, Hq: Hq + Hkv], pos, table)[0].astype(np.float32)
    for i in range(T):
        c.put(c.k, 0, pos[i], kr[i])
        c.put(c.v, 0, pos[i], buf[i, Hq + Hkv:])
    assert np.array_equal(host(k), c.k) and np.array_equal(host(v), c.v)
    want = torch.empty(T, Hq, hd, device="cuda")
    qmm.qmm_rope(rope, dev(buf[:, :Hq]), want, dev(pos))
    got = host(t)
    assert np.array_equal(got[:, :Hq].copy().view(np.int32), host(want).view(np.int32))
    assert np.array_equal(got[:, Hq:], buf[:, Hq:])


def test_two_calls_at_once():
    """Calls on two streams, each with its own scratch, over one cache: the results of the same calls one by one."""
    rng = np.random.default_rng(25)
    c = plain.Cache("q8", 2, 128, 16, 3, 600, seed=7)
    for s, n in enumerate((600, 31, 290)):
        c.fill(s, n, rng)
    pages = on_gpu(c)[0]
    lens = dev(np.array([600, 31, 290], np.int32))
    qs = [dev(rng.standard_normal((3, 8, 128)).astype(np.float32)) for _ in range(2)]
    want = [torch.empty(3, 8, 128, device="cuda") for _ in range(2)]
    got = [[torch.empty(3, 8, 128, device="cuda") for _ in range(10)] for _ in range(2)]
    scratch = [scratch_for(8, c) for _ in range(2)]
    for q, w in zip(qs, want):
        qmm.qmm_kv_attend(pages, q, lens, w, *scratch[0], 0.1)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for i in range(10):
        for j, s in enumerate(streams):
            qmm.qmm_kv_attend(pages, qs[j], lens, got[j][i], *scratch[j], 0.1, stream=s)
    torch.cuda.synchronize()
    for j in range(2):
        for i in range(10):
            assert torch.equal(got[j][i].view(torch.int32), want[j].view(torch.int32))


def test_nan_query_stays_with_its_head():
    rng = np.random.default_rng(22)
    c = plain.Cache("q8", 1, 64, 16, 1, 50, seed=5)
    c.fill(0, 50, rng)
    q = rng.standard_normal((1, 8, 64)).astype(np.float32)
    want, _, bound, _ = plain.attend(c, q, [50], [0], 0.125)
    q[0, 3, 5] = np.nan
    scratch, m = scratch_for(8, c)
    out = torch.empty(q.shape, device="cuda")
    qmm.qmm_kv_attend(on_gpu(c)[0], dev(q), dev(np.array([50], np.int32)), out, scratch, m, 0.125)
    got = host(out)
    assert np.all(np.isnan(got[0, 3]))
    rest = [h for h in range(8) if h != 3]
    assert np.all(np.abs(got[0, rest] - want[0, rest]) <= bound[0, rest])


def test_offsets_beyond_32_bits():
    """Pages 64 MB apart in a 6.4 GB pool, keys and values in one buffer."""
    rng = np.random.default_rng(30)
    Hq, Hkv, hd, page, n = 4, 2, 64, 16, 90 * 16
    pages_n, stride = 100, 64 << 20
    c = plain.Cache("q8", Hkv, hd, page, 1, n, seed=2)
    c.table[0] = rng.permutation(pages_n)[: c.max_pages]
    c.k = np.zeros((pages_n, c.bytes), np.uint8)
    c.v = c.k.copy()
    c.fill(0, n, rng)
    pool = torch.empty(pages_n * stride, dtype=torch.uint8, device="cuda").view(pages_n, stride)
    k, v = pool[:, : c.bytes], pool[:, stride // 2: stride // 2 + c.bytes]
    k.copy_(dev(c.k))
    v.copy_(dev(c.v))
    pages = qmm.KvPages("q8", k, v, dev(c.table), page, Hkv, hd)
    q = rng.standard_normal((1, Hq, hd)).astype(np.float32)
    want, _, bound, _ = plain.attend(c, q, [n], [0], 0.125)
    scratch, m = scratch_for(Hq, c)
    out = torch.empty(q.shape, device="cuda")
    qmm.qmm_kv_attend(pages, dev(q), dev(np.array([n], np.int32)), out, scratch, m, 0.125)
    assert np.all(np.abs(host(out) - want) <= bound)
    x = rng.standard_normal((3, Hkv, hd)).astype(np.float32)
    pos, seq = np.array([5, 700, 1439], np.int32), np.zeros(3, np.int32)
    qmm.qmm_kv_store(pages, dev(x), dev(-x), dev(pos), seq=dev(seq))
    ko, vo = torch.empty(x.shape, device="cuda"), torch.empty(x.shape, device="cuda")
    qmm.qmm_kv_load(pages, dev(pos), ko, vo, seq=dev(seq))
    codes, d = plain.q8(x)
    assert np.array_equal(host(ko), codes.astype(np.float32) * d[..., None])
    assert np.array_equal(host(vo), -codes.astype(np.float32) * d[..., None])


def test_positions_without_a_place():
    """A page id outside the pool, a position behind the table, a sequence outside it: reported, not stored, zeros when
    read, absent in the attention; everything else as ever."""
    rng = np.random.default_rng(40)
    Hq, Hkv, hd, page, n = 4, 2, 64, 16, 60
    c = plain.Cache("q8", Hkv, hd, page, 2, 64, seed=2)
    c.fill(0, 64, rng)
    c.fill(1, 64, rng)
    good = c.table.copy()
    c.table[0, 1] = c.pages  # positions 16 .. 31
    pages, k, v, _ = on_gpu(c)
    x = rng.standard_normal((5, Hkv, hd)).astype(np.float32)
    pos, seq = np.array([20, 64, 3, 2, 2 ** 31 - 1], np.int32), np.array([0, 1, 2, -1, 0], np.int32)
    qmm.qmm_kv_store(pages, dev(x), dev(x), dev(pos), seq=dev(seq))
    assert qmm.qmm_device_status(clear=True) == 2
    assert np.array_equal(host(k), c.k) and np.array_equal(host(v), c.v)
    ko, vo = torch.full(x.shape, 3.0, device="cuda"), torch.full(x.shape, 3.0, device="cuda")
    qmm.qmm_kv_load(pages, dev(pos), ko, vo, seq=dev(seq))
    assert qmm.qmm_device_status(clear=True) == 2
    assert np.all(host(ko) == 0) and np.all(host(vo) == 0)
    q = rng.standard_normal((4, Hq, hd)).astype(np.float32)
    lens, seq = np.array([n, 64, 5, 1000], np.int32), np.array([0, 1, 7, 1], np.int32)
    scratch, m = scratch_for(Hq, c)
    out = torch.full(q.shape, 3.0, device="cuda")
    qmm.qmm_kv_attend(pages, dev(q), dev(lens), out, scratch, m, 0.125, seq=dev(seq))
    assert qmm.qmm_device_status(clear=True) == 2
    got = host(out)
    c.table = good
    kk = np.stack([c.get(c.k, 0, p) for p in range(n) if not 16 <= p < 32])
    vv = np.stack([c.get(c.v, 0, p) for p in range(n) if not 16 <= p < 32])
    for h in range(Hq):  # row 0: as if the 16 positions were not there
        w = np.exp(0.125 * (kk[:, h // 2] @ q[0, h].astype(np.float64)))
        assert np.allclose(got[0, h], (w / w.sum()) @ vv[:, h // 2], rtol=0, atol=1e-5)
    want, _, bound, _ = plain.attend(c, q[[1, 3]], [64, 64], [1, 1], 0.125)  # row 3: cut to the table's room
    assert np.all(np.abs(got[[1, 3]] - want) <= bound)
    assert np.all(got[2] == 0)


def test_one_page_of_a_strided_row():
    """Queries inside a fused projection's rows, the output inside wider rows: what lies between stays as it was."""
    rng = np.random.default_rng(41)
    R, Hq, Hkv, hd = 3, 6, 2, 64
    c = plain.Cache("q8", Hkv, hd, 64, R, 64, seed=2)
    lens = [64, 1, 17]
    for r, n in enumerate(lens):
        c.fill(r, n, rng)
    qkv = rng.standard_normal((R, Hq + 2 * Hkv, hd)).astype(np.float32)
    wide = torch.full((R, Hq + 3, hd), 2.0, device="cuda")
    scratch, m = scratch_for(Hq, c)
    qmm.qmm_kv_attend(on_gpu(c)[0], dev(qkv)[:, :Hq], dev(np.array(lens, np.int32)), wide[:, 1: 1 + Hq], scratch, m, 0.125)
    got = host(wide)
    want, _, bound, _ = plain.attend(c, qkv[:, :Hq], lens, range(R), 0.125)
    assert np.all(np.abs(got[:, 1: 1 + Hq] - want) <= bound)
    assert np.all(got[:, 0] == 2.0) and np.all(got[:, 1 + Hq:] == 2.0)


def test_decode_step_captured_and_replayed():
    """One layer's attention as a decode step runs it -- the projections of a Q8_0 layer, keys and queries rotated and
    stored, the attention, the output projection -- captured once and replayed while the sequences grow: each step
    against the same steps in 64 bits from the projections' outputs.  A second graph with its own scratch replays in
    between on another stream."""
    rng = np.random.default_rng(50)
    S, Hq, Hkv, hd, K, page, steps = 3, 4, 2, 64, 256, 16, 20
    Ns = [Hq * hd, Hkv * hd, Hkv * hd]
    Wh = [oracle.quantize("q8_0", workloads.weights_f32(n, K, seed=60 + i)) for i, n in enumerate(Ns)]
    Ws = [dev(w) for w in Wh]
    Wo = dev(oracle.quantize("q8_0", workloads.weights_f32(K, Hq * hd, seed=70)))
    table = plain.turns(plain.freqs(hd))
    rope = qmm.RopeSpec(dev(table))

    class Step:
        def __init__(self, seed):
            self.c = plain.Cache("q8", Hkv, hd, page, S, 64, seed=seed)
            self.pages = on_gpu(self.c)[0]
            self.x = torch.zeros(S, K, device="cuda")
            self.pos, self.lens = (torch.zeros(S, dtype=torch.int32, device="cuda") for _ in range(2))
            self.q = torch.empty(S, Hq, hd, device="cuda")
            self.k, self.v = (torch.empty(S, Hkv, hd, device="cuda") for _ in range(2))
            self.o, self.y = torch.empty(S, Hq, hd, device="cuda"), torch.empty(S, K, device="cuda")
            self.act = torch.empty(S * qmm.qmm_row_bytes("q8_0", max(K, Hq * hd)), dtype=torch.uint8, device="cuda")
            self.scratch, self.bytes = scratch_for(Hq, self.c)

        def run(self, st=None):
            n = self.act.numel()
            qmm.qmm_linear_group("q8_0", Ws, Ns, self.x, self.act, n, [self.q, self.k, self.v], S, K, stream=st)
            self.raw = (self.q, self.k, self.v)
            qmm.qmm_kv_store(self.pages, self.k, self.v, self.pos, rope=rope, q=self.q, q_out=self.q, stream=st)
            qmm.qmm_kv_attend(self.pages, self.q, self.lens, self.o, self.scratch, self.bytes, hd ** -0.5, stream=st)
            qmm.linear("q8_0", Wo, self.o, self.act, n, self.y, S, K, Hq * hd, stream=st)

    a, b = Step(1), Step(2)
    streams, graphs = [torch.cuda.Stream(), torch.cuda.Stream()], []
    torch.cuda.synchronize()
    for step, s in zip((a, b), streams):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            step.run()
        graphs.append(g)
    lens = np.array([0, 7, 30], np.int32)
    torch.cuda.synchronize()
    for step in (a, b):
        for s in range(S):
            step.c.fill(s, lens[s], rng)
        step.pages.tensors[0].copy_(dev(step.c.k))
        step.pages.tensors[1].copy_(dev(step.c.v))
    for i in range(steps):
        x = rng.standard_normal((S, K)).astype(np.float32)
        torch.cuda.synchronize()
        for step in (a, b):
            step.x.copy_(dev(x))
            step.pos.copy_(dev(lens))
            step.lens.copy_(dev(lens + 1))
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        assert qmm.qmm_device_status(clear=True) == 0
        X = oracle.quantize("q8_0", x)
        for step in (a, b):
            proj = [torch.empty(S, n, device="cuda") for n in Ns]
            qmm.qmm_linear_group("q8_0", Ws, Ns, step.x, step.act, step.act.numel(), proj, S, K)
            q, k, v = [host(p).reshape(S, -1, hd) for p in proj]
            assert np.allclose(q.reshape(S, -1), oracle.matmul("q8_0", Wh[0], X, S, Ns[0], K), rtol=1e-4, atol=1e-4)
            kr = plain.rotate(k, lens, table)[0].astype(np.float32)
            qr = plain.rotate(q, lens, table)[0].astype(np.float32)
            for s in range(S):
                step.c.put(step.c.k, s, lens[s], kr[s])
                step.c.put(step.c.v, s, lens[s], v[s])
            want, _, bound, _ = plain.attend(step.c, qr, lens + 1, range(S), hd ** -0.5)
            assert np.all(np.abs(host(step.o) - want) <= bound), i
        lens = lens + 1
    assert np.array_equal(host(a.pages.tensors[0]), a.c.k) and np.array_equal(host(a.pages.tensors[1]), a.c.v)
    y = torch.empty(S, K, device="cuda")
    qmm.linear("q8_0", Wo, a.o, a.act, a.act.numel(), y, S, K, Hq * hd)
    assert np.array_equal(host(y), host(a.y))


def test_binding_refuses():
    c = plain.Cache("q8", 2, 64, 16, 2, 32)
    pages, k, v, table = on_gpu(c)
    for bad in (("q8", k.cpu(), v, table, 16, 2, 64), ("q8", k, v, table.long(), 16, 2, 64),
                ("q8", k, v, table, 16, 4, 64), ("q8", k, v, table, 12, 2, 64), ("q8", k, v[:-1], table, 16, 2, 64),
                ("f16", k, v, table, 16, 2, 64), ("q8", k, v, table.t(), 16, 2, 64)):
        with pytest.raises(ValueError):
            qmm.KvPages(*bad)
    x, pos = torch.zeros(2, 2, 64, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda")
    for bad in ((x[:, :1], x, pos), (x, x.half(), pos), (x, x, pos.cpu()), (x, x, pos[:1])):
        with pytest.raises(ValueError):
            qmm.qmm_kv_store(pages, *bad)
    with pytest.raises(ValueError):
        qmm.qmm_kv_load(pages, pos, torch.zeros(2, 3, 64, device="cuda"), x)
    q = torch.zeros(2, 4, 64, device="cuda")
    s, n = scratch_for(4, c)
    with pytest.raises(ValueError):
        qmm.qmm_kv_attend(pages, q, pos, x, s, n, 0.1)
    with pytest.raises(ValueError):
        qmm.qmm_kv_attend(pages, q, pos, q, s, n, 0.1, lse=torch.zeros(2, 3, device="cuda"))
    with pytest.raises(ValueError):
        qmm.qmm_kv_attend(pages, q, pos, torch.zeros_like(q), s[:-16], n, 0.1)
    with pytest.raises(ValueError):
        qmm.qmm_kv_store(pages, x, x, pos, q=q)
    pages.device += 1
    with pytest.raises(ValueError):
        qmm.qmm_kv_attend(pages, q, pos, torch.zeros_like(q), s, n, 0.1)
    pages.device -= 1
    with pytest.raises(qmm.QmmError):
        qmm.qmm_kv_attend(pages, q, pos, torch.zeros_like(q), s, n - 1, 0.1)
