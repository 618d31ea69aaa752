"""The rotary and paged-cache kernels where every loop of theirs goes round: rings that wrap, references that rise from tile
to tile, joins of more than 64 parts and of several pieces per CTA, several blocks of tokens per CTA, several tokens side by
side with a remainder."""
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


def same_bits(a, b):
    return torch.equal(a.contiguous().view(torch.int32), b.contiguous().view(torch.int32))


class Cache:
    """A cache on the GPU for tests of its own: pools, a shuffled table, rows written and read by whole sequences."""

    def __init__(self, typ, Hkv, hd, page, seqs, most, seed=0, fill=0xFF):
        self.gen = torch.Generator(device="cuda")
        self.gen.manual_seed(seed)
        self.typ, self.Hkv, self.hd, self.page = typ, Hkv, hd, page
        self.max_pages = -(-most // page)
        total = seqs * self.max_pages + 3
        self.bytes = qmm.qmm_kv_page_bytes(typ, Hkv, page, hd)
        stride = -(-self.bytes // 16) * 16
        self.k = torch.full((total, stride), fill, dtype=torch.uint8, device="cuda")
        self.v = self.k.clone()
        self.table = torch.randperm(total, device="cuda", generator=self.gen)[: seqs * self.max_pages].to(torch.int32)
        self.table = self.table.view(seqs, self.max_pages).contiguous()
        self.pages = qmm.KvPages(typ, self.k, self.v, self.table, page, Hkv, hd)

    def planes(self, pool):
        n, shape = pool.shape[0], (self.Hkv, self.page, self.hd)
        if self.typ == "f16":
            return pool[:, : 2 * self.Hkv * self.page * self.hd].view(torch.float16).unflatten(1, shape), None
        cut = self.Hkv * self.page * self.hd
        assert pool.shape == (n, pool.shape[1])
        return (pool[:, :cut].view(torch.int8).unflatten(1, shape),
                pool[:, cut: cut + 4 * self.Hkv * self.page].view(torch.float32).unflatten(1, shape[:2]))

    def put(self, pool, seq, first, codes, d=None):
        """codes [n][Hkv][hd] (int8, or what f16 rows hold) and scales d [n][Hkv] into positions first .. of sequence seq."""
        p = torch.arange(first, first + codes.shape[0], device="cuda")
        at, off = self.table[seq, p // self.page].long(), p % self.page
        rows, scales = self.planes(pool)
        rows[at, :, off] = codes.to(rows.dtype)
        if scales is not None:
            scales[at, :, off] = torch.ones_like(codes[..., 0], dtype=torch.float32) if d is None else d

    def get(self, pool, seq, pos):
        """f64 rows [n][Hkv][hd] at (seq[i], pos[i]) (a number or a tensor each)."""
        rows, scales = self.planes(pool)
        pos = pos.long()
        at, off = self.table[seq, pos // self.page].long(), pos % self.page
        x = rows[at, :, off].double()
        return x if scales is None else x * scales[at, :, off].double()[..., None]

    def attend(self, q, lens, scale, window=0, seq=None):
        R, Hq = q.shape[:2]
        n = qmm.qmm_kv_attend_scratch_bytes(Hq, self.Hkv, self.hd)
        scratch = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")
        out, lse = torch.full(q.shape, 9.0, device="cuda"), torch.full((R, Hq), 9.0, device="cuda")
        lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
        qmm.qmm_kv_attend(self.pages, q, lens, out, scratch, n, scale, lse=lse, seq=seq, window=window)
        return out, lse


WHOLE = [  # type, Hq, Hkv, hd, page, lens, window
    ("q8", 8, 1, 128, 16, [40001], 0),              # CTAs, some 300 parts of one unit
    ("q8", 8, 2, 128, 64, [200003], 0),             # CTAs whose warps take ten tiles each, 152 parts a unit
    ("q8", 8, 2, 128, 64, [200003], 123457),
    ("q8", 64, 8, 128, 16, [2500], 0),              # 20 parts a unit: several pieces per joining CTA, two batches
    ("q8", 32, 4, 256, 16, [3001, 0, 700], 0),
    ("q8", 14, 2, 64, 16, [150001, 17], 0),
    ("q8", 8, 1, 96, 32, [9000, 60011, -1, 33], 0),  # units of under and over 64 parts side by side
    ("f16", 8, 1, 256, 32, [100003], 0), ("f16", 16, 2, 128, 8, [30011, 5000], 29000), ("f16", 3, 1, 80, 16, [20011], 0),
    ("q8", 64, 8, 64, 16, [137 * i for i in range(40)], 0),     # single warps
    ("q8", 32, 16, 128, 16, [5000, 1, 0, 40000, 300, -1, 2222, 9, 31, 32, 33, 64], 0),
    ("f16", 40, 40, 256, 16, [3000, 0, 1, 900, 17, 2000], 1000)]


@pytest.mark.parametrize("typ,Hq,Hkv,hd,page,lens,window", WHOLE)
def test_every_position_counts_once(typ, Hq, Hkv, hd, page, lens, window):
    """A zero query and whole values up to 20 of scale 1: all weights are 1, every product and sum is exact (below 2^24), so
    the result is the whole sum times f32(1 / n), two roundings; and the log's is n."""
    c = Cache(typ, Hkv, hd, page, len(lens), max(lens), seed=hd)
    sums = torch.zeros(len(lens), Hkv, hd, dtype=torch.float64, device="cuda")
    seen = [min(n, window) if window else n for n in lens]
    for r, n in enumerate(lens):
        if n > 0:
            c.put(c.k, r, 0, torch.randint(-127, 128, (n, Hkv, hd), device="cuda", generator=c.gen))
            x = torch.randint(-20, 21, (n, Hkv, hd), device="cuda", generator=c.gen)
            c.put(c.v, r, 0, x)
            sums[r] = x[n - seen[r]:].sum(0).double()
    out, lse = c.attend(torch.zeros(len(lens), Hq, hd, device="cuda"), lens, 0.125, window)
    for r, n in enumerate(seen):
        if n <= 0:
            assert torch.all(out[r] == (9.0 if n < 0 else 0.0)) and torch.all(lse[r] == (9.0 if n < 0 else -float("inf")))
            continue
        want = (sums[r] / n).repeat_interleave(Hq // Hkv, 0)
        err = (out[r].double() - want).abs()
        assert torch.all(err <= 3 * 2.0 ** -24 * want.abs()), (r, err.max().item())
        assert torch.all((lse[r].double() - np.log(n)).abs() <= 4 * 2.0 ** -24 * np.log(max(n, 2)))


@pytest.mark.parametrize("typ,Hq,Hkv,hd,page,lens", [
    ("q8", 8, 1, 128, 16, [40000]), ("q8", 8, 1, 128, 16, [3000]), ("q8", 16, 2, 128, 16, [200000]),
    ("f16", 8, 1, 256, 32, [60000]), ("q8", 64, 8, 128, 16, [2500]), ("q8", 40, 40, 64, 16, [5000, 700, 2500, 33, 9000])])
@pytest.mark.parametrize("rise", [8.0, 300.0])
def test_a_rising_maximum(typ, Hq, Hkv, hd, page, lens, rise):
    """Scores that rise along the row, a little or by e^300, so that the running reference is raised again and again.  The
    queries have one value only, so a score's terms are |t| in all; per position the kernel is off by delta = |t| (2^-22 +
    (hd / 16) 2^-23 + 5 * 2^-24) and the exponential's 2^-22, in the numerator and in the sum; the split, the product with
    the scale and the matrix steps take 3 * 2^-22 + 2^-24, the additions 2^-24 a tile (of 16 at least), and 2^-24 for each
    of up to 1216 joined parts; 2^-39 of the largest weighted row a position (f16 rows: times 2^9 at most, the span of the
    values).  A reference that is raised scales sums by a power of two, without error."""
    c = Cache(typ, Hkv, hd, page, len(lens), max(lens), seed=hd)
    for r, n in enumerate(lens):
        k = torch.randint(-127, 128, (n, Hkv, hd), device="cuda", generator=c.gen)
        k[:, :, 0] = 127
        climb = torch.linspace(1.0 / n, 1.0, n, device="cuda")[:, None].expand(n, Hkv) / 127.0
        v = torch.randn(n, Hkv, hd, device="cuda", generator=c.gen)
        if typ == "q8":
            c.put(c.k, r, 0, k, climb)
            c.put(c.v, r, 0, torch.randint(-127, 128, (n, Hkv, hd), device="cuda", generator=c.gen),
                  torch.rand(n, Hkv, device="cuda", generator=c.gen) + 0.1)
        else:
            c.put(c.k, r, 0, k * climb[..., None])
            c.put(c.v, r, 0, v.clamp(-4, 4))
    q = torch.zeros(len(lens), Hq, hd, device="cuda")
    q[:, :, 0] = rise * torch.linspace(0.75, 1.0, Hq, device="cuda")
    out, lse = c.attend(q, lens, 1.0)
    for r, n in enumerate(lens):
        p = torch.arange(n, device="cuda")
        ks, vs = c.get(c.k, r, p), c.get(c.v, r, p)
        adds = (n / 16 + 1216) * 2.0 ** -24
        for h in range(0, Hq, 3):
            t, x = q[r, h, 0].double() * ks[:, h * Hkv // Hq, 0], vs[:, h * Hkv // Hq]
            w = torch.exp(t - t.max())
            total = w.sum()
            w = w / total
            want = w @ x
            delta = t.abs() * (2.0 ** -22 + hd / 16 * 2.0 ** -23 + 5 * 2.0 ** -24) + 2.0 ** -22
            off = (w @ delta).item()
            bound = (w * (delta + 3 * 2.0 ** -22 + 2.0 ** -24 + adds)) @ x.abs() + want.abs() * (off + adds + 2.0 ** -23)
            bound += 2.0 ** -39 * n * (w * x.abs().amax(-1)).max() * (512 if typ == "f16" else 1) + 2.0 ** -120
            err = (out[r, h].double() - want).abs()
            assert torch.all(err <= bound), (r, h, (err / bound).max().item())
            wlse = (t.max() + torch.log(total)).item()
            assert abs(lse[r, h].item() - wlse) <= off + adds + 3 * 2.0 ** -24 * abs(wlse) + 2.0 ** -22


ROPE = [(6001, 32, 128, 128, "half"), (6001, 32, 128, 128, "interleaved"), (250007, 1, 16, 16, "interleaved"),
        (60003, 3, 80, 20, "half"), (50001, 5, 48, 30, "interleaved"), (5003, 40, 96, 64, "half")]


@pytest.mark.parametrize("T,H,hd,n_rot,layout", ROPE)
def test_rotation_of_many_tokens(T, H, hd, n_rot, layout):
    """Each token's result against the definition (as in test_gpu_rope.py: rounded once, but for 2^-42 of the pair), into
    another tensor and in place."""
    rng = np.random.default_rng(T)
    x = rng.standard_normal((T, H, hd)).astype(np.float32)
    pos = rng.integers(-1000, 1 << 20, size=T).astype(np.int32)
    table = plain.turns(plain.freqs(n_rot))
    rope, dx, dpos = qmm.RopeSpec(torch.from_numpy(table).cuda(), layout, 1.0), torch.from_numpy(x).cuda(), torch.from_numpy(pos).cuda()
    y = torch.full((T, H, hd), float("nan"), device="cuda")
    qmm.qmm_rope(rope, dx, y, dpos)
    f = torch.from_numpy(table).cuda()
    phase = (dpos.long()[:, None] * f[None, :]).double() * (2 * np.pi / 2.0 ** 64)  # wraps by whole turns
    cs, sn = torch.cos(phase)[:, None], torch.sin(phase)[:, None]
    part = dx[..., :n_rot].double()
    a, b = (part[..., : n_rot // 2], part[..., n_rot // 2:]) if layout == "half" else (part[..., 0::2], part[..., 1::2])
    got = y[..., :n_rot].double()
    ga, gb = (got[..., : n_rot // 2], got[..., n_rot // 2:]) if layout == "half" else (got[..., 0::2], got[..., 1::2])
    size = 2.0 ** -42 * (a.abs() + b.abs()) + 2.0 ** -149
    for g, want in ((ga, a * cs - b * sn), (gb, a * sn + b * cs)):
        assert torch.all((g - want).abs() <= 2.0 ** -24 * want.abs() + size)
    assert torch.equal(y[..., n_rot:], dx[..., n_rot:])
    qmm.qmm_rope(rope, dx, dx, dpos)
    assert same_bits(dx, y)


STORE = [("q8", 8, 128, 16, 20011, 7, 0, 128, "half"), ("q8", 1, 64, 16, 60011, 0, 0, 64, "interleaved"),
         ("f16", 2, 80, 32, 60001, 11, 4, 20, "half"), ("q8", 8, 128, 16, 8003, 3, 32, 128, "half"),
         ("f16", 1, 16, 8, 200003, 0, 0, 0, None), ("q8", 3, 48, 1, 30011, 2, 0, 12, "half")]


@pytest.mark.parametrize("typ,Hkv,hd,page,T,pad,Hq,n_rot,layout", STORE)
def test_many_tokens_stored_are_those_stored_a_few_at_a_time(typ, Hkv, hd, page, T, pad, Hq, n_rot, layout):
    """One call against calls of 97 tokens (whose rows test_gpu_pages.py holds to the definition): every byte of both pools
    and of the queries; then all rows read back at once against the pools' values, rounded once."""
    seqs = 3
    most = -(-T // seqs) + 50
    big, small = (Cache(typ, Hkv, hd, page, seqs, most, seed=T, fill=0xA5) for _ in range(2))
    assert torch.equal(big.table, small.table)
    places = torch.randperm(seqs * most, device="cuda", generator=big.gen)[:T]
    seq, pos = (places // most).to(torch.int32), (places % most).to(torch.int32)
    if pad:
        pos[torch.randperm(T, device="cuda", generator=big.gen)[:pad]] = -1
    k, v = (torch.randn(T, Hkv, hd, device="cuda", generator=big.gen) for _ in range(2))
    q = torch.randn(T, Hq, hd, device="cuda", generator=big.gen) if Hq else None
    rope = qmm.RopeSpec(torch.from_numpy(plain.turns(plain.freqs(n_rot))).cuda(), layout) if layout else None
    one, many = (torch.full((T, Hq, hd), 7.0, device="cuda") if Hq else None for _ in range(2))
    qmm.qmm_kv_store(big.pages, k, v, pos, seq=seq, rope=rope, q=q, q_out=one)
    for t in range(0, T, 97):
        i = slice(t, min(t + 97, T))
        qmm.qmm_kv_store(small.pages, k[i], v[i], pos[i], seq=seq[i], rope=rope, q=q[i] if Hq else None,
                         q_out=many[i] if Hq else None)
    assert torch.equal(big.k, small.k) and torch.equal(big.v, small.v)
    if Hq:
        assert same_bits(one, many)
    ko, vo = (torch.full((T, Hkv, hd), 5.0, device="cuda") for _ in range(2))
    qmm.qmm_kv_load(big.pages, pos, ko, vo, seq=seq)
    there = pos >= 0
    for o, pool in ((ko, big.k), (vo, big.v)):
        want = big.get(pool, seq.long(), pos.clamp(min=0)).float()
        assert torch.equal(o[there], want[there]) and torch.all(o[~there] == 5.0)
    assert int(there.sum()) == T - pad


@pytest.mark.parametrize("typ,Hkv,hd,T", [("q8", 8, 128, 60007), ("f16", 8, 128, 60007), ("q8", 1, 16, 400009), ("f16", 3, 80, 90001)])
def test_many_rows_read_back(typ, Hkv, hd, T):
    """More than 64 tokens per CTA; several tokens name one place."""
    c = Cache(typ, Hkv, hd, 16, 2, 5000, seed=hd)
    for s in range(2):
        for pool in (c.k, c.v):
            c.put(pool, s, 0, torch.randint(-127, 128, (5000, Hkv, hd), device="cuda", generator=c.gen),
                  torch.rand(5000, Hkv, device="cuda", generator=c.gen))
    seq = torch.randint(0, 2, (T,), device="cuda", generator=c.gen).to(torch.int32)
    pos = torch.randint(-1, 5000, (T,), device="cuda", generator=c.gen).to(torch.int32)
    ko, vo = (torch.full((T, Hkv, hd), 5.0, device="cuda") for _ in range(2))
    qmm.qmm_kv_load(c.pages, pos, ko, vo, seq=seq)
    only = torch.full((T, Hkv, hd), 5.0, device="cuda")
    qmm.qmm_kv_load(c.pages, pos, None, only, seq=seq)
    there = pos >= 0
    for o, pool in ((ko, c.k), (vo, c.v), (only, c.v)):
        want = c.get(pool, seq.long(), pos.clamp(min=0)).float()
        assert torch.equal(o[there], want[there]) and torch.all(o[~there] == 5.0)
