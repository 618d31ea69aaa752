"""Plain definitions, in 64 bits on the host, of rotary positions, the paged cache's rows and attention over them: what
tests/test_gpu_rope.py and tests/test_gpu_pages.py compare the kernels with.  Numpy, no code of the library."""
import math

import numpy as np


def turns(freqs):
    """Frequencies in radians per position as the table's 64-bit fractions of a turn (int64 bits)."""
    out = []
    for f in np.asarray(freqs, dtype=np.float64):
        t = float(f) / (2 * math.pi)
        out.append(int((t - math.floor(t)) * 2.0 ** 64) % (1 << 64))
    return np.array(out, dtype=np.uint64).view(np.int64)


def freqs(n_rot, base=10000.0, scaling="plain", factor=1.0, orig_len=0.0, lo=0.0, hi=0.0):
    out = []
    for i in range(n_rot // 2):
        f = base ** (-2.0 * i / n_rot)
        if scaling == "linear":
            f /= factor
        elif scaling == "bands":
            keep = min(max((orig_len * f / (2 * math.pi) - lo) / (hi - lo), 0.0), 1.0)
            f = (1 - keep) * f / factor + keep * f
        elif scaling == "yarn":
            at = [n_rot * math.log(orig_len / (t * 2 * math.pi)) / (2 * math.log(base)) for t in (hi, lo)]
            first, last = max(math.floor(at[0]), 0), min(math.ceil(at[1]), n_rot - 1)
            keep = 1 - min(max((i - first) / max(last - first, 0.001), 0.0), 1.0)
            f = (1 - keep) * f / factor + keep * f
        out.append(f)
    return np.array(out)


def rotate(x, pos, table, layout="half", mscale=1.0, inverse=False):
    """x [T][H][hd] (f32) -> the rotated values in f64, and what their error scales with, m (|a| + |b|)."""
    F = table.view(np.uint64)
    p = np.asarray(pos).astype(np.int64).view(np.uint64)
    y, size = x.astype(np.float64), np.zeros(x.shape)
    for i in range(F.size):
        a, b = (i, i + F.size) if layout == "half" else (2 * i, 2 * i + 1)
        t = (p * F[i]).astype(np.float64) * (2 * math.pi / 2.0 ** 64)
        c, s = np.cos(t)[:, None] * mscale, np.sin(t)[:, None] * mscale * (-1 if inverse else 1)
        xa, xb = x[:, :, a].astype(np.float64), x[:, :, b].astype(np.float64)
        y[:, :, a], y[:, :, b] = xa * c - xb * s, xa * s + xb * c
        size[:, :, a] = size[:, :, b] = mscale * (np.abs(xa) + np.abs(xb))
    return y, size


def q8(x):
    """f32 rows -> (int8 codes, f32 d): d = amax / 127, codes rne(x * (127 / amax)), every step rounded to f32."""
    x = x.astype(np.float32)
    amax = np.abs(x).max(-1)
    with np.errstate(divide="ignore", invalid="ignore"):
        inv = np.where(amax != 0, np.float32(127) / amax, np.float32(0)).astype(np.float32)
        c = np.rint(x * inv[..., None])
    return np.clip(c, -128, 127).astype(np.int8), (amax / np.float32(127)).astype(np.float32)


class Cache:
    """A cache on the host: pools of bytes, a shuffled table, rows written and read one by one."""

    def __init__(self, typ, Hkv, hd, page, seqs, most, seed=0, stride=None, fill=0xFF):
        rng = np.random.default_rng(seed)
        self.typ, self.Hkv, self.hd, self.page = typ, Hkv, hd, page
        self.row = hd if typ == "q8" else 2 * hd
        self.bytes = page * Hkv * (self.row + (4 if typ == "q8" else 0))
        self.stride = stride or -(-self.bytes // 16) * 16
        self.max_pages = -(-most // page)
        self.pages = seqs * self.max_pages + 2
        ids = rng.permutation(self.pages)[: seqs * self.max_pages]
        self.table = ids.reshape(seqs, self.max_pages).astype(np.int32)
        self.k = np.full((self.pages, self.stride), fill, dtype=np.uint8)
        self.v = self.k.copy()

    def place(self, seq, pos):
        return int(self.table[seq, pos // self.page]), pos % self.page

    def put(self, pool, seq, pos, x):
        """x [Hkv][hd] f32 into position pos of sequence seq."""
        page, o = self.place(seq, pos)
        codes, d = q8(x) if self.typ == "q8" else (x.astype(np.float16), None)
        for h in range(self.Hkv):
            at = (h * self.page + o) * self.row
            pool[page, at: at + self.row] = codes[h].view(np.uint8)
            if d is not None:
                at = self.Hkv * self.page * self.hd + 4 * (h * self.page + o)
                pool[page, at: at + 4] = d[h: h + 1].view(np.uint8)

    def get(self, pool, seq, pos):
        """The row's values [Hkv][hd] in f64."""
        page, o = self.place(seq, pos)
        out = np.empty((self.Hkv, self.hd))
        for h in range(self.Hkv):
            at = (h * self.page + o) * self.row
            raw = pool[page, at: at + self.row]
            if self.typ == "q8":
                at = self.Hkv * self.page * self.hd + 4 * (h * self.page + o)
                out[h] = raw.view(np.int8).astype(np.float64) * float(pool[page, at: at + 4].copy().view(np.float32)[0])
            else:
                out[h] = raw.copy().view(np.float16).astype(np.float64)
        return out

    def fill(self, seq, n, rng, loud=True):
        for p in range(n):
            k = rng.standard_normal((self.Hkv, self.hd)).astype(np.float32)
            if loud:
                k[:, :: 17] *= 6
            self.put(self.k, seq, p, k)
            self.put(self.v, seq, p, rng.standard_normal((self.Hkv, self.hd)).astype(np.float32))


def attend(cache, q, lens, seqs, scale, window=0):
    """(out, lse, error bound of out, error bound of lse); rows with a negative length are left NaN.

    The bounds, from the kernel's roundings.  A score's terms are q_i k_i with q as two f16 (2^-22), the codes exact,
    summed by hd / 16 matrix steps that cut off (2^-23 of the largest partial sum each, at most A = scale sum |q k|),
    four f32 products and the softmax's argument (2^-24 of A each): d = A (2^-22 + (hd / 16) 2^-23 + 5 * 2^-24).  A
    weight is off by d and the exponential's 2^-22, twice (numerator and sum), by its split (2^-22) and by the sums: two
    matrix steps per tile and one f32 FMA per tile of its warp, the four warps and the joined parts (2^-24 each).

    A split into two f16 is off by 2^-22 of the value only while its low half is normal; below, by half of f16's least
    step, 2^-25.  Queries are split times 2^(14 - e), 2^e <= max |q|: 2^-39 max |q| a term, so d grows by scale 2^-39
    max |q| sum |k|.  Weights w, relative to 2^m_run, are split as w d 2^(10 - e), 2^e at most the largest value scale d
    (f16 rows: d = 1, e = 0): 2^-35 max(d) a position, times a code: 2^-35 max |v|.  m_run is less than 1 over the
    warp's largest score, so that score's w is over 1/2 and what a join scales by is at most 2^(own maximum - the
    row's): with the softmax's weights relative to the row's largest, 2^-34 max |v| a position, over their sum.
    (Without it: one position takes the softmax and its code is 0, so the result is the others' far smaller weights.)"""
    R, Hq, hd = q.shape
    G = Hq // cache.Hkv
    out, bound = np.full((R, Hq, hd), np.nan), np.zeros((R, Hq, hd))
    lse, lbound = np.full((R, Hq), np.nan), np.zeros((R, Hq))
    for r in range(R):
        n = int(lens[r])
        if n < 0:
            continue
        out[r], lse[r] = 0.0, -np.inf
        if n == 0:
            continue
        first = max(0, n - window) if window else 0
        k = np.stack([cache.get(cache.k, seqs[r], p) for p in range(first, n)])
        v = np.stack([cache.get(cache.v, seqs[r], p) for p in range(first, n)])
        for h in range(Hq):
            t = scale * (k[:, h // G] @ q[r, h].astype(np.float64))
            A = (abs(scale) * (np.abs(k[:, h // G]) @ np.abs(q[r, h].astype(np.float64)))).max()
            w = np.exp(t - t.max())
            total = w.sum()
            out[r, h] = (w / total) @ v[:, h // G]
            lse[r, h] = t.max() + np.log(total)
            d = A * (2.0 ** -22 + hd / 16 * 2.0 ** -23 + 5 * 2.0 ** -24)
            d += abs(scale) * 2.0 ** -39 * np.abs(q[r, h]).max() * np.abs(k[:, h // G]).sum(-1).max()
            steps = 2 * 2.0 ** -22 + ((n - first) / 16 + 8) * 2.0 ** -24
            bound[r, h] = (2 * (d + 2.0 ** -22) + 2.0 ** -22 + steps) * ((w / total) @ np.abs(v[:, h // G])) + 2.0 ** -120
            bound[r, h] += 2.0 ** -34 * np.abs(v[:, h // G]).max() * (n - first) / total
            lbound[r, h] = d + 2.0 ** -22 + steps + 3 * 2.0 ** -24 * abs(lse[r, h])
    return out, lse, bound, lbound
