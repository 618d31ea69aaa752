"""The joins of the paged attention and the values read back, in the bounds-checked library build.

Run as its own process with QMM_LIBRARY naming the bounds-checked libqmm.so: rows whose parts come from a few teams and
from many, by CTAs and by single warps, empty rows among them, with the log of the sum; results must match the plain
definitions and no index check may fire.  Used by tests/test_gpu_checked_join.py; prints "checked joins ok" on success."""
import os
import sys

import numpy as np

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path[:0] = [ROOT, os.path.join(ROOT, "tests")]

import pages_plain as plain  # noqa: E402

import torch  # noqa: E402

import block_quantized_weight_q8_gb300 as qmm  # noqa: E402


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def host(t):
    torch.cuda.synchronize()
    return t.cpu().numpy()


def status(where):
    st = qmm.qmm_device_status(clear=True)
    assert st == 0, "device status %s after %s" % (qmm.STATUS.get(st, st), where)


def main():
    path = os.environ.get("QMM_LIBRARY", "")
    assert path.endswith(os.path.join("_build_checked", "libqmm.so")), path
    assert qmm.load()._name == path
    torch.cuda.set_device(0)
    status("start")
    rng = np.random.default_rng(1)
    # 9000 positions of one KV head: more than 64 parts, 32 values of a head each for a CTA; 900: several parts joined by
    # one CTA; 2000 positions, 8 heads of 256: a CTA has several pieces; 160 units and more: single warps
    for typ, Hq, Hkv, hd, page, lens, window in (
            ("q8", 8, 1, 128, 16, [9000, 0, 900], 0), ("f16", 8, 1, 256, 32, [2000], 0), ("q8", 5, 1, 48, 8, [3000, -1], 1500),
            ("q8", 80, 80, 16, 16, [300, 0, 700, 64], 0), ("f16", 96, 48, 32, 4, [90, 500, 1, 0, 33], 0)):
        c = plain.Cache(typ, Hkv, hd, page, len(lens), max(lens), seed=hd)
        for r, n in enumerate(lens):
            c.fill(r, max(n, 0), rng)
        k, v = dev(c.k), dev(c.v)
        pages = qmm.KvPages(typ, k, v, dev(c.table), page, Hkv, hd)
        R, what = len(lens), "%s %d heads on %d of %d" % (typ, Hq, Hkv, hd)
        q = rng.standard_normal((R, Hq, hd)).astype(np.float32)
        n = qmm.qmm_kv_attend_scratch_bytes(Hq, Hkv, hd)
        scratch = torch.empty(n, dtype=torch.uint8, device="cuda")
        out, lse = torch.full(q.shape, 9.0, device="cuda"), torch.full((R, Hq), 9.0, device="cuda")
        qmm.qmm_kv_attend(pages, dev(q), dev(np.array(lens, np.int32)), out, scratch, n, hd ** -0.5, lse=lse, window=window)
        status("attend " + what)
        want, wlse, bound, lbound = plain.attend(c, q, lens, range(R), hd ** -0.5, window)
        got, glse, kept, some = host(out), host(lse), np.array(lens) >= 0, np.array(lens) > 0
        assert np.all(np.abs(got[kept] - want[kept]) <= bound[kept]), what
        assert np.all(np.abs(glse[some] - wlse[some]) <= lbound[some]), what
        assert np.all(np.isneginf(glse[np.array(lens) == 0])) and np.all(got[~kept] == 9.0) and np.all(glse[~kept] == 9.0)
        T = 50
        pos, seq = rng.integers(0, lens[0], size=T).astype(np.int32), np.zeros(T, np.int32)
        ko, vo = torch.empty(T, Hkv, hd, device="cuda"), torch.empty(T, Hkv, hd, device="cuda")
        qmm.qmm_kv_load(pages, dev(pos), ko, vo, seq=dev(seq))
        status("load " + what)
        for o, pool in ((ko, c.k), (vo, c.v)):
            assert np.array_equal(host(o), np.stack([c.get(pool, 0, p) for p in pos]).astype(np.float32)), what
    print("checked joins ok")


if __name__ == "__main__":
    main()
