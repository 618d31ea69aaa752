"""The rotary and paged-cache kernels of the bounds-checked library build on small, odd shapes.

Run as its own process with QMM_LIBRARY naming the bounds-checked libqmm.so, as tests/checked_build_run.py is: results
must match the plain definitions and the device status must stay QMM_OK, i.e. no index check fired.  Used by
tests/test_gpu_checked_pages.py; prints "checked pages ok" on success."""
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
    for T, H, hd, n_rot, layout in ((1, 1, 16, 2, "half"), (37, 3, 80, 20, "half"), (5, 33, 256, 256, "interleaved"),
                                    (9, 2, 48, 12, "interleaved"), (3, 5, 96, 64, "half")):
        x = rng.standard_normal((T, H, hd)).astype(np.float32)
        pos = rng.integers(0, 9000, size=T).astype(np.int32)
        table = plain.turns(plain.freqs(n_rot))
        y = torch.empty(x.shape, device="cuda")
        qmm.qmm_rope(qmm.RopeSpec(dev(table), layout), dev(x), y, dev(pos))
        want, size = plain.rotate(x, pos, table, layout)
        assert np.all(np.abs(host(y) - want) <= 2.0 ** -24 * np.abs(want) + 2.0 ** -42 * size)
        status("rope %s" % ((T, H, hd, n_rot, layout),))
    for typ, Hq, Hkv, hd, page, lens, window in (
            ("q8", 8, 2, 64, 16, [33, 0, 100, -1, 1], 0), ("q8", 12, 1, 128, 4, [77, 300], 40),
            ("f16", 6, 2, 80, 8, [17, 90], 0), ("f16", 3, 1, 256, 32, [65], 0), ("q8", 5, 5, 192, 1, [40, 9], 0),
            ("q8", 40, 40, 32, 16, [20, 33, 7, 64], 0), ("f16", 80, 40, 128, 16, [20, 33, 7, 64, 700], 0)):
        c = plain.Cache(typ, Hkv, hd, page, len(lens), max(lens), seed=hd)
        k, v = dev(c.k), dev(c.v)
        pages = qmm.KvPages(typ, k, v, dev(c.table), page, Hkv, hd)
        seq = np.concatenate([np.full(max(n, 0), s) for s, n in enumerate(lens)]).astype(np.int32)
        pos = np.concatenate([np.arange(max(n, 0)) for n in lens]).astype(np.int32)
        T = len(pos)
        kx, vx = (rng.standard_normal((T, Hkv, hd)).astype(np.float32) for _ in range(2))
        q = rng.standard_normal((T, Hq, hd)).astype(np.float32)
        table = plain.turns(plain.freqs(hd))
        qo = torch.empty(q.shape, device="cuda")
        qmm.qmm_kv_store(pages, dev(kx), dev(vx), dev(pos), seq=dev(seq), rope=qmm.RopeSpec(dev(table)), q=dev(q), q_out=qo)
        kr = plain.rotate(kx, pos, table)[0].astype(np.float32)
        for t in range(T):
            c.put(c.k, seq[t], pos[t], kr[t])
            c.put(c.v, seq[t], pos[t], vx[t])
        assert np.array_equal(host(k), c.k) and np.array_equal(host(v), c.v)
        status("store " + typ)
        ko, vo = torch.empty(kx.shape, device="cuda"), torch.empty(kx.shape, device="cuda")
        qmm.qmm_kv_load(pages, dev(pos), ko, vo, seq=dev(seq))
        want = np.stack([c.get(c.k, seq[t], pos[t]) for t in range(T)]).astype(np.float32)
        assert np.array_equal(host(ko), want)
        status("load " + typ)
        R = len(lens)
        qa = rng.standard_normal((R, Hq, hd)).astype(np.float32)
        n = qmm.qmm_kv_attend_scratch_bytes(Hq, Hkv, hd)
        scratch = torch.empty(n, dtype=torch.uint8, device="cuda")
        out, lse = torch.zeros(qa.shape, device="cuda"), torch.zeros(R, Hq, device="cuda")
        qmm.qmm_kv_attend(pages, dev(qa), dev(np.array(lens, np.int32)), out, scratch, n, hd ** -0.5, lse=lse, window=window)
        ref, _, bound, _ = plain.attend(c, qa, lens, range(R), hd ** -0.5, window)
        kept = np.array(lens) >= 0
        assert np.all(np.abs(host(out) - ref)[kept] <= bound[kept])
        status("attend " + typ)
    print("checked pages ok")


if __name__ == "__main__":
    main()
