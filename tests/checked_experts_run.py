"""The added norm, the routing and the experts' products of the bounds-checked library build on small, odd shapes.

Run as its own process with QMM_LIBRARY naming the bounds-checked libqmm.so, as tests/checked_build_run.py is: results
must match the plain definitions and the device status must stay QMM_OK, i.e. no index check fired.  Used by
tests/test_gpu_checked_experts.py; prints "checked experts ok" on success."""
import os
import sys

import numpy as np

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path[:0] = [ROOT, os.path.join(ROOT, "tests")]

import experts_plain as plain  # noqa: E402
import workloads  # noqa: E402

import torch  # noqa: E402

import block_quantized_weight_q8_gb300 as qmm  # noqa: E402
from test_gpu_experts import dev, host, picks, run_glu, run_sum  # noqa: E402


def status(where):
    st = qmm.qmm_device_status(clear=True)
    assert st == 0, "device status %s after %s" % (qmm.STATUS.get(st, st), where)


def main():
    path = os.environ.get("QMM_LIBRARY", "")
    assert path.endswith(os.path.join("_build_checked", "libqmm.so")), path
    assert qmm.load()._name == path
    torch.cuda.set_device(0)
    status("start")
    for act, M, K in (("q8_0", 1, 32), ("q8_0", 3, 4128), ("q8_0", 700, 416), ("q8_K", 5, 768), ("q8_K", 400, 16640), ("q8_0", 2, 20000)):
        x, r = workloads.activations_f32(M, K, seed=1), workloads.activations_f32(M, K, seed=2)
        w = np.random.default_rng(3).uniform(0.5, 1.5, K).astype(np.float32)
        s, h = torch.empty(M, K, device="cuda"), torch.empty(M, K, device="cuda")
        xq = torch.empty(M, qmm.qmm_row_bytes(act, K), dtype=torch.uint8, device="cuda")
        qmm.qmm_add_rmsnorm_quantize(act, dev(x), dev(r), dev(w), plain.EPS, xq=xq, sum=s, h=h)
        ws, wh, wq = plain.add_norm(act, x, r, w, plain.EPS)
        assert np.array_equal(host(s), ws) and np.array_equal(host(h), wh) and np.array_equal(host(xq), wq.reshape(M, -1))
        status("add_rmsnorm %s" % ((act, M, K),))
    for T, E, k, groups, kept, top in ((1, 1, 1, 1, 1, 1), (5, 60, 6, 1, 1, 1), (33, 1024, 32, 1, 1, 1), (70, 256, 8, 8, 4, 2),
                                       (9, 128, 4, 64, 3, 1), (3, 90, 5, 5, 2, 2), (2000, 40, 4, 2, 1, 2)):
        lg = np.random.default_rng(T).standard_normal((T, E)).astype(np.float32)
        bias = np.random.default_rng(E).standard_normal(E).astype(np.float32)
        ids, w = torch.empty(T, k, dtype=torch.int32, device="cuda"), torch.empty(T, k, device="cuda")
        qmm.qmm_route(dev(lg), ids, w, score="sigmoid", bias=dev(bias), groups=groups, groups_kept=kept, group_top=top)
        want = plain.route(lg, bias, k, "sigmoid", groups, kept, top)[0]
        assert np.array_equal(host(ids), want)
        status("route %s" % ((T, E, k, groups),))
    for wtype in qmm.WEIGHT_TYPES:
        for T, k, E, N, K in ((1, 3, 5, 37, 512), (7, 2, 3, 100, 768), (1100, 2, 3, 77, 1024)):
            run_glu(wtype, T, k, E, N, K, absent=0.1)
            run_sum(wtype, T, k, E, N, K, absent=0.1)
            status("%s %s" % (wtype, (T, k, E, N, K)))
    for wtype in ("q4_0", "q8_0", "q5_1"):
        run_glu(wtype, 1500, 2, 3, 131, 288)
        run_sum(wtype, 1500, 2, 3, 131, 288, ids=picks(1500, 2, 3, 1))
        status(wtype + " rows of 9 blocks")
    run_sum("q4_0", 1, 8, 2, 5, 65536)
    status("choice by choice")
    print("checked experts ok")


if __name__ == "__main__":
    main()
