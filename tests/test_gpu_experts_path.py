"""The experts' products on the tensor cores, at shapes where the query says that they take them, whatever the format: rows of
one block, of nine, tiles and chunks that end inside, extreme scales; and the bounds-checked build."""
import os
import subprocess
import sys

import numpy as np
import pytest

import experts_plain as plain
import oracle
import workloads
from conftest import ROOT
from test_gpu_experts import K_of, TYPES, dev, gpu, host, picks, run_glu, run_sum, scratch_of  # noqa: F401
from test_gpu_experts_many import extreme_weights

torch = pytest.importorskip("torch")
import block_quantized_weight_q8_gb300 as qmm  # noqa: E402
from block_quantized_weight_q8_gb300 import buildlib  # noqa: E402

pytestmark = pytest.mark.gpu

SHAPES = [(2000, 2, 3, 129, 1024), (12000, 1, 2, 77, 288), (16000, 1, 1, 130, 32), (1600, 4, 13, 100, 1312)]


def on_tensor_cores(wtype, gated, *shape):
    assert qmm.qmm_experts_path(wtype, gated, *shape) == 1, (wtype, gated, shape)


def test_both_paths_are_reported():
    for wtype in TYPES:
        for gated in (False, True):
            assert qmm.qmm_experts_path(wtype, gated, 1, 8, 64, 1024, 2048) == 0
            assert qmm.qmm_experts_path(wtype, gated, 4096, 8, 64, 1024, 2048) == 1


@pytest.mark.parametrize("wtype", TYPES)
@pytest.mark.parametrize("T,k,E,N,K", SHAPES)
def test_glu(wtype, T, k, E, N, K):
    on_tensor_cores(wtype, True, T, k, E, N, K_of(wtype, K))
    run_glu(wtype, T, k, E, N, K_of(wtype, K), kind="gelu" if T == 1600 else "silu", absent=0.05)


@pytest.mark.parametrize("wtype", TYPES)
@pytest.mark.parametrize("T,k,E,N,K", SHAPES)
def test_sum(wtype, T, k, E, N, K):
    on_tensor_cores(wtype, False, T, k, E, N, K_of(wtype, K))
    run_sum(wtype, T, k, E, N, K_of(wtype, K), weighted=T != 1600, residual=T != 12000, absent=0.05)


@pytest.mark.parametrize("wtype", TYPES)
def test_extreme_scales(wtype):
    """As in tests/test_gpu_experts_many.py, for every format on the tensor cores: an error against 1e-5 of the sum of the
    values' shares; the operands' 2^-21 each and at most 32 steps truncated to 2^-23 are 2^-20 + 32 2^-23 = 4.8e-6."""
    T, E, N, K = 4500, 2, 120, 1024
    on_tensor_cores(wtype, False, T, 1, E, N, K)
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


def test_bounds_checked():
    """Every format on the tensor cores in the bounds-checked build, in a process of its own."""
    lib = buildlib.build(checked=True)
    run = ("import os, sys; sys.path[:0] = [%r, %r]\n"
           "import block_quantized_weight_q8_gb300 as qmm\n"
           "from test_gpu_experts_path import on_tensor_cores, run_glu, run_sum\n"
           "assert qmm.load()._name == os.environ['QMM_LIBRARY']\n"
           "assert qmm.qmm_device_status(clear=True) == 0\n"
           "for wtype in qmm.WEIGHT_TYPES:\n"
           "    for gated, run in ((True, run_glu), (False, run_sum)):\n"
           "        on_tensor_cores(wtype, gated, 5000, 2, 3, 77, 768)\n"
           "        run(wtype, 5000, 2, 3, 77, 768, absent=0.1)\n"
           "        assert qmm.qmm_device_status(clear=True) == 0, (wtype, gated)\n"
           "print('checked path ok')\n") % (ROOT, os.path.join(ROOT, "tests"))
    r = subprocess.run([sys.executable, "-c", run], env=dict(os.environ, QMM_LIBRARY=lib), capture_output=True, text=True,
                       timeout=900)
    assert r.returncode == 0 and "checked path ok" in r.stdout, r.stdout[-2000:] + r.stderr[-3000:]
