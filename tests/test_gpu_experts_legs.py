"""Summed products of more choices than the CTA has threads: long rows of many choices leave shared memory for one warp."""
import os
import subprocess
import sys

import pytest

from conftest import ROOT
from test_gpu_experts import gpu, picks, run_sum  # noqa: F401

torch = pytest.importorskip("torch")
from block_quantized_weight_q8_gb300 import buildlib  # noqa: E402

pytestmark = pytest.mark.gpu

# (format, K, k): at these the plan for 96 output rows has a single warp of 32 threads
ONE_WARP = [("q4_0", 2848, 62), ("q4_0", 4896, 36), ("q8_0", 2848, 62), ("q8_0", 5408, 33), ("q4_1", 3872, 46), ("q5_0", 2848, 62),
            ("q5_1", 4640, 37), ("q4_K", 3584, 50), ("q4_K", 5888, 33), ("q5_K", 3328, 58), ("q6_K", 3328, 58), ("q6_K", 5376, 36),
            ("q2_K", 4096, 45), ("q2_K", 4352, 45)]


@pytest.mark.parametrize("T", [1, 4])
@pytest.mark.parametrize("wtype,K,k", ONE_WARP)
def test_more_choices_than_threads(wtype, K, k, T):
    run_sum(wtype, T, k, 5, 96, K, absent=0.1)


@pytest.mark.parametrize("wtype,K,k", [("q8_0", 2560, 64), ("q4_K", 2048, 64), ("q6_K", 768, 40), ("q2_K", 1280, 33), ("q5_1", 992, 63)])
def test_many_choices_of_long_rows(wtype, K, k):
    for T in (1, 3):
        run_sum(wtype, T, k, 6, 200, K, absent=0.1)


def test_choices_behind_the_first_warp_alone():
    """Only the choices beyond the 32nd are there."""
    for T in (1, 4):
        ids = picks(T, 50, 5, 3)
        ids[:, :32] = -1
        run_sum("q4_K", T, 50, 5, 96, 3584, ids=ids)


def test_bounds_checked():
    """The same calls of the bounds-checked build, in a process of its own: results checked and no index check fired."""
    lib = buildlib.build(checked=True)
    run = ("import os, sys; sys.path[:0] = [%r, %r]\n"
           "import block_quantized_weight_q8_gb300 as qmm\n"
           "from test_gpu_experts_legs import ONE_WARP, run_sum\n"
           "assert qmm.load()._name == os.environ['QMM_LIBRARY']\n"
           "assert qmm.qmm_device_status(clear=True) == 0\n"
           "for wtype, K, k in ONE_WARP:\n"
           "    for T in (1, 4):\n"
           "        run_sum(wtype, T, k, 5, 96, K, absent=0.1)\n"
           "        assert qmm.qmm_device_status(clear=True) == 0, (wtype, K, k, T)\n"
           "print('checked legs ok')\n") % (ROOT, os.path.join(ROOT, "tests"))
    r = subprocess.run([sys.executable, "-c", run], env=dict(os.environ, QMM_LIBRARY=lib), capture_output=True, text=True,
                       timeout=900)
    assert r.returncode == 0 and "checked legs ok" in r.stdout, r.stdout[-2000:] + r.stderr[-3000:]
