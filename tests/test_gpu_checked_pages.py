"""The rotary and paged-cache kernels of the bounds-checked build on the GPU: tests/checked_pages_run.py in a process of
its own, results checked and no index check fired."""
import os
import subprocess
import sys

import pytest

from conftest import ROOT

torch = pytest.importorskip("torch")
from block_quantized_weight_q8_gb300 import buildlib  # noqa: E402

pytestmark = pytest.mark.gpu


def test_bounds_checked_pages_run_clean():
    if not torch.cuda.is_available():
        pytest.fail("this test needs a CUDA GPU")
    lib = buildlib.build(checked=True)
    env = dict(os.environ, QMM_LIBRARY=lib)
    r = subprocess.run([sys.executable, os.path.join(ROOT, "tests", "checked_pages_run.py")], env=env, capture_output=True,
                       text=True, timeout=900)
    assert r.returncode == 0 and "checked pages ok" in r.stdout, r.stdout[-2000:] + r.stderr[-3000:]
