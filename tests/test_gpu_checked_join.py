"""The paged attention's joins in the bounds-checked build on the GPU: tests/checked_join_run.py in a process of its own."""
import os
import subprocess
import sys

import pytest

from conftest import ROOT

torch = pytest.importorskip("torch")
from block_quantized_weight_q8_gb300 import buildlib  # noqa: E402

pytestmark = pytest.mark.gpu


def test_bounds_checked_joins_run_clean():
    if not torch.cuda.is_available():
        pytest.fail("this test needs a CUDA GPU")
    env = dict(os.environ, QMM_LIBRARY=buildlib.build(checked=True))
    r = subprocess.run([sys.executable, os.path.join(ROOT, "tests", "checked_join_run.py")], env=env, capture_output=True,
                       text=True, timeout=900)
    assert r.returncode == 0 and "checked joins ok" in r.stdout, r.stdout[-2000:] + r.stderr[-3000:]
