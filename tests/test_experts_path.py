"""The query of the experts' path on the CPU: bad arguments."""
import pytest

import block_quantized_weight_q8_gb300 as qmm
from test_experts_abi import EXPERT_SHAPES, lib  # noqa: F401


def test_bad_arguments(lib):
    base = dict(T=5, k=2, E=4, N=64, K=512)
    for over in EXPERT_SHAPES:
        a = dict(base, **over)
        assert lib.qmm_experts_path(qmm.QMM_Q4_K, 0, a["T"], a["k"], a["E"], a["N"], a["K"]) == -1, over
        with pytest.raises(ValueError):
            qmm.qmm_experts_path("q4_K", True, *(a[n] for n in ("T", "k", "E", "N", "K")))
    assert lib.qmm_experts_path(qmm.QMM_Q8_K, 1, 5, 2, 4, 64, 512) == -1
    assert lib.qmm_experts_path(99, 1, 5, 2, 4, 64, 512) == -1
