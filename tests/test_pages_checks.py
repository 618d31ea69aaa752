"""The cache kernels' computed accesses stand behind index checks (host-side, by reading the sources): every line that
forms an address in the outputs, the workspace, the page table or a pool has a QMM_IN_BOUNDS on it or a few lines before."""
import os
import re

import pytest

from block_quantized_weight_q8_gb300 import buildlib

ACCESSES = {
    # outputs and log-sums, parts and notes of the joins, the table's entries
    "attend.cu": {r"\(a\.out \+": 3, r"a\.lse\[": 3, r"a\.joins\[": 3, r"\(out \+": 3, r"\(part \+": 3, r"part\[": 3,
                  r"\? p : a\.parts": 3, r"__ldg\(pages": 3},
    # rows' scales and codes (one check for all of a share's codes)
    "kvpages.cu": {r"\(pool_scale \+": 3, r"\(scales \+": 6, r"\(pool \+": 36},
}


def body(path):
    lines = open(path).read().split("\n")
    # device code: up to the host's entry points
    end = next(i for i, x in enumerate(lines) if x.startswith('extern "C"'))
    return [x.split("//", 1)[0] for x in lines[:end]]


@pytest.mark.parametrize("name", sorted(ACCESSES))
def test_accesses_are_checked(name):
    lines = body(os.path.join(buildlib.CSRC, name))
    for pattern, lines_before in ACCESSES[name].items():
        at = [i for i, x in enumerate(lines) if re.search(pattern, x)]
        assert at, pattern
        for i in at:
            near = "\n".join(lines[max(0, i - lines_before): i + 1])
            assert "QMM_IN_BOUNDS" in near, "%s:%d: %s" % (name, i + 1, lines[i].strip())
