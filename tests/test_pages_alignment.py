"""Host-side checks (no GPU) of types that the rotary and cache kernels read in wider pieces than their members."""
import os
import subprocess

from block_quantized_weight_q8_gb300 import buildlib

SOURCE = """#include "kvpages.cuh"
#include "rope_device.cuh"
static_assert(alignof(qmm::TurnTable) % alignof(float4) == 0, "entries of the turn table are read as float4");
static_assert(sizeof(qmm::TurnTable) == qmm::kTurnSteps * sizeof(float4), "and stand side by side");
"""


def test_the_turn_table_is_aligned_for_16_byte_reads(tmp_path):
    src = tmp_path / "align.cu"
    src.write_text(SOURCE)
    cmd = [buildlib._nvcc(), *buildlib.ARCH, *buildlib.NVCC_FLAGS, "-I", buildlib.INCLUDE, "-I", buildlib.CSRC, "-c", str(src),
           "-o", os.devnull]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
