"""Host-side checks of the mixture-of-experts calls (no GPU): every refusal happens before any CUDA call."""
import ctypes
import os
import subprocess

import pytest

import block_quantized_weight_q8_gb300 as qmm

from conftest import ROOT

A = 1 << 20  # a fake, 16-byte aligned address that is never dereferenced
NULL, SHAPE, TYPE, ALIGN, SCRATCH = 1, 2, 3, 4, 5
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    qmm.build()
    return qmm.load()


def test_spec_layout_matches_the_header(tmp_path):
    lines = ['printf("%zu\\n", sizeof(qmm_route_spec));']
    lines += ['printf("%%zu\\n", offsetof(qmm_route_spec, %s));' % n for n, _ in qmm.RouteSpec._fields_]
    src, exe = tmp_path / "layout.c", tmp_path / "layout"
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "qmm.h"\nint main(void){%s return 0;}\n' % "".join(lines))
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)],
                   check=True)
    got = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    assert got == [ctypes.sizeof(qmm.RouteSpec)] + [getattr(qmm.RouteSpec, n).offset for n, _ in qmm.RouteSpec._fields_]


def test_add_rmsnorm_quantize_refusals(lib):
    ok = dict(act=1, x=A, r=A, sum=A, w=A, h=A, xq=A, M=3, K=512)

    def call(**over):
        a = dict(ok, **over)
        return lib.qmm_add_rmsnorm_quantize(a["act"], a["x"], a["r"], a["sum"], a["w"], 1e-6, a["h"], a["xq"], a["M"], a["K"],
                                            None)
    for act in (0, 2, -1, 10):
        assert call(act=act) == TYPE, act
    for over in (dict(x=None), dict(r=None), dict(w=None), dict(h=None, xq=None)):
        assert call(**over) == NULL, over
    for over in (dict(M=0), dict(M=1 << 31), dict(K=0), dict(K=48), dict(act=5, K=96), dict(K=65536 + 32)):
        assert call(**over) == SHAPE, over
    for name in ("x", "r", "sum", "w", "h", "xq"):
        assert call(**{name: A + 8}) == ALIGN, name


def test_route_refusals(lib):
    ok = dict(score=0, k=4, groups=4, groups_kept=2, group_top=2, renorm=1, scale=1.0)

    def call(spec=True, logits=A, ld=64, bias=A, ids=A, weights=A, T=5, E=64, **over):
        s = qmm.RouteSpec(*[dict(ok, **over)[n] for n, _ in qmm.RouteSpec._fields_])
        return lib.qmm_route(ctypes.addressof(s) if spec else None, logits, ld, bias, ids, weights, T, E, None)
    for over in (dict(spec=False), dict(logits=None), dict(ids=None), dict(weights=None)):
        assert call(**over) == NULL, over
    assert call(score=2) == TYPE and call(score=-1) == TYPE
    for over in (dict(T=0), dict(T=1 << 31), dict(E=0), dict(E=1028, ld=2000), dict(ld=63), dict(groups=0), dict(groups=5),
                 dict(groups=65, E=65, ld=65, k=1), dict(groups_kept=0), dict(groups_kept=5), dict(group_top=0),
                 dict(group_top=3), dict(k=0), dict(k=33, groups_kept=4), dict(k=33, groups=1, groups_kept=1),
                 dict(k=17, groups_kept=1), dict(scale=NAN), dict(scale=INF)):
        assert call(**over) == SHAPE, over
    for name in ("logits", "bias", "ids", "weights"):
        assert call(**{name: A + 2}) == ALIGN, name


EXPERT_SHAPES = [dict(T=0), dict(T=1 << 31), dict(k=0), dict(k=65), dict(E=0), dict(E=1025), dict(N=0), dict(K=0),
                 dict(K=500), dict(K=65536 + 256), dict(T=1 << 22, k=8), dict(E=1024, N=1 << 21)]


def test_scratch_bytes(lib):
    for wt in qmm.WEIGHT_TYPES:
        assert qmm.qmm_experts_scratch_bytes(wt, 1, 8, 64, 1024, 2048) > 0
        assert qmm.qmm_experts_scratch_bytes(wt, 4096, 8, 64, 1024, 2048) > 0
    base = dict(T=5, k=2, E=4, N=64, K=512)
    for over in EXPERT_SHAPES:
        a = dict(base, **over)
        assert lib.qmm_experts_scratch_bytes(qmm.QMM_Q4_K, a["T"], a["k"], a["E"], a["N"], a["K"]) == 0, over
    assert lib.qmm_experts_scratch_bytes(qmm.QMM_Q8_K, 5, 2, 4, 64, 512) == 0


def test_experts_glu_refusals(lib):
    need = qmm.qmm_experts_scratch_bytes("q4_K", 5, 2, 4, 64, 512)
    ok = dict(wt=qmm.QMM_Q4_K, kind=0, Wg=A, Wu=A, xq=A, ids=A, h=A, scratch=A, bytes=need, T=5, k=2, E=4, N=64, K=512)

    def call(**over):
        a = dict(ok, **over)
        return lib.qmm_experts_glu(a["wt"], a["kind"], a["Wg"], a["Wu"], a["xq"], a["ids"], a["h"], a["scratch"], a["bytes"],
                                   a["T"], a["k"], a["E"], a["N"], a["K"], None)
    for name in ("Wg", "Wu", "xq", "ids", "h", "scratch"):
        assert call(**{name: None}) == NULL, name
        assert call(**{name: A + 2}) == ALIGN, name
    assert call(wt=qmm.QMM_Q8_K) == TYPE and call(wt=99) == TYPE and call(kind=2) == TYPE and call(kind=-1) == TYPE
    for over in EXPERT_SHAPES:
        assert call(**over) == SHAPE, over
    assert call(bytes=need - 1) == SCRATCH


def test_experts_sum_refusals(lib):
    need = qmm.qmm_experts_scratch_bytes("q6_K", 5, 2, 4, 64, 512)
    ok = dict(wt=qmm.QMM_Q6_K, W=A, h=A, ids=A, weights=A, residual=A, y=A, scratch=A, bytes=need, T=5, k=2, E=4, N=64, K=512)

    def call(**over):
        a = dict(ok, **over)
        return lib.qmm_experts_sum(a["wt"], a["W"], a["h"], a["ids"], a["weights"], a["residual"], a["y"], a["scratch"],
                                   a["bytes"], a["T"], a["k"], a["E"], a["N"], a["K"], None)
    for name in ("W", "h", "ids", "y", "scratch"):
        assert call(**{name: None}) == NULL, name
    for name in ("W", "h", "ids", "weights", "residual", "y", "scratch"):
        assert call(**{name: A + 2}) == ALIGN, name
    assert call(wt=qmm.QMM_Q8_K) == TYPE and call(wt=-1) == TYPE
    for over in EXPERT_SHAPES:
        assert call(**over) == SHAPE, over
    assert call(bytes=need - 1) == SCRATCH
