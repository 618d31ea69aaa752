"""Host-side checks of the rotary and paged-cache calls (no GPU): every refusal happens before any CUDA call."""
import ctypes

import pytest

import block_quantized_weight_q8_gb300 as qmm

A = 1 << 20  # a fake, 16-byte aligned address that is never dereferenced
NULL, SHAPE, TYPE, ALIGN, SCRATCH = 1, 2, 3, 4, 5


@pytest.fixture(scope="module")
def lib():
    qmm.build()
    return qmm.load()


def spec(freqs=A, n_rot=64, layout=0, mscale=1.0):
    s = qmm.RopeSpec.__new__(qmm.RopeSpec)
    ctypes.Structure.__init__(s, freqs, n_rot, layout, mscale)
    return s


def pages(**over):
    f = dict(k=A, v=A, table=A, num_pages=10, page_stride=16 * 8 * 132, num_seqs=4, max_pages=3, Hkv=8, hd=128, type=0,
             page_size=16)
    f.update(over)
    s = qmm.KvPages.__new__(qmm.KvPages)
    ctypes.Structure.__init__(s, *[f[n] for n, _ in qmm.KvPages._fields_])
    return s


def at(s):
    return ctypes.addressof(s) if s is not None else None


def test_struct_layouts_match_the_header(tmp_path):
    """The binding's structs have the C compiler's sizes and offsets."""
    import os
    import subprocess
    from conftest import ROOT
    lines = []
    for c, py in (("qmm_kv_pages", qmm.KvPages), ("qmm_rope_spec", qmm.RopeSpec)):
        lines.append('printf("%%zu\\n", sizeof(%s));' % c)
        lines += ['printf("%%zu\\n", offsetof(%s, %s));' % (c, n) for n, _ in py._fields_]
    src = tmp_path / "layout.c"
    src.write_text('#include <stdio.h>\n#include "qmm.h"\nint main(void){%s return 0;}\n' % "".join(lines))
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)],
                   check=True)
    got = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    want = []
    for py in (qmm.KvPages, qmm.RopeSpec):
        want += [ctypes.sizeof(py)] + [getattr(py, n).offset for n, _ in py._fields_]
    assert got == want


def test_page_bytes(lib):
    assert qmm.qmm_kv_page_bytes("q8", 8, 16, 128) == 16 * 8 * 132
    assert qmm.qmm_kv_page_bytes("f16", 2, 32, 80) == 32 * 2 * 160
    for t, Hkv, ps, hd in ((2, 8, 16, 128), (-1, 8, 16, 128), (0, 0, 16, 128), (0, 8, 24, 128), (0, 8, 0, 128),
                           (0, 8, 8192, 128), (0, 8, 16, 120), (0, 8, 16, 272), (0, 2000, 16, 128)):
        assert lib.qmm_kv_page_bytes(t, Hkv, ps, hd) == 0, (t, Hkv, ps, hd)


def test_rope_freqs_refusals(lib):
    f = lib.qmm_rope_freqs
    ok = dict(freqs=A, n_rot=64, base=1e4, scaling=2, factor=8.0, orig=8192.0, lo=1.0, hi=4.0)

    def call(**over):
        x = dict(ok, **over)
        return f(x["freqs"], x["n_rot"], x["base"], x["scaling"], x["factor"], x["orig"], x["lo"], x["hi"], None)
    assert call(freqs=None) == NULL
    assert call(scaling=4) == TYPE and call(scaling=-1) == TYPE
    nan, inf = float("nan"), float("inf")
    for over in (dict(n_rot=0), dict(n_rot=7), dict(n_rot=258), dict(base=1.0), dict(base=nan), dict(base=inf),
                 dict(factor=0.0), dict(factor=nan), dict(orig=0.0), dict(lo=0.0), dict(lo=4.0), dict(hi=nan),
                 dict(hi=inf), dict(scaling=3, orig=-1.0), dict(scaling=1, factor=-2.0)):
        assert call(**over) == SHAPE, over
    assert call(freqs=A + 8) == ALIGN


def test_rope_refusals(lib):
    f = lib.qmm_rope
    ok = dict(spec=spec(), x=A, ldx=256, y=2 * A, ldy=256, pos=A, T=3, H=2, hd=128)

    def call(**over):
        a = dict(ok, **over)
        return f(at(a["spec"]), a["x"], a["ldx"], a["y"], a["ldy"], a["pos"], a["T"], a["H"], a["hd"], 0, None)
    for over in (dict(spec=None), dict(spec=spec(freqs=None)), dict(x=None), dict(y=None), dict(pos=None)):
        assert call(**over) == NULL, over
    assert call(spec=spec(layout=2)) == TYPE
    for over in (dict(T=0), dict(H=0), dict(hd=120), dict(hd=0), dict(ldx=252), dict(ldx=258), dict(ldy=128),
                 dict(spec=spec(n_rot=130)), dict(spec=spec(n_rot=63)), dict(spec=spec(n_rot=0)), dict(T=1 << 31),
                 dict(y=A, ldy=512), dict(H=65537, ldx=65537 * 128, ldy=65537 * 128)):
        assert call(**over) == SHAPE, over
    for over in (dict(x=A + 4), dict(y=2 * A + 8), dict(pos=A + 2), dict(spec=spec(freqs=A + 8))):
        assert call(**over) == ALIGN, over


BAD_PAGES = [(dict(k=None), NULL), (dict(v=None), NULL), (dict(table=None), NULL), (dict(type=2), TYPE),
             (dict(type=-1), TYPE), (dict(hd=100), SHAPE), (dict(Hkv=0), SHAPE), (dict(page_size=12), SHAPE),
             (dict(page_size=0), SHAPE), (dict(num_pages=0), SHAPE), (dict(num_pages=1 << 31), SHAPE),
             (dict(num_seqs=0), SHAPE), (dict(max_pages=0), SHAPE), (dict(page_stride=16 * 8 * 132 - 16), SHAPE),
             (dict(page_stride=16 * 8 * 132 + 8), SHAPE), (dict(k=A + 8), ALIGN), (dict(v=A + 4), ALIGN),
             (dict(table=A + 2), ALIGN)]


def test_store_and_load_refusals(lib):
    ok = dict(c=pages(), k=A, ldk=1024, v=A, ldv=1024, pos=A, seq=A, T=3, rope=spec(), q=A, ldq=4096, qo=A, ldqo=4096,
              Hq=32)

    def store(**over):
        a = dict(ok, **over)
        return lib.qmm_kv_store(at(a["c"]), a["k"], a["ldk"], a["v"], a["ldv"], a["pos"], a["seq"], a["T"], at(a["rope"]),
                                a["q"], a["ldq"], a["qo"], a["ldqo"], a["Hq"], None)

    def load(**over):
        a = dict(ok, **over)
        return lib.qmm_kv_load(at(a["c"]), a["pos"], a["seq"], a["T"], a["k"], a["ldk"], a["v"], a["ldv"], None)
    for over, want in BAD_PAGES:
        assert store(c=pages(**over)) == want, over
        assert load(c=pages(**over)) == want, over
    for over in (dict(c=None), dict(k=None), dict(v=None), dict(pos=None), dict(rope=None), dict(qo=None),
                 dict(rope=spec(freqs=None))):
        assert store(**over) == NULL, over
    assert load(k=None, v=None) == NULL and load(pos=None) == NULL and load(c=None) == NULL
    for over in (dict(T=0), dict(T=1 << 31), dict(ldk=1020), dict(ldv=1026), dict(seq=None, T=5)):
        assert store(**over) == SHAPE, over
        assert load(**over) == SHAPE, over
    for over in (dict(Hq=0), dict(ldq=4092), dict(ldqo=4098), dict(ldqo=8192), dict(rope=spec(n_rot=130))):
        assert store(**over) == SHAPE, over
    for over in (dict(k=A + 4), dict(v=A + 8), dict(pos=A + 1), dict(seq=A + 2)):
        assert store(**over) == ALIGN, over
        assert load(**over) == ALIGN, over
    assert store(q=A + 4) == ALIGN and store(qo=A + 4) == ALIGN and store(rope=spec(freqs=A + 4)) == ALIGN


def test_attend_refusals(lib):
    need = qmm.qmm_kv_attend_scratch_bytes(32, 8, 128)
    assert need > 0 and need % 4 == 0
    for Hq, Hkv, hd in ((32, 6, 128), (0, 8, 128), (32, 0, 128), (32, 8, 100), (65, 1, 128)):
        assert qmm.qmm_kv_attend_scratch_bytes(Hq, Hkv, hd) == 0
    ok = dict(c=pages(), q=A, ldq=4096, lens=A, seq=A, out=A, ldo=4096, lse=A, scratch=A, bytes=need, R=3, Hq=32,
              window=0)

    def call(**over):
        a = dict(ok, **over)
        return lib.qmm_kv_attend(at(a["c"]), a["q"], a["ldq"], a["lens"], a["seq"], a["out"], a["ldo"], a["lse"],
                                 a["scratch"], a["bytes"], a["R"], a["Hq"], 0.1, a["window"], None)
    for over, want in BAD_PAGES:
        assert call(c=pages(**over)) == want, over
    for over in (dict(c=None), dict(q=None), dict(lens=None), dict(out=None), dict(scratch=None)):
        assert call(**over) == NULL, over
    for over in (dict(R=0), dict(R=1 << 31), dict(Hq=30), dict(Hq=0), dict(Hq=8 * 65, ldq=8 * 65 * 128, ldo=8 * 65 * 128),
                 dict(ldq=4092), dict(ldo=4090), dict(window=-1), dict(seq=None, R=5)):
        assert call(**over) == SHAPE, over
    for over in (dict(q=A + 4), dict(out=A + 8), dict(lens=A + 2), dict(seq=A + 1), dict(lse=A + 2), dict(scratch=A + 8)):
        assert call(**over) == ALIGN, over
    assert call(bytes=need - 1) == SCRATCH
