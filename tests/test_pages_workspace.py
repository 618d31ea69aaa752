"""The attention's workspace: as much as a call can use, and no byte beyond it."""
import pytest

torch = pytest.importorskip("torch")
import block_quantized_weight_q8_gb300 as qmm  # noqa: E402


def test_size():
    """152 SMs, two CTAs of four warps each (four CTAs for 8-bit rows of up to 64 values), two parts of eight heads' values,
    references and sums and two notes of 16 bytes each per warp."""
    qmm.build()
    for hd in range(16, 257, 16):
        runs = 152 * 4 * (4 if hd <= 64 else 2)
        assert qmm.qmm_kv_attend_scratch_bytes(32, 8, hd) == runs * 2 * (8 * (hd + 2) * 4 + 16), hd


@pytest.mark.gpu
@pytest.mark.parametrize("typ,hd", [("q8", 64), ("q8", 48), ("q8", 80), ("q8", 128), ("q8", 256), ("f16", 64), ("f16", 256)])
@pytest.mark.parametrize("rows", [1, 80])
def test_no_byte_beyond_it(typ, hd, rows):
    """Work for every run, by CTAs and by single warps, with a workspace of just that size between bytes that stay as they
    are; an equal result from a larger workspace."""
    if not torch.cuda.is_available():
        pytest.fail("this test needs a CUDA GPU")
    qmm.build()
    gen = torch.Generator(device="cuda")
    gen.manual_seed(hd)
    Hkv, page, n = 2, 16, 40000 if rows == 1 else 3000
    size = qmm.qmm_kv_page_bytes(typ, Hkv, page, hd)
    most = -(-n // page)
    k, v = (torch.zeros(most, -(-size // 16) * 16, dtype=torch.uint8, device="cuda") for _ in range(2))
    for pool in (k, v):  # rows of small whole values; 8-bit ones with scales of 1
        if typ == "f16":
            pool[:, :size].view(torch.float16).copy_(torch.randint(-9, 10, (most, size // 2), device="cuda", generator=gen))
        else:
            cut = Hkv * page * hd
            pool[:, :cut] = torch.randint(-9, 10, (most, cut), device="cuda", generator=gen).to(torch.int8).view(torch.uint8)
            pool[:, cut:size].view(torch.float32).fill_(1.0)
    table = torch.randperm(most, device="cuda", generator=gen).to(torch.int32)[None].contiguous()
    pages = qmm.KvPages(typ, k, v, table, page, Hkv, hd)
    q = torch.randn(rows, 8, hd, device="cuda", generator=gen)
    lens = torch.randint(n // 2, n, (rows,), device="cuda", generator=gen).to(torch.int32)
    seq = torch.zeros(rows, dtype=torch.int32, device="cuda")
    need, got = qmm.qmm_kv_attend_scratch_bytes(8, Hkv, hd), []
    for room in (need, 4 * need):
        buf = torch.full((room + 8192,), 0xA5, dtype=torch.uint8, device="cuda")
        out = torch.empty_like(q)
        qmm.qmm_kv_attend(pages, q, lens, out, buf[4096: 4096 + room], room, hd ** -0.5, seq=seq)
        torch.cuda.synchronize()
        assert torch.all(buf[:4096] == 0xA5) and torch.all(buf[4096 + need:] == 0xA5)
        got.append(out)
    assert torch.equal(got[0].view(torch.int32), got[1].view(torch.int32)) and torch.all(torch.isfinite(got[0]))
    assert qmm.qmm_device_status(clear=True) == 0
