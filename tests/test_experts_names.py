"""Choices by name and spec fields that the mixture-of-experts calls refuse with ValueError, before anything else (no GPU)."""
import pytest

torch = pytest.importorskip("torch")
import block_quantized_weight_q8_gb300 as qmm  # noqa: E402


def test_unknown_names():
    qmm.build()
    f, i, b = torch.zeros(2, 4), torch.zeros(2, 1, dtype=torch.int32), torch.zeros(2, 34, dtype=torch.uint8)
    h, W = torch.zeros(2, 1, 32), torch.zeros(3, 32, 34, dtype=torch.uint8)
    for score in ("relu", None, 0, []):
        with pytest.raises(ValueError, match="score"):
            qmm.qmm_route(f, i, f[:, :1], score=score)
    for gate in ("relu", None, 0, []):
        with pytest.raises(ValueError, match="gate"):
            qmm.qmm_experts_glu("q8_0", W, W, b, i, h, b, 34, gate=gate)
    with pytest.raises(ValueError, match="type"):
        qmm.qmm_experts_glu("q9_0", W, W, b, i, h, b, 34)
    with pytest.raises(ValueError, match="type"):
        qmm.qmm_experts_sum("q9_0", W, h, i, None, f, b, 34)
    with pytest.raises(ValueError, match="type"):
        qmm.qmm_add_rmsnorm_quantize("q9_0", f, f, f[0], 1e-6, b)
    with pytest.raises(ValueError, match="type"):
        qmm.qmm_experts_path("q9_0", True, 1, 1, 1, 32, 32)
    with pytest.raises(ValueError, match="type"):
        qmm.qmm_experts_scratch_bytes("q9_0", 1, 1, 1, 32, 32)


@pytest.mark.parametrize("over", [dict(groups=(1 << 32) + 1), dict(groups=2, groups_kept=(1 << 32) + 1),
                                  dict(group_top=1 << 31), dict(group_top=(1 << 40) + 2)])
def test_fields_beyond_32_bits(over):
    """They would arrive as other numbers."""
    with pytest.raises(ValueError, match="groups"):
        qmm.qmm_route(torch.zeros(2, 4), torch.zeros(2, 1, dtype=torch.int32), torch.zeros(2, 1), **over)
