"""Sizes that the layer's entry points refuse because no launch could take them (no GPU needed)."""
import pytest

L = pytest.importorskip("fp8_block_scaled_pf8_amd._lib", reason="libpf8.so not built (run __graft_entry__.build())")

P = [0x10000 * i for i in range(1, 9)]  # fake, aligned device addresses: validation never dereferences them


def _act_quant(rows, width, gated, bias):
    cols = width // 2 if gated else width
    ws = L.pf8_act_bwd_quant_workspace(rows, cols, gated)
    assert ws == rows // 128 * width * 4
    return L.pf8_act_bwd_quant(rows, cols, P[0], cols, P[1], width, 3, gated, P[2], width, P[3], rows, P[4], rows, P[5], width,
                               P[6] if bias else 0, 0, P[7] if bias else 0, ws if bias else 0, 0)


@pytest.mark.parametrize("gated", [0, 1])
def test_widest_column_sums(gated):
    """Joining partial column sums takes 32 threads a column, of which a grid has under 2^32."""
    assert _act_quant(256, 2 ** 27, gated, True) == L.PF8_ESHAPE
    assert _act_quant(256, 2 ** 30, gated, True) == L.PF8_ESHAPE
    import torch

    if not torch.cuda.is_available():  # on a GPU machine these would be launched
        assert _act_quant(256, 2 ** 27 - 256, gated, True) == L.PF8_ENODEV
        assert _act_quant(256, 2 ** 27, gated, False) == L.PF8_ENODEV
        assert _act_quant(128, 2 ** 27, gated, True) == L.PF8_ENODEV  # one workgroup's sums are the sums
