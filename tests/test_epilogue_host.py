"""Checks of the epilogue's operands that need no GPU."""
import pytest
import torch

pytest.importorskip("fp8_block_scaled_pf8_amd._lib", reason="libpf8.so not built (run __graft_entry__.build())")

from fp8_block_scaled_pf8_amd.epilogue import _aligned_rows  # noqa: E402


@pytest.mark.parametrize("rows", [0, 1, 2])
@pytest.mark.parametrize("cols", [1, 250, 256])
def test_a_pitch_counts_from_two_rows_on(rows, cols):
    t = torch.zeros((rows, cols), dtype=torch.bfloat16)
    if rows > 1 and cols % 8:
        with pytest.raises(ValueError, match="pitch"):
            _aligned_rows(t, "residual", t.shape, t.device)
    else:
        p, ld = _aligned_rows(t, "residual", t.shape, t.device)
        assert p == t.data_ptr() and ld % 8 == 0 and ld >= cols
