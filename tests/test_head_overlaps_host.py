"""Which tensors of the head norm count as sharing memory (no GPU needed: addresses and strides alone)."""
import pytest
import torch

pytest.importorskip("fp8_block_scaled_pf8_amd._lib", reason="libpf8.so not built (run __graft_entry__.build())")

from fp8_block_scaled_pf8_amd.heads import _may_write  # noqa: E402


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_weights_beside_a_result(dtype):
    """A weight takes as many bytes as its type: a result may begin right behind a bf16 weight, and none in it."""
    size = 64 * torch.empty((), dtype=dtype).element_size()
    buf = torch.zeros(4096, dtype=torch.uint8)
    w = buf[256:256 + size].view(dtype)

    def heads(first):
        return buf[first:first + 2 * 3 * 64 * 2].view(torch.bfloat16).view(2, 3, 64)

    _may_write(heads(256 + size), "q_out", [(w, False)])
    _may_write(heads(1024), "q_out", [(w, False)])
    for first in (256 + size - 16, 256, 0):
        with pytest.raises(ValueError, match="overlaps"):
            _may_write(heads(first), "q_out", [(w, False)])
