"""Calls of the block norm that its documentation allows, or has to refuse, beside those of test_gpu_norm.py."""
import pytest
import torch

import fp8_block_scaled_pf8_amd as pf8
from tests.gpu_helpers import DEV

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def _rand(shape, seed, scale=1.0):
    return (torch.randn(shape, generator=torch.Generator().manual_seed(seed)) * scale).to(BF).to(DEV)


@pytest.mark.parametrize("rows,cols", [(700, 1536), (37, 2051), (1, 200)])
def test_captured_backward_adds_to_the_callers_buffers(rows, cols):
    """The sums of a pass come out the same each time, and are added in FP32: equal to eager gradients added one by one."""
    k = dict(h=_rand((rows, cols), 1, 2.0), y=_rand((rows, cols), 2), w_pre=_rand((cols,), 3), w_post=_rand((cols,), 4),
             gate=_rand((cols,), 5))
    dr, dx = _rand((rows, cols), 6), _rand((rows, cols), 7)
    names = ("dw_pre", "dw_post", "dgate")
    sums = {n + "_out": _rand((cols,), 8 + i).float() for i, n in enumerate(names)}
    want = [t.clone() for t in sums.values()]
    warm = {n: t.clone() for n, t in sums.items()}
    pf8.block_norm_backward(dr, dx, **k, **warm, accumulate=True)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g = pf8.block_norm_backward(dr, dx, **k, **sums, accumulate=True)
    for i in range(4):
        k["h"].copy_(_rand((rows, cols), 50 + i, 2.0))
        dx.copy_(_rand((rows, cols), 60 + i))
        graph.replay()
        eager = pf8.block_norm_backward(dr, dx, **k)
        for w, n in zip(want, names):
            w.add_(getattr(eager, n))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(sums.values(), want)), i
        assert torch.equal(g.dh, eager.dh) and torch.equal(g.dy, eager.dy)
    assert g.dw_pre is sums["dw_pre_out"] and g.dw_post is sums["dw_post_out"] and g.dgate is sums["dgate_out"]


def test_a_gate_without_a_branch_is_refused():
    """As block_norm refuses it: there is nothing that the gate could multiply."""
    norm = pf8.BlockNorm(256, device=DEV)
    h, gate = _rand((4, 256), 1), _rand((4, 256), 2)
    for call in (norm, norm.quantised):
        with pytest.raises(ValueError, match="gate"):
            call(h, None, gate)
        call(h)
    learned = pf8.BlockNorm(256, gate=True, device=DEV)
    assert learned(h)[1].shape == h.shape  # the first block's norm: the module's own gate waits for a branch
