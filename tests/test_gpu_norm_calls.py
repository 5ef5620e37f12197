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


def test_results_beside_their_inputs_in_one_buffer():
    """Column ranges of one buffer: their rows lie between one another's, and none is shared."""
    buf = torch.zeros((9, 1024), dtype=BF, device=DEV)
    h, y, r, x = (buf[:, 256 * i:256 * i + 256] for i in range(4))
    h.copy_(_rand((9, 256), 1, 2.0))
    y.copy_(_rand((9, 256), 2))
    w = _rand((256,), 3)
    want = pf8.block_norm(h, y, w, w)
    got = pf8.block_norm(h, y, w, w, r_out=r, x_out=x)
    assert got[0] is r and got[1] is x
    assert torch.equal(r, want[0]) and torch.equal(x, want[1])
    for r_bad in (buf[:, 200:456], buf[:, 500:756], buf[:, 255:511]):
        with pytest.raises(ValueError, match="overlaps"):
            pf8.block_norm(h, y, w, w, r_out=r_bad)
    # another pitch over the same memory
    wide = torch.zeros((4, 512), dtype=BF, device=DEV)
    with pytest.raises(ValueError, match="overlaps"):
        pf8.block_norm(wide[:, :256], None, w, x_out=wide.view(-1)[256:1280].view(4, 256))


def test_orthogonalised_beside_its_gradient_in_one_buffer():
    buf = torch.zeros((3, 40, 160), dtype=BF, device=DEV)
    g, out = buf[..., :80], buf[..., 80:]
    g.copy_(_rand((3, 40, 80), 1))
    want = pf8.newton_schulz(g)
    assert pf8.newton_schulz(g, out=out) is out and torch.equal(out, want)
    out.zero_()
    assert torch.equal(pf8.newton_schulz(g[1], out=out[1]), want[1])
    assert torch.equal(pf8.newton_schulz(g[:, :1], out=out[:, :1]), pf8.newton_schulz(g[:, :1]))
    for bad in (buf[..., 79:159], buf[..., :80], buf[:, :, 40:120]):
        with pytest.raises(ValueError, match="overlaps"):
            pf8.newton_schulz(g, out=bad)


def test_orthogonalisation_takes_whole_numbers_of_steps_of_any_type():
    g = _rand((20, 30), 1)
    want = pf8.newton_schulz(g, steps=3)
    assert torch.equal(pf8.newton_schulz(g, steps=3.0), want)
    assert torch.equal(pf8.newton_schulz(g, steps=torch.tensor(3)), want)
    for bad in (dict(steps=2.5), dict(steps=float("inf")), dict(steps=float("nan")), dict(coefficients=())):
        with pytest.raises(ValueError):
            pf8.newton_schulz(g, **bad)
