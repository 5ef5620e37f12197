"""A layer that is first used without gradients, then trained."""
import pytest
import torch

import fp8_block_scaled_pf8_amd as pf8
from tests.gpu_helpers import DEV

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def _rand(shape, seed, scale=1.0, dtype=BF):
    return (torch.randn(shape, generator=torch.Generator().manual_seed(seed)) * scale).to(dtype).to(DEV)


@pytest.mark.parametrize("mode", [torch.no_grad, torch.inference_mode])
@pytest.mark.parametrize("first", ["infer", "call"])
@pytest.mark.parametrize("kw", [dict(), dict(bias=True, activation="silu", gated=True)])
def test_trained_after(mode, first, kw):
    """The weight's codes that a pass without gradients made serve the training passes after it."""
    torch.manual_seed(1)
    lin, other = pf8.Fp8Linear(256, 512, device=DEV, **kw), pf8.Fp8Linear(256, 512, device=DEV, **kw)
    with torch.no_grad():
        other.weight.copy_(lin.weight)
    x = _rand((128, 256), 1).requires_grad_()
    with mode():
        y = lin.infer(x[:5]) if first == "infer" else lin(x)
    assert y.shape[0] == (5 if first == "infer" else 128)
    codes = lin.weight_codes()
    grads = []
    for m in (lin, other):
        d = m(x)
        d.backward(_rand(d.shape, 2, 1e-2))
        grads.append([x.grad, m.weight.grad])
        x.grad = None
    assert lin.weight_codes() is codes
    assert all(torch.equal(a, b) for a, b in zip(*grads))


@pytest.mark.parametrize("kw", [dict(), dict(bias=True, activation="silu", gated=True)])
def test_first_used_in_a_capture(kw):
    """Codes that a graph makes are the graph's: an eager pass makes its own, before a replay as after one."""
    torch.manual_seed(1)
    lin, other = pf8.Fp8Linear(256, 512, device=DEV, **kw), pf8.Fp8Linear(256, 512, device=DEV, **kw)
    with torch.no_grad():
        other.weight.copy_(lin.weight)
    x = _rand((3, 256), 1)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = lin.infer(x)
    for i in range(3):
        e = _rand((5, 256), 10 + i)
        assert torch.equal(lin.infer(e), other.infer(e))
        x.copy_(_rand((3, 256), 20 + i))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, other.infer(x))
        if i == 1:  # the graph follows the weight
            with torch.no_grad():
                lin.weight.mul_(2), other.weight.mul_(2)


def test_graph_keeps_the_codes_it_was_captured_with():
    """Codes made before a capture are baked into its graph: their memory stays theirs when new ones replace them."""
    torch.manual_seed(1)
    lin = pf8.Fp8Linear(256, 512, device=DEV, bias=True, activation="silu", gated=True)
    x = _rand((3, 256), 1)
    lin.infer(x)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = lin.infer(x)
    old = pf8.Fp8Linear(256, 512, device=DEV, bias=True, activation="silu", gated=True, weight=lin.weight.detach().clone())
    held = [t.data_ptr() for t in lin.weight_codes()]
    for i in range(3):
        with torch.no_grad():
            lin.weight.add_(1)
        if i == 1:
            lin.invalidate_weight_codes()
        new = lin.weight_codes()
        filled = [torch.full_like(t, 3) for t in new]  # would take the old codes' place
        assert not {t.data_ptr() for t in (*new, *filled)} & set(held)
        x.copy_(_rand((3, 256), 20 + i))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, old.infer(x))
