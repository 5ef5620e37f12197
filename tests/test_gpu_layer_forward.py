"""What the FP8 linear layer's forward makes where no gradient is asked for: the result, and nothing for a backward pass."""
import pytest
import torch

import fp8_block_scaled_pf8_amd as pf8
from fp8_block_scaled_pf8_amd import epilogue, ops
from tests.gpu_helpers import DEV

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def _rand(shape, seed, scale=1.0, dtype=BF):
    return (torch.randn(shape, generator=torch.Generator().manual_seed(seed)) * scale).to(dtype).to(DEV)


@pytest.fixture
def made(monkeypatch):
    """How often transposed codes of X and the value before the activation were made."""
    counts = {"dual": 0, "z": 0}
    dual, fprop = ops.quant_act_dual, epilogue.fprop_act

    def counted_dual(x):
        counts["dual"] += 1
        return dual(x)

    def counted_fprop(*args, save_z=False, **kw):
        counts["z"] += bool(save_z)
        return fprop(*args, save_z=save_z, **kw)

    monkeypatch.setattr(ops, "quant_act_dual", counted_dual)
    monkeypatch.setattr(epilogue, "fprop_act", counted_fprop)
    return counts


@pytest.mark.parametrize("mode", [torch.no_grad, torch.inference_mode])
@pytest.mark.parametrize("activation,gated", [("silu", True), ("gelu", False), (None, False)])
def test_without_gradients(made, mode, activation, gated):
    lin = pf8.Fp8Linear(256, 512, device=DEV, bias=True, activation=activation, gated=gated)
    x, r = _rand((2, 128, 256), 1), _rand((2, 128, 256 if gated else 512), 2)
    trained = lin(x, r)
    assert trained.requires_grad and made == {"dual": 1, "z": int(activation is not None)}
    with mode():
        got = lin(x, r)
    assert made == {"dual": 1, "z": int(activation is not None)}
    assert torch.equal(got, trained) and not got.requires_grad
    for p in lin.parameters():
        p.requires_grad_(False)
    assert torch.equal(lin(x, r), trained) and made["dual"] == 1
    assert lin(x[:0], r[:0]).shape == (0, 128, r.shape[-1])


def test_a_gradient_of_the_residual_alone(made):
    x, w, r = _rand((128, 256), 1), _rand((512, 256), 2, 0.05), _rand((128, 256), 3).requires_grad_()
    dd = _rand((128, 256), 4)
    d = pf8.fp8_linear_act(x, w, None, "silu", True, r)
    d.backward(dd)
    assert torch.equal(r.grad, dd) and made == {"dual": 0, "z": 0}


def test_a_checkpointed_layer(made):
    """A reentrant checkpoint's first pass runs without gradients; its second one makes what the backward pass needs."""
    from torch.utils.checkpoint import checkpoint

    lin = pf8.Fp8Linear(256, 512, device=DEV, bias=True, activation="silu", gated=True)
    x, dd = _rand((128, 256), 1).requires_grad_(), _rand((128, 256), 4, 1e-2)
    lin(x).backward(dd)
    want = [x.grad.clone(), lin.weight.grad.clone(), lin.bias.grad.clone()]
    x.grad = lin.weight.grad = lin.bias.grad = None
    before = dict(made)
    y = checkpoint(lin, x, use_reentrant=True)
    assert made == before
    y.backward(dd)
    assert made["dual"] == before["dual"] + 1 and made["z"] == before["z"] + 1
    assert all(torch.equal(a, b) for a, b in zip(want, (x.grad, lin.weight.grad, lin.bias.grad)))
