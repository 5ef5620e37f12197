"""Gradients of the head norm under autograd where only one of queries and keys has a weight.

dx is compared bit for bit with the functional form's. A weight's gradient is compared with the float64 oracle: its FP32 sum
takes another order where both tensors share a call. Under 2^10 roundings of 2^-24 each: 2^-14 of the sum of
magnitudes; a main gradient adds one more rounding (2^-24 of the result), a BF16 gradient half a step of BF16 (2^-8)."""
import pytest
import torch

import fp8_block_scaled_pf8_amd as pf8
from oracle import layer
from tests.gpu_helpers import DEV

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def _rand(shape, seed, scale=1.0, dtype=BF):
    return (torch.randn(shape, generator=torch.Generator().manual_seed(seed)) * scale).to(dtype).to(DEV)


def _np(t):
    return t.detach().cpu().double().numpy()


@pytest.mark.parametrize("main", [False, True])
@pytest.mark.parametrize("used", ["both", "weighted", "other"])
@pytest.mark.parametrize("weighted", [0, 1])
@pytest.mark.parametrize("rotated", [False, True])
def test_one_weight(weighted, used, main, rotated):
    """Without positions the tensor without a weight is a copy, and its gradient is its result's, whichever results
    gradients come from and wherever the weight's goes."""
    x = [_rand((2, 9, 4, 64), 1, 3.0).requires_grad_(), _rand((2, 9, 3, 64), 2, 3.0).requires_grad_()]
    w = (1 + _rand((64,), 3, 0.2)).requires_grad_()
    weights, mains = [None, None], [None, None]
    weights[weighted] = w
    if main:
        mains[weighted] = torch.ones(64, device=DEV)
    pos = torch.arange(9, device=DEV) if rotated else None
    freq = torch.linspace(1, 0.01, 32, device=DEV) if rotated else None
    y = pf8.fp8_qk_norm_rope(*x, pos, freq, *weights, main_grads=tuple(mains) if main else None)
    d = [_rand(t.shape, 5 + i) for i, t in enumerate(x)]
    at = {"both": [0, 1], "weighted": [weighted], "other": [1 - weighted]}[used]
    torch.autograd.backward([y[i] for i in at], [d[i] for i in at])
    for i in (0, 1):
        if i not in at:
            assert x[i].grad is None
            continue
        flat = lambda t: t.detach().reshape(18, -1, 64)  # noqa: E731
        if weights[i] is None and pos is None:
            assert torch.equal(y[i], x[i]) and torch.equal(x[i].grad, d[i])
            continue
        g = pf8.qk_norm_rope_backward(flat(d[i]), None, flat(x[i]), None, None if pos is None else pos.repeat(2), freq,
                                      None if weights[i] is None else w.detach())
        assert torch.equal(flat(x[i].grad), g.dq)
        if i == weighted:
            rot = {} if pos is None else dict(positions=_np(pos.repeat(2)), inv_freq=_np(freq))
            _, _, want, size = layer.head_norm_grads(_np(flat(d[i])), _np(flat(x[i])), _np(w), eps=1e-6, **rot)
            got = _np(mains[i]) - 1 if main else _np(w.grad)
            step = 2.0 ** -24 * (1 + abs(want)) if main else 2.0 ** -8 * abs(want)
            assert (abs(got - want) <= 2.0 ** -14 * size + step).all()
    if weighted not in at:
        assert w.grad is None and (not main or (mains[weighted] == 1).all())
    elif main:
        assert w.grad is None
