"""Calls on tensors of a device that is not the current one make it current around the launch.

One GPU is enough: what counts as the current device is replaced by another number, and every entry into a device is
recorded. (On the current device no entry is made: it costs as much as half a launch.)"""
import pytest
import torch

import fp8_block_scaled_pf8_amd as pf8
from fp8_block_scaled_pf8_amd import ops
from tests.gpu_helpers import DEV

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def _rand(shape, seed, scale=1.0):
    return (torch.randn(shape, generator=torch.Generator().manual_seed(seed)) * scale).to(BF).to(DEV)


def _calls():
    x, w, dd = _rand((128, 256), 1), _rand((512, 256), 2, 0.05), _rand((128, 256), 3, 1e-2)
    codes, weights = pf8.quant_act_dual(x), pf8.quant_w_128x128(w)
    qx, sx, qxt, sxt = codes
    qw, qwt, sw = weights
    z = _rand((128, 512), 4)
    q, norm, pos = _rand((5, 3, 64), 5), 1 + _rand((64,), 6, 0.2), torch.arange(5, device=DEV)
    freq = torch.linspace(1, 0.1, 32, device=DEV)
    lin = pf8.Fp8Linear(256, 512, device=DEV, weight=w, bias=True, activation="silu", gated=True)
    one = lambda t: (t,)  # noqa: E731
    return {
        "quant_act_1x128": lambda: pf8.quant_act_1x128(x),
        "quant_act_dual": lambda: pf8.quant_act_dual(x),
        "quant_w_128x128": lambda: pf8.quant_w_128x128(w),
        "fprop": lambda: one(pf8.fprop(qx, sx, qw, sw)),
        "wgrad_f32": lambda: one(pf8.wgrad_f32(qxt, sxt, qxt, sxt)),
        "gemm_bf16": lambda: one(pf8.gemm_bf16(x, w)),
        "fprop_act": lambda: pf8.fprop_act(qx, sx, qw, sw, activation="silu", gated=True, save_z=True),
        "act_backward": lambda: one(pf8.act_backward(dd, z, "silu", True).dz),
        "act_backward_quant": lambda: pf8.act_backward_quant(dd, z, "silu", True)[:4],
        "qk_norm_rope": lambda: one(pf8.qk_norm_rope(q, None, pos, freq, norm)[0]),
        "qk_norm_rope_backward": lambda: one(pf8.qk_norm_rope_backward(q, None, q, None, pos, freq, norm).dq),
        "block_norm": lambda: one(pf8.block_norm(x, w_pre=1 + _rand((256,), 7))[1]),
        "newton_schulz": lambda: one(pf8.newton_schulz(w)),
        "fp8_linear_act": lambda: one(pf8.fp8_linear_act(x, w, None, "silu", True).detach()),
        "infer": lambda: one(lin.infer(x)),
    }


NAMES = ["quant_act_1x128", "quant_act_dual", "quant_w_128x128", "fprop", "wgrad_f32", "gemm_bf16", "fprop_act", "act_backward",
         "act_backward_quant", "qk_norm_rope", "qk_norm_rope_backward", "block_norm", "newton_schulz", "fp8_linear_act", "infer"]


@pytest.mark.parametrize("name", NAMES)
def test_the_tensors_device_is_entered(name, monkeypatch):
    calls = _calls()
    assert set(calls) == set(NAMES)
    call = calls[name]
    want = [t.clone() for t in call()]
    entered, device = [], torch.cuda.device

    class Recorded(device):
        def __init__(self, d):
            entered.append(torch.device(d) if not isinstance(d, int) else torch.device("cuda", d))
            super().__init__(d)

    monkeypatch.setattr(torch.cuda, "device", Recorded)
    call()
    assert not entered
    monkeypatch.setattr(ops, "_current_device", lambda: 5)
    got = call()
    assert entered and all(d == torch.device(DEV) for d in entered)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
