"""The layer's steps on tensors of more than 2^31 values or bytes: the last rows of a large call are those of a call on them
alone, bit for bit (sums are of whole numbers or of one value, so that no order matters)."""
import pytest
import torch

import fp8_block_scaled_pf8_amd as pf8
from tests.gpu_helpers import DEV

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def _fill(shape, seed):
    """Cheap bf16 values that differ from row to row."""
    row = torch.randn(shape[1:], generator=torch.Generator().manual_seed(seed)).to(BF).to(DEV)
    t = row.expand(shape).contiguous()
    t[:, ..., 0] = torch.arange(shape[0], device=DEV).remainder(251).to(BF).reshape(-1, *[1] * (len(shape) - 2)) / 64
    return t


def test_head_norms():
    tokens, heads, dim, last = (2 ** 31) // (16 * 128) + 1000, 16, 128, 4096
    q, w = _fill((tokens, heads, dim), 1), _fill((2, dim), 2)[0]
    assert q.numel() > 2 ** 31
    pos = torch.arange(tokens, device=DEV)
    rot = dict(positions=pos, inv_freq=torch.linspace(1, 1e-4, dim // 2, device=DEV), w_q=w)
    end = {**rot, "positions": pos[-last:]}
    got = pf8.qk_norm_rope(q, **rot)[0]
    assert torch.equal(got[-last:], pf8.qk_norm_rope(q[-last:].clone(), **end)[0])
    assert torch.equal(got[:last], pf8.qk_norm_rope(q[:last].clone(), **{**rot, "positions": pos[:last]})[0])
    del got
    d = torch.zeros_like(q)
    d[-1, -1] = _fill((2, dim), 3)[0]
    g = pf8.qk_norm_rope_backward(d, None, q, **rot)
    one = pf8.qk_norm_rope_backward(d[-last:].clone(), None, q[-last:].clone(), **end)
    assert torch.equal(g.dq[-last:], one.dq) and torch.equal(g.dw_q, one.dw_q) and one.dw_q.any()
    assert not g.dq[:-1].any()


def test_activation_backward():
    rows, cols, last = 2 ** 31 // 8192 + 128, 8192, 128
    assert rows % 128 == 0
    dd, z = torch.zeros((rows, cols), dtype=BF, device=DEV), _fill((rows, 2 * cols), 2)
    dd[-1] = _fill((2, cols), 3)[0]  # one row: its sums are itself
    g = pf8.act_backward(dd, z, "silu", gated=True, bias_grad=True)
    one = pf8.act_backward(dd[-last:].clone(), z[-last:].clone(), "silu", gated=True, bias_grad=True)
    assert torch.equal(g.dz[-last:], one.dz) and torch.equal(g.dbias, one.dbias) and one.dz.any()
    assert not g.dz[:-1].any()
    del g
    g = pf8.act_backward_quant(dd, z, "silu", gated=True, bias_grad=True)
    q, s, qt, st = pf8.quant_act_dual(one.dz)
    assert torch.equal(g.q[-last:], q) and torch.equal(g.s[:, -last:], s) and torch.equal(g.dbias, one.dbias)
    assert torch.equal(g.qt[:, -last:], qt) and torch.equal(g.st[-1:], st)


def _whole(shape, seed):
    """Codes of -2 .. 2: sums of their products are exact."""
    v = torch.tensor([0x00, 0x38, 0x40, 0xB8, 0xC0], dtype=torch.uint8)
    return v[torch.randint(0, 5, shape, generator=torch.Generator().manual_seed(seed))].to(DEV)


@pytest.mark.parametrize("gated", [False, True])
def test_product_of_many_tokens(gated):
    n, k, last = 2048, 128, 300
    m = 2 ** 31 // (n // 2 if gated else n) + 1001
    cols = n // 2 if gated else n
    qx = _whole((4099, k), 1).repeat(m // 4099 + 1, 1)[:m].contiguous()
    qw, bias = _whole((n, k), 2), torch.arange(n, device=DEV, dtype=torch.float32) % 7
    sx, sw = torch.ones((1, m), device=DEV), torch.ones((n // 128, 1), device=DEV)
    act = dict(bias=bias, activation="relu" if gated else None, gated=gated)
    res = _fill((m, cols), 4)
    d = pf8.fprop_act(qx, sx, qw, sw, residual=res, **act)
    assert d.numel() > 2 ** 31
    want, z = pf8.fprop_act(qx[-last:].contiguous(), sx[:, -last:].contiguous(), qw, sw, residual=res[-last:].clone(), save_z=True,
                            **act)
    assert torch.equal(d[-last:], want)
    del d, res
    m = min(m, 2 ** 31 // n + 1001)
    qx, sx = qx[-m:].contiguous(), sx[:, -m:].contiguous()
    assert torch.equal(pf8.fprop_act(qx, sx, qw, sw, save_z=True, **act)[1][-last:], z)


def test_product_of_one_token_and_many_weights():
    n, k = 2 ** 31 // 1024 + 1000, 1024
    qx, qw = _whole((1, k), 1), _whole((4099, k), 2).repeat(n // 4099 + 1, 1)[:n].contiguous()
    assert qw.numel() > 2 ** 31
    sx, sw = torch.ones((k // 128, 1), device=DEV), torch.ones((-(-n // 128), k // 128), device=DEV)
    bias = (torch.arange(n, device=DEV) % 7).to(BF)
    d = pf8.fprop_act(qx, sx, qw, sw, bias)
    cut = n - n % 128 - 256
    want = pf8.fprop_act(qx, sx, qw[cut:].contiguous(), sw[cut // 128:].contiguous(), bias[cut:].clone())
    assert torch.equal(d[:, cut:], want) and want.any()


def test_rows_wider_than_a_tile_addresses():
    """A tile's 256 rows are addressed by 32 bits: wider results are refused."""
    n, k = 2 ** 31 // 128 + 1000, 128
    qw = torch.zeros((n, k), dtype=torch.uint8, device=DEV)
    with pytest.raises(RuntimeError, match="pitch too large"):
        pf8.fprop_act(qw[:1], torch.ones((1, 1), device=DEV), qw, torch.ones((-(-n // 128), 1), device=DEV))
