"""Scales of the product with its epilogue whose product lies past FP32's range, on the GPU.

Every scale is a power of two in [2^-127, 2^127]; what the sum over K and the result have to hold is the scaled sum, not the
product of two scales. The operands are chosen so that each sum is exact (equal products, few bits), so results are
compared for equality."""
import pytest
import torch

import fp8_block_scaled_pf8_amd as pf8
from tests.gpu_helpers import DEV

pytestmark = pytest.mark.gpu

LARGEST = 0x7E  # 448


def _operands(m, n, k, ex, ew, code=LARGEST):
    q = lambda rows: torch.full((rows, k), code, dtype=torch.uint8, device=DEV)  # noqa: E731
    s = lambda a, b, e: torch.ldexp(torch.ones((a, b), dtype=torch.float64), torch.tensor(e)).float().to(DEV)  # noqa: E731
    return q(m), s(k // 128, m, ex), q(n), s(-(-n // 128), k // 128, ew)


# 1 to 300 tokens: the kernel for few; 2100: tiles
@pytest.mark.parametrize("m", [1, 20, 100, 300, 2100])
@pytest.mark.parametrize("gated", [False, True])
def test_large_scales_of_zero_rows(m, gated):
    """Rows of zeros in W give the bias, however large the scales of their tile and of the token are."""
    n, k = 256, 384
    qx, sx, qw, sw = _operands(m, n, k, 100, 60)
    qw[1::2] = 0
    bias = (torch.arange(n, device=DEV) % 5 + 1).float()
    d, z = pf8.fprop_act(qx, sx, qw, sw, bias, "relu", gated=gated, save_z=True)
    want = bias.expand(m, n).clone()
    want[:, ::2] = float("inf")
    assert torch.equal(z.float(), want)
    assert torch.equal(d.float(), want[:, :n // 2] * want[:, n // 2:] if gated else want)


@pytest.mark.parametrize("m", [1, 20, 100, 300])
@pytest.mark.parametrize("ex,ew", [(-90, -60), (-60, -90), (-127, -23), (-23, -127)])
def test_small_scales(m, ex, ew):
    """448^2 * 128 = 49 * 2^19; times 2^-150 that is a normal value, though 2^-150 itself is under FP32's range."""
    d = pf8.fprop_act(*_operands(m, 200, 128, ex, ew))
    assert (d.double() == 49 * 2.0 ** (19 - 150)).all()


@pytest.mark.parametrize("m", [1, 20, 100, 300, 2100])
@pytest.mark.parametrize("ex,ew", [(127, -127), (-127, 127), (120, -110), (-126, 121)])
def test_scales_far_apart(m, ex, ew):
    """Products of codes 2 * 2 over 256 of K: 2^10 times both scales."""
    d = pf8.fprop_act(*_operands(m, 512, 256, ex, ew, code=0x40))
    assert (d.double() == 2.0 ** (10 + ex + ew)).all()
