"""The activation's backward pass at the most columns that its entry takes."""
import pytest
import torch

import fp8_block_scaled_pf8_amd as pf8
from tests.gpu_helpers import DEV

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


@pytest.mark.parametrize("cols", [2 ** 31 - 1, 2 ** 31 - 8])
@pytest.mark.parametrize("bias_grad", [False, True])
def test_widest_rows(cols, bias_grad):
    """relu keeps or drops each gradient, and one row is its own column sums: equal value by value."""
    part = 1 << 27
    dd, z = (torch.empty((1, cols), dtype=BF, device=DEV) for _ in range(2))
    for i, t in enumerate((dd, z)):
        some = torch.randn(100003, generator=torch.Generator().manual_seed(i)).to(BF).to(DEV)
        some = some.repeat(part // 100003 + 1)[:part]
        for a in range(0, cols, part):
            t[0, a:a + part] = some[:min(part, cols - a)]
    g = pf8.act_backward(dd, z, "relu", bias_grad=bias_grad)
    for a in range(0, cols, part):
        want = torch.where(z[0, a:a + part] > 0, dd[0, a:a + part], 0)
        assert torch.equal(g.dz[0, a:a + part], want)
        assert not bias_grad or torch.equal(g.dbias[a:a + part], want.float())
