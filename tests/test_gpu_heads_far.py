"""Angles of far positions against exact fractions of a turn.

Turns are position * fl(inv_freq * fl(1 / 2 pi)) in float64: three roundings, of the constant (2^-53.3 of it), of its product
and of the position's, together under 2^-51.4 of the angle; taking off whole turns is exact. The fraction in FP32 and the
sine add under 2^-21.9 (derived with the tests of many tokens; 2^-21 allowed). So an angle phi is off by 2^-51.4 |phi| +
2^-21, and a value by that times |a| + |b|, beside its FP32 roundings (2^-17 of the size) and its rounding to bf16 (2^-8)."""
import fractions

import numpy as np
import pytest
import torch

import fp8_block_scaled_pf8_amd as pf8
from tests.gpu_helpers import DEV

pytestmark = pytest.mark.gpu

TWO_PI = fractions.Fraction("6.28318530717958647692528676655900576839433879875021164194988918461563281257")
POSITIONS = [0, 1, -1, 100003, 2 ** 31 + 5, -(2 ** 33) - 1, 2 ** 40 + 1, 2 ** 44 - 1, 2 ** 48 + 3, -(2 ** 50) - 3, 2 ** 52 - 1]


@pytest.mark.parametrize("dtype", [torch.float32, torch.float64])
@pytest.mark.parametrize("powers", [True, False])
@pytest.mark.parametrize("back", [False, True])
def test_far_positions(dtype, powers, back):
    n, pairs = len(POSITIONS), 48
    freq = [2.0 ** -i for i in range(pairs)] if powers else [float(np.float32(1e12) ** (-i / pairs)) for i in range(pairs)]
    freq = torch.tensor(freq, dtype=dtype, device=DEV)
    x = torch.randn((n, 3, 2 * pairs), generator=torch.Generator().manual_seed(1)).bfloat16().to(DEV)
    pos = torch.tensor(POSITIONS, device=DEV)
    got = pf8.qk_norm_rope_backward(x, None, None, None, pos, freq).dq if back else pf8.qk_norm_rope(x, None, pos, freq)[0]
    exact = [[fractions.Fraction(p) * fractions.Fraction(f) for f in freq.tolist()] for p in POSITIONS]
    turns = np.array([[float(e / TWO_PI % 1) for e in row] for row in exact])
    c, s = np.cos(2 * np.pi * turns)[:, None], np.sin(2 * np.pi * turns)[:, None] * (-1 if back else 1)
    a, b = (t.cpu().double().numpy() for t in (x[..., :pairs], x[..., pairs:]))
    want = np.concatenate([a * c - b * s, a * s + b * c], -1)
    size = np.concatenate([abs(a * c) + abs(b * s), abs(a * s) + abs(b * c)], -1)
    off = np.array([[abs(float(e)) for e in row] for row in exact])[:, None] * 2.0 ** -51.4 + 2.0 ** -21
    loose = np.concatenate([off * (abs(a) + abs(b))] * 2, -1)
    # (an angle that is off by over a turn's part says nothing: these count from 2^-4 radians down, at every position)
    known = np.concatenate([np.broadcast_to(off, a.shape)] * 2, -1) < 2.0 ** -4
    assert known.any((1, 2)).all()
    tol = 2.0 ** -8 * abs(want) + 2.0 ** -17 * size + loose
    assert (abs(got.cpu().double().numpy() - want) <= tol)[known].all()
