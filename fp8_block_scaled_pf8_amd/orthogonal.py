"""Newton-Schulz orthogonalisation of a weight's gradient.

What an orthogonalising optimiser does with a weight matrix's momentum, or with the FP32
``main_grad`` that ``Fp8Linear`` accumulates: every singular value is drawn towards one while the
singular vectors stay, by a few odd polynomials of the matrix (include/pf8_train.h).
"""
from __future__ import annotations

import ctypes
from typing import Optional, Sequence

import torch

from . import _lib as L
from .norm import _call, _rows_meet

# Steep at zero (slope 3.4445), so that small singular values grow fast; after five steps values
# above 1e-2 of the norm lie between 0.7 and 1.2.
QUINTIC = (3.4445, -4.7750, 2.0315)


def newton_schulz(g: torch.Tensor, steps: int = 5, coefficients: Sequence = QUINTIC, eps: float = 1e-7,
                  out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """X <- a X + b (X X^T) X + c (X X^T)^2 X for ``steps`` steps, from X = g / (|g| + eps).

    g: bf16 or float32 [m, n], or a stack [count, m, n] of matrices, each with rows of any pitch.
    coefficients: (a, b, c), or one such triple per step. Returns bf16 of g's shape (``out`` if given).
    An empty stack gives an empty result.
    """
    if not isinstance(g, torch.Tensor) or g.dim() not in (2, 3):
        raise ValueError("g must be a matrix [m, n] or a stack of matrices [count, m, n]")
    if g.dtype not in (torch.bfloat16, torch.float32):
        raise TypeError(f"g must be torch.bfloat16 or torch.float32, got {g.dtype}")
    if not g.is_cuda:
        raise ValueError("g must be on a HIP device")
    m, n = g.shape[-2:]
    batch = g.shape[0] if g.dim() == 3 else 1
    if m < 1 or n < 1 or min(m, n) > L.PF8_NS_MAX_SHORT or max(m, n) > L.PF8_NS_MAX_LONG:
        raise ValueError(f"newton_schulz takes matrices with sides from 1 to {L.PF8_NS_MAX_SHORT} (the shorter) and "
                         f"{L.PF8_NS_MAX_LONG} (the longer), got {m} x {n}")
    if batch > L.PF8_NS_MAX_BATCH:
        raise ValueError(f"newton_schulz takes up to {L.PF8_NS_MAX_BATCH} matrices at once, got {batch}")
    if isinstance(steps, bool) or not 1 <= steps <= L.PF8_NS_MAX_STEPS or int(steps) != steps:
        raise ValueError(f"steps must be 1 to {L.PF8_NS_MAX_STEPS}, got {steps}")
    steps = int(steps)
    if len(coefficients) == 0:
        raise ValueError("coefficients must not be empty")
    triples = [tuple(coefficients)] * steps if not hasattr(coefficients[0], "__len__") else [tuple(c) for c in coefficients]
    if len(triples) != steps or any(len(c) != 3 for c in triples):
        raise ValueError(f"coefficients must be one (a, b, c) or {steps} of them")
    if out is None:
        out = torch.empty(g.shape, dtype=torch.bfloat16, device=g.device)
    elif out.dtype != torch.bfloat16 or out.shape != g.shape or out.device != g.device:
        raise ValueError(f"out must be torch.bfloat16 of shape {tuple(g.shape)} on {g.device}")
    if batch == 0:
        return out
    layouts = []
    for t, name in ((g, "g"), (out, "out")):
        ld = t.stride(-2) if m > 1 else n
        stride = t.stride(0) if batch > 1 else 0
        if (n > 1 and t.stride(-1) != 1) or ld < n or (batch > 1 and stride < (m - 1) * ld + n):
            raise ValueError(f"{name} must have contiguous rows, and neither its rows nor its matrices may overlap")
        first, size = t.data_ptr(), t.element_size()
        # one pitch for all rows of a stack, or all its matrices as single pieces
        whole = batch > 1 and m > 1 and stride % ld
        width = (m - 1) * ld + n if whole else n
        pitch = stride if whole or m == 1 else ld
        layouts.append((ld, stride, (first, first + ((batch - 1) * stride + (m - 1) * ld + n) * size, width * size, pitch * size)))
    (ldg, sg, at_g), (ldo, so, at_o) = layouts
    if _rows_meet(at_g, at_o):
        raise ValueError("out overlaps g")
    coef = (ctypes.c_float * (3 * steps))(*(v for c in triples for v in c))
    size = L.pf8_newton_schulz_workspace(batch, m, n)
    ws = torch.empty(size, dtype=torch.uint8, device=g.device)
    _call(L.pf8_newton_schulz, g.device, batch, m, n, at_g[0], ldg, sg, L.PF8_F32 if g.dtype == torch.float32 else L.PF8_BF16,
          steps, coef, eps, at_o[0], ldo, so, ws.data_ptr(), size)
    return out
