"""Float64 reference of the training operators around the FP8 linear layer (numpy only).

block_norm / block_norm_grads: the norm after a block, its gate, the residual sum and the norm before
the next block. Formulas in include/pf8_train.h. Each also returns, per output, a "size": the same
expression with every term replaced by its magnitude, which the FP32 roundings of a kernel are
relative to.

newton_schulz: the odd polynomial iteration X <- a X + b (X X^T) X + c (X X^T)^2 X from G / (|G| + eps).
newton_schulz_operands: the same, with FP16 operands in the products as the library documents them.
"""
from __future__ import annotations

from types import SimpleNamespace

import numpy as np


def _parts(h, y, w_pre, w_post, gate, beta, alpha, eps, offset):
    p = SimpleNamespace()
    f = lambda a: None if a is None else np.asarray(a, dtype=np.float64)  # noqa: E731
    p.h, p.y = f(h), f(y)
    p.wn = None if w_pre is None else f(w_pre) + offset
    p.wp = None if w_post is None else f(w_post) + offset
    p.g = np.ones(1) if gate is None else f(gate)
    with np.errstate(all="ignore"):
        if p.y is not None:
            p.rho_y = 1.0 / np.sqrt(np.mean(p.y * p.y, axis=1, keepdims=True) + eps) if p.wp is not None else 1.0
            p.yn = p.y * p.rho_y
            p.u = p.yn if p.wp is None else p.yn * p.wp
            p.r = beta * p.h + alpha * p.g * p.u
            p.r_size = np.abs(beta * p.h) + np.abs(alpha * p.g * p.u)
        else:
            p.r, p.r_size = p.h, np.abs(p.h)
        p.rho = 1.0 / np.sqrt(np.mean(p.r * p.r, axis=1, keepdims=True) + eps)
        p.rn, p.rn_size = p.r * p.rho, p.r_size * p.rho
    return p


def block_norm(h, y=None, w_pre=None, w_post=None, gate=None, beta=1.0, alpha=1.0, eps=1e-6, offset=0.0):
    """(r, x, r_size, x_size); x is None without w_pre."""
    p = _parts(h, y, w_pre, w_post, gate, beta, alpha, eps, offset)
    if p.wn is None:
        return p.r, None, p.r_size, None
    with np.errstate(all="ignore"):
        return p.r, p.rn * p.wn, p.r_size, p.rn_size * np.abs(p.wn)


def block_norm_grads(dr, dx, h, y=None, w_pre=None, w_post=None, gate=None, beta=1.0, alpha=1.0, eps=1e-6,
                     offset=0.0):
    """(values, sizes): namespaces with dh, dy, dgate, dw_pre, dw_post (None where there is none)."""
    p = _parts(h, y, w_pre, w_post, gate, beta, alpha, eps, offset)
    v, s = SimpleNamespace(), SimpleNamespace()
    v.dy = v.dgate = v.dw_pre = v.dw_post = s.dy = s.dgate = s.dw_pre = s.dw_post = None
    mean = lambda a: np.mean(a, axis=1, keepdims=True)  # noqa: E731
    d = np.zeros_like(p.h) if dr is None else np.asarray(dr, dtype=np.float64)
    d_size = np.abs(d)
    if dx is not None:
        dx = np.asarray(dx, dtype=np.float64)
        t = dx * p.wn
        d = d + p.rho * (t - p.rn * mean(t * p.rn))
        d_size = d_size + p.rho * (np.abs(t) + p.rn_size * mean(np.abs(t) * p.rn_size))
        v.dw_pre, s.dw_pre = np.sum(dx * p.rn, axis=0), np.sum(np.abs(dx) * p.rn_size, axis=0)
    v.dh, s.dh = beta * d, np.abs(beta) * d_size
    if p.y is None:
        return v, s
    b, b_size = alpha * d, np.abs(alpha) * d_size
    if gate is not None:
        v.dgate, s.dgate = b * p.u, b_size * np.abs(p.u)
        if np.ndim(gate) == 1:
            v.dgate, s.dgate = v.dgate.sum(axis=0), s.dgate.sum(axis=0)
    du, du_size = b * p.g, b_size * np.abs(p.g)
    v.dy, s.dy = du, du_size
    if p.wp is not None:
        v.dw_post, s.dw_post = np.sum(du * p.yn, axis=0), np.sum(du_size * np.abs(p.yn), axis=0)
        t, t_size = du * p.wp, du_size * np.abs(p.wp)
        v.dy = p.rho_y * (t - p.yn * mean(t * p.yn))
        s.dy = p.rho_y * (t_size + np.abs(p.yn) * mean(t_size * np.abs(p.yn)))
    return v, s


def newton_schulz(g, coefficients, eps=1e-7):
    """Float64 iterates: `coefficients` holds one (a, b, c) per step; g [..., m, n]."""
    x = np.asarray(g, dtype=np.float64)
    x = x / (np.sqrt(np.sum(x * x, axis=(-2, -1), keepdims=True)) + eps)
    tall = x.shape[-2] > x.shape[-1]
    x = np.swapaxes(x, -2, -1) if tall else x
    for a, b, c in coefficients:
        gram = x @ np.swapaxes(x, -2, -1)
        x = a * x + (b * gram + c * (gram @ gram)) @ x
    return np.swapaxes(x, -2, -1) if tall else x


def newton_schulz_operands(g, coefficients, eps=1e-7, pairs=False):
    """newton_schulz with the FP16 roundings of a kernel's product operands, all else in float64.

    X is kept; its rounding enters the products (with `pairs`, in B X as value plus remainder). The
    diagonals of A = X X^T and of B = b A + c A A are kept, their other elements rounded, B's times a
    power of two that holds singular values up to 8 (half of what b s^2 + c s^4 can differ by). The
    diagonal of B multiplies X's rounding as the rest of B does, and X itself in the last step (with
    `pairs`, in every step).
    """
    f16 = lambda a, s: (a * s).astype(np.float16).astype(np.float64) / s  # noqa: E731
    x = np.asarray(g, dtype=np.float64)
    x = x / (np.sqrt(np.sum(x * x)) + eps)
    tall = x.shape[0] > x.shape[1]
    x = x.T if tall else x
    off = 1.0 - np.eye(x.shape[0])
    for step, (a, b, c) in enumerate(coefficients):
        xh = f16(x, 2.0 ** 12)
        xp = xh + (f16(x - xh, 2.0 ** 12) if pairs else 0.0)
        gram = xh @ xh.T
        d = np.diag(gram).copy()
        gram = f16(gram * off, 2.0 ** 10)
        square = gram @ gram
        poly = b * gram + c * (square + (d[:, None] + d[None, :]) * gram)
        diag = (b * d + c * (np.diag(square) + d * d))[:, None]
        own = x if pairs or step + 1 == len(coefficients) else xh
        scale = 2.0 ** min(9.0, np.floor(np.log2(60000.0 / (32.0 * abs(b) + 2048.0 * abs(c) + 1e-9))))
        x = a * x + diag * own + f16(poly * off, scale) @ xp
    return x.T if tall else x
