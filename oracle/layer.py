"""Float64 reference of a decoder layer's steps around its FP8 products (numpy only).

head_norm / head_norm_grads: the norm of every head and the rotation of its first pairs by positions.
act / act_grads: activations, gated or not, and their backward pass. Formulas in include/pf8_layer.h.
Each also returns a "size": the same expression with every term replaced by its magnitude, which the FP32
roundings of a kernel are relative to.
"""
from __future__ import annotations

import math

import numpy as np


def pair_axes(pairs, sections=None, order="blocked"):
    """The position axis of each rotated pair."""
    axis = np.zeros(pairs, dtype=np.int64)
    if sections is None:
        return axis
    if order == "blocked":
        return np.repeat(np.arange(len(sections)), sections)
    for a in range(1, len(sections)):
        axis[a + len(sections) * np.arange(sections[a])] = a
    return axis


def _rotation(positions, inv_freq, sections, order, scale, back):
    """(cosines, sines) [tokens, 1, pairs]; `back`: of the opposite angles."""
    freq = np.asarray(inv_freq, dtype=np.float64)
    pos = np.asarray(positions, dtype=np.float64)
    pos = pos.reshape(1, -1) if pos.ndim == 1 else pos
    angle = pos[pair_axes(len(freq), sections, order)].T * freq
    return scale * np.cos(angle)[:, None], (-scale if back else scale) * np.sin(angle)[:, None]


def _turn(x, cs, interleaved, size=False):
    if cs is None:
        return x
    c, s = np.abs(cs[0]) if size else cs[0], np.abs(cs[1]) if size else cs[1]
    pairs = c.shape[-1]
    a_at = slice(0, 2 * pairs, 2) if interleaved else slice(0, pairs)
    b_at = slice(1, 2 * pairs, 2) if interleaved else slice(pairs, 2 * pairs)
    y = x.copy()
    y[..., a_at] = x[..., a_at] * c + (x[..., b_at] * s if size else -x[..., b_at] * s)
    y[..., b_at] = x[..., a_at] * s + x[..., b_at] * c
    return y


def head_norm(x, w=None, positions=None, inv_freq=None, sections=None, order="blocked", interleaved=False, scale=1.0,
              eps=1e-6, offset=0.0):
    """(values, sizes) of x [tokens, heads, head_dim]."""
    x = np.asarray(x, dtype=np.float64)
    cs = None if positions is None else _rotation(positions, inv_freq, sections, order, scale, False)
    with np.errstate(all="ignore"):
        n = x
        if w is not None:
            n = x / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps) * (np.asarray(w, dtype=np.float64) + offset)
        return _turn(n, cs, interleaved), _turn(np.abs(n), cs, interleaved, True)


def head_norm_grads(d, x=None, w=None, positions=None, inv_freq=None, sections=None, order="blocked", interleaved=False,
                    scale=1.0, eps=1e-6, offset=0.0):
    """(dx, its size, dw or None, its size or None) from d, the gradient of head_norm's values."""
    d = np.asarray(d, dtype=np.float64)
    cs = None if positions is None else _rotation(positions, inv_freq, sections, order, scale, True)
    with np.errstate(all="ignore"):
        size = _turn(np.abs(d), cs, interleaved, True)
        d = _turn(d, cs, interleaved)
        if w is None:
            return d, size, None, None
        x, w = np.asarray(x, dtype=np.float64), np.asarray(w, dtype=np.float64) + offset
        rho = 1.0 / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps)
        y, t = x * rho, d * w
        dx = rho * (t - y * np.mean(t * y, axis=-1, keepdims=True))
        ts = size * np.abs(w)
        dxs = rho * (ts + np.abs(y) * np.mean(ts * np.abs(y), axis=-1, keepdims=True))
        return dx, dxs, np.sum(d * y, axis=(0, 1)), np.sum(size * np.abs(y), axis=(0, 1))


_erf = np.vectorize(math.erf, otypes=[np.float64])


def act(z, name):
    """act(z), and act'(z)."""
    z = np.asarray(z, dtype=np.float64)
    with np.errstate(all="ignore"):
        if name == "relu":
            return np.maximum(z, 0.0), (z > 0).astype(np.float64)
        if name == "relu2":
            return np.maximum(z, 0.0) ** 2, 2 * np.maximum(z, 0.0)
        if name == "silu":
            s = 1 / (1 + np.exp(-z))
            return z * s, s + z * s * (1 - s)
        if name == "gelu":
            p = 0.5 * (1 + _erf(z / math.sqrt(2)))
            return z * p, p + z * np.exp(-z * z / 2) / math.sqrt(2 * math.pi)
        if name == "gelu_tanh":
            c = math.sqrt(2 / math.pi)
            t = np.tanh(c * (z + 0.044715 * z ** 3))
            return 0.5 * z * (1 + t), 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)
    return z, np.ones_like(z)


def act_out(z, name, gated):
    """d from z: act(z), or act of the first half of the columns times the second."""
    if not gated:
        return act(z, name)[0]
    n = z.shape[1] // 2
    return act(z[:, :n], name)[0] * np.asarray(z[:, n:], dtype=np.float64)


def act_grads(dd, z, name, gated):
    """dz."""
    dd = np.asarray(dd, dtype=np.float64)
    if not gated:
        return dd * (1.0 if name is None else act(z, name)[1])
    z = np.asarray(z, dtype=np.float64)
    n = dd.shape[1]
    value, slope = act(z[:, :n], name)
    return np.concatenate([dd * z[:, n:] * slope, dd * value], axis=1)
