"""The head norm's kernels for many tokens against the float64 oracle.

Where there is work enough a group of lanes takes four heads of a token forward, two backward (from tokens * heads * lanes
of 327680 and 262144 on). Every size here has twice that. Numbers of heads that four and two do not divide, every number
of lanes and layout of pairs, one axis and several.

Tolerances: as for few tokens 2^-8 of the value for its rounding to bf16 and 2^-17 of the "size" (the same expression of
magnitudes) for the FP32 roundings before it; a lane sums few heads, a workgroup its groups and the last kernel 24 rows for
each of 32 threads, under the 2^10 roundings that 2^-14 of a weight gradient's size allows. A sine's or cosine's own error is
absolute, not relative to it: the fraction of a turn, up to 1/2 in FP32, is off by half a step, 2^-26 turns or
2 pi 2^-26 < 2^-23 radians, and the instructions are off by up to 2^-22.9 (measured at each multiple of 2^-25 of a turn). Among
millions of values some a cos - b sin nearly vanishes with a and the sine both small: there b times the sine's error
counts, whatever the size is. 2^-23 + 2^-22.9 < 2^-21.9; allowed: 2^-21 (|a| + |b|), taken through the norm's gradient where
there is one."""
import numpy as np
import pytest
import torch

import fp8_block_scaled_pf8_amd as pf8
from oracle import layer
from tests.gpu_helpers import DEV
from tests.test_gpu_heads import _freq, _np, _oracle, _rand

pytestmark = pytest.mark.gpu

# head_dim, pairs, neighbours, query and key heads, lanes of a head
SIZES = [
    (64, 32, False, 5, 3, 4), (128, 64, False, 7, 1, 8), (72, 36, False, 6, 5, 8), (256, 128, False, 3, 2, 16),
    (192, 32, False, 9, 2, 16), (512, 256, False, 1, 2, 32), (40, 10, True, 5, 3, 4), (128, 64, True, 7, 1, 8),
    (192, 80, True, 3, 6, 16), (512, 100, True, 2, 1, 32), (50, 20, False, 5, 2, 64), (33, 16, True, 6, 1, 64),
    (128, 64, False, 16, 8, 8),
]


def _close(got, ref, size, loose, what):
    got, near = _np(got), 2.0 ** -8 * abs(ref) + 2.0 ** -17 * size if got.dtype == torch.bfloat16 else 2.0 ** -14 * size
    assert got.shape == ref.shape, what
    tol = near + 2.0 ** -21 * loose + 2.0 ** -134
    off = abs(got - ref)
    assert (off <= tol).all(), f"{what}: {np.max(off / tol)} of the tolerance"


def _check(q, k, w_q, w_k, rot, **kw):
    o = _oracle(rot, kw)
    oq, ok = pf8.qk_norm_rope(q, k, w_q=w_q, w_k=w_k, **rot, **kw)
    dq, dk = _rand(q.shape, 9), None if k is None else _rand(k.shape, 10)
    g = pf8.qk_norm_rope_backward(dq, dk, q, k, w_q=w_q, w_k=w_k, **rot, **kw)
    ones = np.full((1, 1, len(o.get("inv_freq", ()))), o.get("scale", 1.0))

    def sines(v):
        """|a| + |b| in the places of both."""
        return layer._turn(abs(v), (ones, ones), o.get("interleaved", False), True) if "positions" in o else 0 * v

    for n, x, w, got, d, dx, dw in (("q", q, w_q, oq, dq, g.dq, g.dw_q), ("k", k, w_k, ok, dk, g.dk, g.dw_k)):
        if x is None:
            assert got is None and dx is None and dw is None
            continue
        x, w, d = _np(x), _np(w), _np(d)
        ref, size = layer.head_norm(x, w, **o)
        plain = layer.head_norm(x, w, eps=o["eps"], offset=o["offset"])[0]
        _close(got, ref, size, sines(plain), n)
        rx, sx, rw, sw = layer.head_norm_grads(d, x, w, **o)
        loose = sines(d)
        assert (dw is None) == (w is None)
        if w is not None:
            rho = 1 / np.sqrt(np.mean(x * x, -1, keepdims=True) + o["eps"])
            y, t = abs(x * rho), loose * abs(w + o["offset"])
            _close(dw, rw, sw, np.sum(loose * y, (0, 1)), "dw_" + n)
            loose = rho * (t + y * np.mean(t * y, -1, keepdims=True))
        _close(dx, rx, sx, loose, "d" + n)


@pytest.mark.parametrize("axes", [1, 3])
@pytest.mark.parametrize("dim,pairs,interleaved,hq,hk,lanes", SIZES)
def test_sizes(dim, pairs, interleaved, hq, hk, lanes, axes):
    tokens = 2 * 327680 // (lanes * (hq + hk)) + 3
    q, k = _rand((tokens, hq, dim), 1, 3.0), _rand((tokens, hk, dim), 2, 3.0)
    pos = torch.arange(tokens, device=DEV) * 37 % 100003
    rot = dict(positions=pos, inv_freq=_freq(pairs), interleaved=interleaved)
    if axes == 3:
        rest = pairs - 2 * (pairs // 3)
        rot.update(positions=torch.stack([pos, pos // 7, pos % 61]), sections=(rest, pairs // 3, pairs // 3),
                   section_order="cycled" if interleaved else "blocked")
    _check(q, k, 1 + _rand((dim,), 3, 0.2), 1 + _rand((dim,), 4, 0.2), rot)


@pytest.mark.parametrize("norm", ["q", "k", "none"])
def test_one_norm_or_none(norm):
    q, k = _rand((10243, 7, 128), 1, 3.0), _rand((10243, 1, 128), 2, 3.0)
    w = 1 + _rand((128,), 3, 0.2, torch.float32)
    _check(q, k, w if norm == "q" else None, w if norm == "k" else None,
           dict(positions=torch.arange(10243, device=DEV, dtype=torch.int32), inv_freq=_freq(64)))


def test_queries_alone_and_norms_alone():
    q, w = _rand((14001, 6, 128), 1, 3.0), 1 + _rand((128,), 3, 0.2)
    _check(q, None, w, None, dict(positions=torch.arange(14001, device=DEV), inv_freq=_freq(64)))
    _check(q, _rand((14001, 1, 128), 2), w, w, {}, unit_offset=True)


def test_packed_and_in_place():
    """Views of a packed projection, results in their inputs' places, the last heads of a token beside the next tensor's."""
    t, hq, hk, dim = 10243, 7, 1, 128
    qkv = _rand((t, (hq + 2 * hk) * dim), 1, 3.0)
    q, k = qkv[:, :hq * dim].unflatten(1, (hq, dim)), qkv[:, hq * dim:(hq + hk) * dim].unflatten(1, (hk, dim))
    v = qkv[:, (hq + hk) * dim:].clone()
    w = 1 + _rand((dim,), 3, 0.2)
    rot = dict(positions=torch.arange(t, device=DEV), inv_freq=_freq(64))
    _check(q, k, w, w, rot)
    want = pf8.qk_norm_rope(q, k, w_q=w, w_k=w, **rot)
    d = _rand(qkv.shape, 5)
    dq, dk = d[:, :hq * dim].unflatten(1, (hq, dim)), d[:, hq * dim:(hq + hk) * dim].unflatten(1, (hk, dim))
    dv = d[:, (hq + hk) * dim:].clone()
    g = pf8.qk_norm_rope_backward(dq, dk, q, k, w_q=w, w_k=w, **rot)
    p = pf8.qk_norm_rope_backward(dq, dk, q, k, w_q=w, w_k=w, dq_out=dq, dk_out=dk, **rot)
    assert torch.equal(dq, g.dq) and torch.equal(dk, g.dk) and torch.equal(d[:, (hq + hk) * dim:], dv)
    assert torch.equal(p.dw_q, g.dw_q) and torch.equal(p.dw_k, g.dw_k)
    pf8.qk_norm_rope(q, k, w_q=w, w_k=w, q_out=q, k_out=k, **rot)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1]) and torch.equal(qkv[:, (hq + hk) * dim:], v)
