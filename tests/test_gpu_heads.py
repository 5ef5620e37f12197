"""The head norm with rotation on the GPU against the float64 oracle.

Tolerances, fixed before the first run. A bf16 output is rounded once: half a step, 2^-8 of the value, plus
2^-134 below bf16's smallest step. Before it: sums of up to 512 values along a lane (16), a group (6 levels) and
about 20 further FP32 roundings, under 2^6 roundings of 2^-24; sines and cosines from instructions that take turns,
each held to 2^-18 of one: together 2^-17 of the oracle's "size" (the same expression of magnitudes). The FP32
sums of the weights add at most one rounding for each of a lane's heads, of the groups of a workgroup and of the
partial rows, under 2^10 here: 2^-14 of their size.
"""
import itertools

import numpy as np
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
    return None if t is None else t.detach().cpu().double().numpy()


def _freq(pairs, base=1e4, dtype=torch.float32):
    return (float(base) ** (-torch.arange(pairs, dtype=torch.float64) / pairs)).to(dtype).to(DEV)


def _close(got, ref, size, what):
    low = got.dtype == BF
    got = _np(got)
    assert got.shape == ref.shape, what
    fine = np.isfinite(ref)
    np.testing.assert_array_equal(np.isfinite(got), fine, err_msg=what)
    tol = (2.0 ** -8 * np.abs(ref) + 2.0 ** -17 * size if low else 2.0 ** -14 * size) + 2.0 ** -134
    off = np.abs(got - ref)[fine]
    assert (off <= tol[fine]).all(), f"{what}: {np.max(off / tol[fine])} of the tolerance"


def _oracle(rot, kw):
    o = dict(rot)
    o = {n: _np(t) if isinstance(t, torch.Tensor) else t for n, t in o.items()}
    if "section_order" in o:
        o["order"] = o.pop("section_order")
    if "rotary_scale" in o:
        o["scale"] = o.pop("rotary_scale")
    return dict(o, eps=float(np.float32(kw.get("eps", 1e-6))), offset=1.0 if kw.get("unit_offset") else 0.0)


def _check(q, k, w_q, w_k, rot, seed=9, **kw):
    o = _oracle(rot, kw)
    oq, ok = pf8.qk_norm_rope(q, k, w_q=w_q, w_k=w_k, **rot, **kw)
    dq, dk = _rand(q.shape, seed), None if k is None else _rand(k.shape, seed + 1)
    g = pf8.qk_norm_rope_backward(dq, dk, q, k, w_q=w_q, w_k=w_k, **rot, **kw)
    for n, x, w, got, d, dx, dw in (("q", q, w_q, oq, dq, g.dq, g.dw_q), ("k", k, w_k, ok, dk, g.dk, g.dw_k)):
        if x is None:
            assert got is None and dx is None and dw is None
            continue
        ref, size = layer.head_norm(_np(x), _np(w), **o)
        _close(got, ref, size, n)
        rx, sx, rw, sw = layer.head_norm_grads(_np(d), _np(x), _np(w), **o)
        _close(dx, rx, sx, "d" + n)
        assert (dw is None) == (rw is None)
        if rw is not None:
            _close(dw, rw, sw, "dw_" + n)


# head_dim, pairs: whole steps of 8 pairs, ragged ones, nearly all and hardly any rotated, odd, tiny, the largest
DIMS = [(128, 64), (64, 32), (96, 48), (80, 20), (72, 36), (32, 16), (256, 128), (512, 256), (192, 32), (40, 10),
        (74, 37), (50, 25), (30, 11), (66, 8), (16, 8), (2, 1), (7, 3), (3, 1), (33, 16), (511, 200), (130, 60), (22, 9)]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dim,pairs", DIMS)
def test_sizes(dim, pairs, interleaved):
    q, k = _rand((5, 6, dim), 1, 3.0), _rand((5, 3, dim), 2, 3.0)
    pos = torch.tensor([0, 1, 77, 4095, 999983], device=DEV)
    _check(q, k, 1 + _rand((dim,), 3, 0.2), 1 + _rand((dim,), 4, 0.2),
           dict(positions=pos, inv_freq=_freq(pairs), interleaved=interleaved))


@pytest.mark.parametrize("tokens,hq,hk", [(1, 1, 1), (1, 16, 8), (3, 7, 1), (257, 16, 8), (65, 1, 5), (33, 64, 4), (2, 300, 1)])
@pytest.mark.parametrize("norm", ["both", "q", "none"])
def test_tokens_and_heads(tokens, hq, hk, norm):
    q, k = _rand((tokens, hq, 64), 1, 3.0), _rand((tokens, hk, 64), 2, 3.0)
    w_q = _rand((64,), 3, 0.2, torch.float32) if norm != "none" else None
    w_k = _rand((64,), 4, 0.2, torch.float32) if norm == "both" else None
    _check(q, k, w_q, w_k, dict(positions=torch.arange(tokens, device=DEV, dtype=torch.int32) * 1001, inv_freq=_freq(32)),
           unit_offset=True)


@pytest.mark.parametrize("order", ["blocked", "cycled"])
@pytest.mark.parametrize("sections", [(16, 24, 24), (24, 20, 20), (40, 24), (64,), (31, 11, 11, 11)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_axes(sections, order, interleaved):
    if order == "cycled" and sections == (16, 24, 24):
        sections = (22, 21, 21)
    pos = torch.randint(-5, 70000, (len(sections), 19), generator=torch.Generator().manual_seed(1)).to(DEV)
    rot = dict(positions=pos, inv_freq=_freq(sum(sections), 1e6, torch.float64), sections=sections, section_order=order,
               interleaved=interleaved, rotary_scale=1.25)
    _check(_rand((19, 4, 144), 1), _rand((19, 2, 144), 2), None, 1 + _rand((144,), 3, 0.2), rot)
    _check(_rand((19, 4, 141), 1), None, 1 + _rand((141,), 3, 0.2), None, rot)


def test_norm_alone_and_queries_alone():
    q = _rand((9, 5, 128), 1, 3.0)
    _check(q, None, 1 + _rand((128,), 3, 0.2), None, {}, eps=1e-3)
    _check(q, _rand((9, 2, 128), 2), None, 1 + _rand((128,), 3, 0.2), {})
    _check(_rand((9, 5, 1), 1), None, 1 + _rand((1,), 3, 0.2), None, {})
    oq, ok = pf8.qk_norm_rope(q, _rand((9, 2, 128), 2), w_k=1 + _rand((128,), 3, 0.2))
    assert torch.equal(oq, q)  # neither normalised nor rotated


def test_far_positions():
    """An angle is right to a fraction of a turn at any position an int64 of 2^50 can name."""
    pos = torch.tensor([2 ** 31 + 5, 2 ** 40 + 1, 2 ** 50 + 3, -(2 ** 33) - 1], device=DEV)
    q = _rand((4, 3, 64), 1)
    freq = torch.tensor([2.0 ** -i for i in range(32)], device=DEV, dtype=torch.float64)  # products exact in float64
    # turns = pos * f / 2 pi: 2^50 / 2 pi has 2^-5 turns a step of float64, so the oracle reduces exactly
    import fractions
    two_pi = fractions.Fraction("6.28318530717958647692528676655900576839433879875021164194988918461563281257")
    angle = np.array([[float((fractions.Fraction(int(p)) * fractions.Fraction(float(f)) / two_pi) % 1) for f in freq]
                      for p in pos[[0, 1, 3]]])
    got = _np(pf8.qk_norm_rope(q, None, pos, freq)[0])[[0, 1, 3]]
    x = _np(q)[[0, 1, 3]]
    c, s = np.cos(2 * np.pi * angle)[:, None], np.sin(2 * np.pi * angle)[:, None]
    want = np.concatenate([x[..., :32] * c - x[..., 32:] * s, x[..., :32] * s + x[..., 32:] * c], -1)
    size = np.concatenate([np.abs(x[..., :32]) + np.abs(x[..., 32:])] * 2, -1)
    # float64 turns at 2^40: 1 / 2 pi is off by 2^-55 of itself and the product by 2^-53: 2^-53 * 2^38 turns
    assert (np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + (2.0 ** -17 + 2 * np.pi * 2.0 ** -14) * size).all()


@pytest.mark.parametrize("dim,pairs", [(128, 64), (74, 37)])
def test_strides_and_packed_views(dim, pairs):
    hq, hk, t = 4, 2, 21
    qkv = _rand((t, (hq + 2 * hk) * dim + 3), 1, 3.0)
    q = qkv[:, :hq * dim].unflatten(1, (hq, dim))
    k = qkv[:, hq * dim:(hq + hk) * dim].unflatten(1, (hk, dim))
    rot = dict(positions=torch.arange(3 * t, device=DEV)[::3], inv_freq=_freq(pairs))
    w = 1 + _rand((dim,), 3, 0.2)
    _check(q, k, w, w, rot)
    heads_first = _rand((hq, t, dim), 5).transpose(0, 1)
    _check(heads_first, k, w, w, rot)
    want_q, want_k = pf8.qk_norm_rope(q, k, w_q=w, w_k=w, **rot)
    # results into places beside other values, which stay
    out = torch.full_like(qkv, 5.0)
    oq, ok = out[:, :hq * dim].unflatten(1, (hq, dim)), out[:, hq * dim:(hq + hk) * dim].unflatten(1, (hk, dim))
    got = pf8.qk_norm_rope(q, k, w_q=w, w_k=w, q_out=oq, k_out=ok, **rot)
    assert got[0] is oq and torch.equal(oq, want_q) and torch.equal(ok, want_k)
    assert (out[:, (hq + hk) * dim:] == 5.0).all()
    # in place
    values = qkv[:, (hq + hk) * dim:].clone()
    dq, dk = _rand((t, hq, dim), 6), _rand((t, hk, dim), 7)
    g = pf8.qk_norm_rope_backward(dq, dk, q, k, w_q=w, w_k=w, **rot)
    g2 = pf8.qk_norm_rope_backward(dq, dk, q, k, w_q=w, w_k=w, dq_out=oq, dk_out=dk, **rot)
    assert torch.equal(g2.dq, g.dq) and torch.equal(dk, g.dk) and torch.equal(g2.dw_q, g.dw_q)
    pf8.qk_norm_rope(q, k, w_q=w, w_k=w, q_out=q, k_out=k, **rot)
    assert torch.equal(q, want_q) and torch.equal(k, want_k) and torch.equal(qkv[:, (hq + hk) * dim:], values)


def test_zero_infinite_and_huge_heads():
    q = _rand((6, 4, 64), 1)
    q[0, 1] = 0.0
    q[1, 2, 5] = float("inf")
    q[2, 0, 60] = float("nan")
    q[3, 3] *= 2.0 ** 60
    q[4, 0] *= 2.0 ** -70
    w = 1 + _rand((64,), 3, 0.2)
    rot = dict(positions=torch.arange(6, device=DEV), inv_freq=_freq(32))
    got = pf8.qk_norm_rope(q, None, w_q=w, **rot)[0]
    clean = torch.ones(6, 4, dtype=torch.bool, device=DEV)
    clean[1, 2] = clean[2, 0] = False
    o = _oracle(rot, {})
    ref, size = layer.head_norm(_np(q), _np(w), **o)
    c = clean.cpu().numpy()
    _close(got[clean], ref[c], size[c], "q")
    assert (got[0, 1] == 0).all() and got[2, 0].isnan().all()
    assert got[1, 2, 5].isnan() or got[1, 2, 5].isinf()
    d = _rand((6, 4, 64), 5)
    g = pf8.qk_norm_rope_backward(d, None, q, None, w_q=w, **rot)
    rx, sx, _, _ = layer.head_norm_grads(_np(d), _np(q), _np(w), **o)
    _close(g.dq[clean], rx[c], sx[c], "dq")


def test_no_tokens():
    q, k, w = _rand((0, 4, 64), 1), _rand((0, 2, 64), 1), 1 + _rand((64,), 3, 0.2)
    rot = dict(positions=torch.zeros(0, dtype=torch.int64, device=DEV), inv_freq=_freq(32))
    oq, ok = pf8.qk_norm_rope(q, k, w_q=w, w_k=w, **rot)
    assert oq.shape == q.shape and ok.shape == k.shape
    g = pf8.qk_norm_rope_backward(q, k, q, k, w_q=w, w_k=w, **rot)
    assert (g.dw_q == 0).all() and (g.dw_k == 0).all() and g.dq.shape == q.shape
    m = pf8.QKNormRope(64, device=DEV)
    x = torch.zeros(0, 4, 64, dtype=BF, device=DEV, requires_grad=True)
    m(x, None, rot["positions"])[0].sum().backward()
    assert x.grad.shape == x.shape


def test_accumulates_and_repeats():
    q, k, w = _rand((700, 8, 128), 1, 3.0), _rand((700, 2, 128), 2), 1 + _rand((128,), 3, 0.2)
    dq, dk = _rand(q.shape, 4), _rand(k.shape, 5)
    rot = dict(positions=torch.arange(700, device=DEV), inv_freq=_freq(64))
    a = pf8.qk_norm_rope_backward(dq, dk, q, k, w_q=w, w_k=w, **rot)
    b = pf8.qk_norm_rope_backward(dq, dk, q, k, w_q=w, w_k=w, **rot)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    base = [_rand((128,), 6, 1.0, torch.float32), _rand((128,), 7, 1.0, torch.float32)]
    want = [base[0] + a.dw_q, base[1] + a.dw_k]
    c = pf8.qk_norm_rope_backward(dq, dk, q, k, w_q=w, w_k=w, dw_q_out=base[0], dw_k_out=base[1], accumulate=True, **rot)
    assert c.dw_q is base[0] and torch.equal(base[0], want[0]) and torch.equal(base[1], want[1])


@pytest.mark.parametrize("batch", [1, 2, 3, 4])
def test_positions_broadcast_behind_their_axes(batch):
    """[axes, seq] for q [batch, seq, ...] are every batch's positions, whatever the batch's size is."""
    q = _rand((batch, 5, 2, 64), 3)
    pos = torch.randint(0, 100, (3, 5), generator=torch.Generator().manual_seed(1)).to(DEV)
    rot = dict(inv_freq=torch.linspace(1, 0.01, 32, device=DEV), sections=(16, 8, 8))
    got = pf8.fp8_qk_norm_rope(q, None, pos, **rot)[0]
    for i in range(batch):
        assert torch.equal(got[i], pf8.qk_norm_rope(q[i], None, pos, **rot)[0])
    assert torch.equal(got, pf8.fp8_qk_norm_rope(q, None, pos[:, None], **rot)[0])
    one = pf8.fp8_qk_norm_rope(q, None, pos[0], rot["inv_freq"])[0]
    assert torch.equal(one[batch - 1], pf8.qk_norm_rope(q[batch - 1], None, pos[0], rot["inv_freq"])[0])
    with pytest.raises((RuntimeError, ValueError)):
        pf8.fp8_qk_norm_rope(q, None, pos[:, :4], **rot)


def test_one_weight_for_both_with_one_main_grad():
    q, k, w = _rand((9, 4, 64), 1).requires_grad_(), _rand((9, 2, 64), 2).requires_grad_(), _rand((64,), 3)
    dq, dk = _rand((9, 4, 64), 4), _rand((9, 2, 64), 5)
    a, b, m = (torch.zeros(64, device=DEV) for _ in range(3))
    for main in ((a, b), (m, m)):
        ww = w.clone().requires_grad_()
        torch.autograd.backward(pf8.fp8_qk_norm_rope(q, k, w_q=ww, w_k=ww, main_grads=main), [dq, dk])
        assert ww.grad is None
    assert torch.equal(m, a + b)


def test_module_gradients_against_differences_of_the_oracle():
    """The module's gradients along random directions against central differences of the float64 oracle, from bf16
    gradients: each of n products is off by 2^-8 of its own (gradient's rounding)."""
    m = pf8.QKNormRope(64, rotary_dim=32, sections=(10, 3, 3), section_order="cycled", device=DEV, unit_offset=True)
    with torch.no_grad():
        m.w_q.copy_(_rand((64,), 1, 0.2))
        m.w_k.copy_(_rand((64,), 2, 0.2))
    q = _rand((2, 7, 4, 64), 3).requires_grad_()
    k = _rand((2, 7, 2, 64), 4).requires_grad_()
    pos = torch.stack([torch.arange(7, device=DEV)] * 3)[:, None]  # [axes, 1, seq]: broadcast over the batch
    oq, ok = m(q, k, pos)
    dq, dk = _rand(oq.shape, 5), _rand(ok.shape, 6)
    torch.autograd.backward([oq, ok], [dq, dk])
    o = dict(positions=_np(pos.expand(3, 2, 7).reshape(3, -1)), inv_freq=_np(m.inv_freq), sections=(10, 3, 3),
             order="cycled", eps=float(np.float32(1e-6)), offset=1.0)
    for x, w, d in ((q, m.w_q, dq), (k, m.w_k, dk)):
        xn, wn, dn = _np(x).reshape(14, -1, 64), _np(w), _np(d).reshape(14, -1, 64)
        rng = np.random.default_rng(7)
        vx, vw = rng.standard_normal(xn.shape), rng.standard_normal(64)
        f = lambda e: np.sum(layer.head_norm(xn + e * vx, wn + e * vw, **o)[0] * dn)  # noqa: E731
        num = (f(1e-5) - f(-1e-5)) / 2e-5
        gx, gw = _np(x.grad).reshape(xn.shape), _np(w.grad)
        got = np.sum(gx * vx) + np.sum(gw * vw)
        tol = 2.0 ** -7 * (np.sum(np.abs(gx * vx)) + np.sum(np.abs(gw * vw))) / np.sqrt(gx.size) * 8
        assert abs(got - num) <= tol


def test_module_main_grads_casts_and_captures():
    m = pf8.QKNormRope(64, device=DEV, fp32_main_grad=True)
    freq = m.inv_freq.clone()
    m.to(torch.bfloat16)
    assert m.inv_freq.dtype == torch.float32 and torch.equal(m.inv_freq, freq)
    q, k = _rand((33, 4, 64), 1), _rand((33, 2, 64), 2)
    pos = torch.arange(33, device=DEV)
    dq, dk = _rand(q.shape, 3), _rand(k.shape, 4)
    g = pf8.qk_norm_rope_backward(dq, dk, q, k, pos, m.inv_freq, m.w_q.detach(), m.w_k.detach())
    x, y = q.clone().requires_grad_(), k.clone().requires_grad_()
    for i in range(2):
        torch.autograd.backward(m(x, y, pos), [dq, dk])
    assert m.w_q.grad is None and torch.equal(m.w_q.main_grad, g.dw_q + g.dw_q) and torch.equal(x.grad, (g.dq + g.dq))
    # one of the two without a gradient
    m.w_q.main_grad.zero_(), m.w_k.main_grad.zero_()
    m(x, y, pos)[1].backward(dk)
    assert (m.w_q.main_grad == 0).all() and torch.equal(m.w_k.main_grad, g.dw_k)
    # captured, replayed with other inputs, against eager calls
    qs, ks = q.clone(), k.clone()
    pf8.qk_norm_rope(qs, ks, pos, m.inv_freq, m.w_q.detach(), m.w_k.detach())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        oq, ok = pf8.qk_norm_rope(qs, ks, pos, m.inv_freq, m.w_q.detach(), m.w_k.detach())
        gg = pf8.qk_norm_rope_backward(dq, dk, qs, ks, pos, m.inv_freq, m.w_q.detach(), m.w_k.detach())
    for i in range(3):
        qs.copy_(_rand(q.shape, 20 + i))
        ks.copy_(_rand(k.shape, 30 + i))
        graph.replay()
        eq, ek = pf8.qk_norm_rope(qs, ks, pos, m.inv_freq, m.w_q.detach(), m.w_k.detach())
        eg = pf8.qk_norm_rope_backward(dq, dk, qs, ks, pos, m.inv_freq, m.w_q.detach(), m.w_k.detach())
        torch.cuda.synchronize()
        assert torch.equal(oq, eq) and torch.equal(ok, ek) and all(torch.equal(a, b) for a, b in zip(gg, eg))
    # a captured backward that would hand a gradient to a leaf is refused
    leaf = q.clone().requires_grad_()
    with pytest.raises(RuntimeError, match="leaf"):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            pf8.fp8_qk_norm_rope(leaf, None, pos, m.inv_freq)[0].backward(dq)


def test_refusals():
    q, k, w = _rand((5, 4, 64), 1), _rand((5, 2, 64), 2), 1 + _rand((64,), 3, 0.2)
    pos, f = torch.arange(5, device=DEV), _freq(32)
    bad = [dict(q=q.float()), dict(q=q[0]), dict(q=q.cpu()), dict(k=k[:4]), dict(k=_rand((5, 2, 32), 1)), dict(w_q=w[:63]),
           dict(w_q=w.float()), dict(w_q=w.half()), dict(positions=pos[:4]), dict(positions=pos.float()),
           dict(positions=None), dict(inv_freq=None), dict(inv_freq=f.half()), dict(inv_freq=_freq(33)), dict(inv_freq=f[::2]),
           dict(sections=(16, 16)), dict(sections=(16, 17), positions=pos.expand(2, 5)),
           dict(sections=(8, 24), section_order="cycled", positions=pos.expand(2, 5)), dict(section_order="by turns"),
           dict(q=q.transpose(1, 2).contiguous().transpose(1, 2)), dict(q=q[:, :1].expand(5, 4, 64)), dict(k=None),
           dict(q_out=q[:, :3]), dict(q_out=k), dict(k_out=q[:, :2]), dict(q=_rand((5, 1, 513), 1), k=None, w_k=None, w_q=None),
           dict(eps=-1.0), dict(eps=float("nan")), dict(rotary_scale=float("inf")),
           dict(positions=pos.cpu()), dict(positions=None, inv_freq=None, w_q=None, w_k=None)]
    good = dict(q=q, k=k, positions=pos, inv_freq=f, w_q=w, w_k=w)
    pf8.qk_norm_rope(**good)
    for b in bad:
        with pytest.raises((ValueError, TypeError, RuntimeError)):
            pf8.qk_norm_rope(**{**good, **b})
    buf = _rand((5, 8, 64), 1)
    with pytest.raises(ValueError, match="overlap"):
        pf8.qk_norm_rope(buf[:, 1:5], None, pos, f, q_out=buf[:, :4])
    with pytest.raises(ValueError, match="overlap"):
        pf8.qk_norm_rope(q, k, pos, f, q_out=buf[:, :4], k_out=buf[:, 3:5])
    with pytest.raises(ValueError, match="overlap"):
        pf8.qk_norm_rope(q, None, pos, f, q_out=buf[:1, :4].expand(5, 4, 64))
    pf8.qk_norm_rope(buf[:, :4], None, pos, f, q_out=buf[:, 4:])
    dq, dk = _rand(q.shape, 4), _rand(k.shape, 5)
    for b in (dict(q=None), dict(accumulate=True), dict(dw_q_out=torch.zeros(63, device=DEV)), dict(dq=dq[:4]),
              dict(dk=None), dict(dw_k_out=w)):
        with pytest.raises((ValueError, TypeError)):
            pf8.qk_norm_rope_backward(**{**dict(dq=dq, dk=dk, q=q, k=k, positions=pos, inv_freq=f, w_q=w, w_k=w), **b})


def test_another_stream():
    q, w = _rand((4000, 16, 128), 1, 3.0), 1 + _rand((128,), 3, 0.2)
    pos, f = torch.arange(4000, device=DEV), _freq(64)
    want = pf8.qk_norm_rope(q, None, pos, f, w)[0]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        x = q * 1
        got = pf8.qk_norm_rope(x, None, pos, f, w)[0]
    s.synchronize()
    assert torch.equal(got, want)


def test_drawn_sizes():
    rng = np.random.default_rng(11)
    for i, _ in zip(range(40), itertools.count()):
        dim = int(rng.integers(2, 300))
        pairs = int(rng.integers(1, dim // 2 + 1))
        t, hq, hk = int(rng.integers(1, 40)), int(rng.integers(1, 12)), int(rng.integers(1, 9))
        inter = bool(rng.integers(2))
        w = 1 + _rand((dim,), i, 0.2)
        _check(_rand((t, hq, dim), i + 1, 3.0), _rand((t, hk, dim), i + 2, 3.0), w if i % 3 else None, w,
               dict(positions=torch.from_numpy(rng.integers(0, 1 << 20, t)).to(DEV), inv_freq=_freq(pairs), interleaved=inter))
