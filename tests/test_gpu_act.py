"""The activation's backward pass on the GPU against the float64 oracle.

Tolerances, fixed before the first run. dz is rounded once: 2^-8 of the value plus 2^-134. Before it, in FP32: the
value and slope of an activation are held to 2^-18 of max(1, |z|)^2 (the exponential's argument is off by 2^-24 of
itself, which the exponential turns into an error of |z| 2^-24 or z^2 2^-24 of its value, and the result is a
handful of such factors and differences from one), times |dd| and, with a gate, the other factor. Column sums: those errors
summed, plus a rounding of 2^-24 for each row of the running magnitude, under 2^12 rows here: 2^-12 of the
summed magnitudes.
"""
import numpy as np
import pytest
import torch

import fp8_block_scaled_pf8_amd as pf8
from oracle import layer
from tests.gpu_helpers import DEV

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
ACTS = ["relu", "relu2", "silu", "gelu", "gelu_tanh"]


def _rand(shape, seed, scale=1.0):
    return (torch.randn(shape, generator=torch.Generator().manual_seed(seed)) * scale).to(BF).to(DEV)


def _np(t):
    return t.detach().cpu().double().numpy()


def _check(dd, z, act, gated, got, bias=True):
    d, zn = _np(dd), None if z is None else _np(z)
    ref = layer.act_grads(d, zn, act, gated)
    if z is None:
        loose = np.zeros_like(ref)
    else:
        n = d.shape[1]
        grow = np.maximum(1.0, np.abs(zn[:, :n])) ** 2
        loose = 2.0 ** -18 * grow * np.abs(d)
        if gated:
            loose = np.concatenate([loose * np.abs(zn[:, n:]), loose], axis=1)
    tol = 2.0 ** -8 * np.abs(ref) + loose + 2.0 ** -134
    off = np.abs(_np(got.dz) - ref)
    assert (off <= tol).all(), f"dz: {np.max(off / tol)} of the tolerance"
    if bias:
        tol = loose.sum(0) + 2.0 ** -12 * np.abs(ref).sum(0) + 2.0 ** -134
        off = np.abs(_np(got.dbias) - ref.sum(0))
        assert (off <= tol).all(), f"dbias: {np.max(off / tol)} of the tolerance"
    else:
        assert got.dbias is None


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 8), (3, 7), (5, 9), (2, 2048), (300, 15), (130, 333), (17, 2049), (9, 4100)])
def test_sizes(act, gated, rows, cols):
    dd, z = _rand((rows, cols), 1), _rand((rows, 2 * cols if gated else cols), 2, 2.0)
    _check(dd, z, act, gated, pf8.act_backward(dd, z, act, gated=gated, bias_grad=True))
    _check(dd, z, act, gated, pf8.act_backward(dd, z, act, gated=gated), bias=False)


@pytest.mark.parametrize("rows,cols", [(1, 1), (300, 15), (2000, 512), (9, 4100)])
def test_bias_alone(rows, cols):
    dd = _rand((rows, cols), 1)
    got = pf8.act_backward(dd, None, None, bias_grad=True)
    assert got.dz is dd
    _check(dd, None, None, False, got)


@pytest.mark.parametrize("act", ACTS)
def test_far_values(act):
    """Far from zero a slope is 0 or what the limit is, and nothing overflows on the way."""
    vals = torch.tensor([0.0, -0.0, 1e-30, -1e-30, 5.0, -5.0, 15.0, -15.0, 40.0, -40.0, 100.0, -100.0, 1e4, -1e4, 1e18, -1e18],
                        dtype=BF, device=DEV)
    z = vals.reshape(1, -1)
    dd = torch.ones_like(z)
    got = _np(pf8.act_backward(dd, z, act).dz)[0]
    zn = _np(z)[0]
    near = np.abs(zn) <= 100
    ref = layer.act(zn, act)[1]
    assert (np.abs(got - ref)[near] <= (2.0 ** -8 * np.abs(ref) + 2.0 ** -18 * np.maximum(1, np.abs(zn)) ** 2)[near]).all()
    far = {"relu": [1, 0, 1, 0], "silu": [1, 0, 1, 0], "gelu": [1, 0, 1, 0], "gelu_tanh": [1, 0, 1, 0],
           "relu2": [2 * zn[12], 0, 2 * zn[14], 0]}[act]
    np.testing.assert_array_equal(got[12:], far)
    gate = pf8.act_backward(dd, torch.cat([z, torch.ones_like(z)], 1), act, gated=True).dz[0, 16:]
    assert gate.isfinite().all() or act == "relu2"


def test_not_a_number_stays():
    z = torch.full((1, 16), float("nan"), dtype=BF, device=DEV)
    for act in ("silu", "gelu", "gelu_tanh"):
        assert pf8.act_backward(torch.ones_like(z), z, act).dz.isnan().all()
    zz = torch.cat([z, z], 1)
    for act in ACTS:
        assert pf8.act_backward(torch.ones_like(z), zz, act, gated=True).dz[:, 16:].isnan().all()


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("cols", [64, 61, 5])
def test_pitches_in_place_and_neighbours(gated, cols):
    rows, w = 37, 2 * cols if gated else cols
    buf = _rand((rows, cols + w + 11), 3)
    dd, z = buf[:, :cols], buf[:, cols + 3:cols + 3 + w]
    want = pf8.act_backward(dd.contiguous(), z.contiguous(), "silu", gated=gated, bias_grad=True)
    out = torch.full((rows, w + 9), 7.0, dtype=BF, device=DEV)
    got = pf8.act_backward(dd, z, "silu", gated=gated, bias_grad=True, dz_out=out[:, 4:4 + w])
    assert torch.equal(out[:, 4:4 + w], want.dz) and torch.equal(got.dbias, want.dbias)
    assert (out[:, :4] == 7).all() and (out[:, 4 + w:] == 7).all()
    keep = buf.clone()
    if not gated:
        d2 = dd.contiguous()
        pf8.act_backward(d2, z, "silu", dz_out=d2)
        assert torch.equal(d2, want.dz)
    pf8.act_backward(dd, z, "silu", gated=gated, dz_out=z)
    assert torch.equal(z, want.dz)
    keep[:, cols + 3:cols + 3 + w] = want.dz
    assert torch.equal(buf, keep)


def test_accumulates_repeats_and_replays():
    dd, z = _rand((900, 500), 1), _rand((900, 1000), 2)
    a = pf8.act_backward(dd, z, "gelu", gated=True, bias_grad=True)
    b = pf8.act_backward(dd, z, "gelu", gated=True, bias_grad=True)
    assert torch.equal(a.dz, b.dz) and torch.equal(a.dbias, b.dbias)
    base = _rand((1000,), 3).float()
    want = base + a.dbias
    c = pf8.act_backward(dd, z, "gelu", gated=True, bias_grad=True, dbias_out=base, accumulate=True)
    assert c.dbias is base and torch.equal(base, want)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g = pf8.act_backward(dd, z, "gelu", gated=True, bias_grad=True)
    for i in range(3):
        z.copy_(_rand((900, 1000), 10 + i))
        graph.replay()
        e = pf8.act_backward(dd, z, "gelu", gated=True, bias_grad=True)
        torch.cuda.synchronize()
        assert torch.equal(g.dz, e.dz) and torch.equal(g.dbias, e.dbias)


def test_no_rows_and_refusals():
    dd, z = _rand((4, 64), 1), _rand((4, 64), 2)
    e = pf8.act_backward(dd[:0], z[:0], "silu", bias_grad=True)
    assert e.dz.shape == (0, 64) and (e.dbias == 0).all()
    for bad in (dict(activation="swish"), dict(activation=None), dict(z=None), dict(gated=True), dict(z=z.float()),
                dict(dd=dd[0]), dict(dd=dd.cpu()), dict(dd=dd.t()), dict(z=z[:3]), dict(accumulate=True),
                dict(dbias_out=torch.zeros(64, device=DEV)), dict(bias_grad=True, dbias_out=torch.zeros(63, device=DEV)),
                dict(bias_grad=True, accumulate=True), dict(dz_out=z[:, :63]), dict(activation=None, z=None)):
        with pytest.raises((ValueError, TypeError)):
            pf8.act_backward(**{**dict(dd=dd, z=z, activation="silu"), **bad})
    with pytest.raises(ValueError):
        pf8.act_backward(dd, None, None, gated=True, bias_grad=True)
    buf = _rand((4, 200), 1)
    with pytest.raises(ValueError, match="overlap"):
        pf8.act_backward(buf[:, :64], z, "silu", dz_out=buf[:, 32:96])
    with pytest.raises(ValueError, match="overlap"):
        pf8.act_backward(buf[:, :64], buf[:, 64:192], "silu", gated=True, dz_out=buf[:, 63:191])


@pytest.mark.parametrize("act", ACTS + [None])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("rows,cols", [(128, 128), (256, 384), (640, 128), (1152, 256)])
def test_codes_are_the_quantised_gradient(act, gated, rows, cols):
    """Codes and scales equal those of the two steps bit for bit; the bias's sums to the tolerance above."""
    if gated and act is None:
        pytest.skip("a gate needs an activation")
    w = 2 * cols if gated else cols
    buf = _rand((rows, cols + w + 24), 11, 2.0)
    dd, z = buf[:, 8:8 + cols], None if act is None else buf[:, cols + 16:cols + 16 + w]
    dd[3, :] = 0  # a row and a column group without a value
    dd[:128, 5] = 0
    keep = buf.clone()
    two = pf8.act_backward(dd, z, act, gated=gated, bias_grad=True)
    want = pf8.quant_act_dual(two.dz.contiguous())
    got = pf8.act_backward_quant(dd, z, act, gated=gated, bias_grad=True)
    for a, b in zip(got[:4], want):
        assert a.shape == b.shape and torch.equal(a, b)
    _check(dd, z, act, gated, pf8.ActGrads(two.dz, got.dbias))
    plain = pf8.act_backward_quant(dd, z, act, gated=gated)
    assert plain.dbias is None and all(torch.equal(a, b) for a, b in zip(plain[:4], want))
    assert torch.equal(buf, keep)


def test_codes_of_values_that_are_no_numbers():
    rows, cols = 128, 256
    dd, z = _rand((rows, cols), 1), _rand((rows, 2 * cols), 2)
    dd[1, 7], z[5, 9], z[6, 300], z[7, 11] = float("nan"), float("inf"), float("-inf"), float("nan")
    want = pf8.quant_act_dual(pf8.act_backward(dd, z, "silu", gated=True).dz)
    got = pf8.act_backward_quant(dd, z, "silu", gated=True)
    assert all(torch.equal(a, b) for a, b in zip(got[:4], want))


def test_codes_accumulate_replay_and_another_stream():
    dd, z = _rand((384, 256), 1), _rand((384, 512), 2)
    a = pf8.act_backward_quant(dd, z, "gelu", gated=True, bias_grad=True)
    base = torch.ones(512, dtype=torch.float32, device=DEV)
    c = pf8.act_backward_quant(dd, z, "gelu", gated=True, bias_grad=True, dbias_out=base, accumulate=True)
    assert c.dbias is base and torch.equal(base, 1 + a.dbias)
    one = torch.full((512,), 2.0, dtype=torch.float32, device=DEV)  # a single row of tiles adds without partial sums
    s = pf8.act_backward_quant(dd[:128], z[:128], "gelu", gated=True, bias_grad=True)
    pf8.act_backward_quant(dd[:128], z[:128], "gelu", gated=True, bias_grad=True, dbias_out=one, accumulate=True)
    assert torch.equal(one, 2 + s.dbias)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        b = pf8.act_backward_quant(dd, z, "gelu", gated=True, bias_grad=True)
    side.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g = pf8.act_backward_quant(dd, z, "gelu", gated=True, bias_grad=True)
    for i in range(3):
        dd.copy_(_rand((384, 256), 20 + i))
        graph.replay()
        e = pf8.act_backward_quant(dd, z, "gelu", gated=True, bias_grad=True)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(g, e))


def test_codes_refusals():
    dd, z = _rand((128, 128), 1), _rand((128, 128), 2)
    bad = [dict(dd=dd[:64], z=z[:64]), dict(dd=dd[:0], z=z[:0]), dict(dd=dd[:, :64], z=z[:, :64]), dict(z=None),
           dict(activation=None), dict(gated=True), dict(dbias_out=torch.zeros(128, device=DEV)), dict(accumulate=True),
           dict(dd=_rand((128, 136), 3)[:, 1:129]), dict(z=_rand((128, 132), 3)[:, :128])]
    for kw in bad:
        with pytest.raises((ValueError, TypeError)):
            pf8.act_backward_quant(**{**dict(dd=dd, z=z, activation="silu"), **kw})
    with pytest.raises((ValueError, TypeError)):
        pf8.act_backward_quant(dd.cpu(), z, "silu")
