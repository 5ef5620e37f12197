"""The float64 reference of the layer's steps against central differences, closed forms and complex numbers."""
import numpy as np
import pytest

from oracle import layer

ROT = [dict(positions=np.array([0, 5, 123456]), inv_freq=np.array([1.0, 0.3, 1e-3])),
       dict(positions=np.array([[0, 5, 9], [3, 3, 4]]), inv_freq=np.array([1.0, 0.3, 1e-3]), sections=(2, 1)),
       dict(positions=np.array([[0, 5, 9], [3, 3, 4]]), inv_freq=np.array([1.0, 0.3, 1e-3]), sections=(2, 1), order="cycled"),
       {}]


@pytest.mark.parametrize("rot", ROT)
@pytest.mark.parametrize("interleaved", [False, True])
def test_head_norm_gradients_match_central_differences(rot, interleaved):
    rng = np.random.default_rng(1)
    x, d, w = rng.standard_normal((3, 2, 9)), rng.standard_normal((3, 2, 9)), 1 + 0.2 * rng.standard_normal(9)
    kw = dict(rot, interleaved=interleaved, scale=1.25 if rot else 1.0, eps=1e-3, offset=0.5)
    dx, _, dw, _ = layer.head_norm_grads(d, x, w, **kw)
    step = 1e-5  # O(step^2) curvature + 1e-16 / step rounding

    def num(a):
        out = np.zeros_like(a)
        for i in np.ndindex(a.shape):
            keep = a[i]
            a[i] = keep + step
            hi = np.sum(layer.head_norm(x, w, **kw)[0] * d)
            a[i] = keep - step
            lo = np.sum(layer.head_norm(x, w, **kw)[0] * d)
            a[i] = keep
            out[i] = (hi - lo) / (2 * step)
        return out

    np.testing.assert_allclose(dx, num(x), rtol=0, atol=1e-7)
    np.testing.assert_allclose(dw, num(w), rtol=0, atol=1e-7)


def test_rotation_is_a_product_of_complex_numbers():
    rng = np.random.default_rng(2)
    x, pos, f = rng.standard_normal((4, 3, 10)), np.array([0, 1, 7, 1000]), np.array([1.0, 0.1, 0.01, 0.001])
    turn = np.exp(1j * pos[:, None] * f)[:, None]
    got = layer.head_norm(x, positions=pos, inv_freq=f)[0]
    want = (x[..., :4] + 1j * x[..., 4:8]) * turn
    np.testing.assert_allclose(got, np.concatenate([want.real, want.imag, x[..., 8:]], -1), atol=1e-12)
    got = layer.head_norm(x, positions=pos, inv_freq=f, interleaved=True)[0]
    want = (x[..., 0:8:2] + 1j * x[..., 1:8:2]) * turn
    np.testing.assert_allclose(got[..., 0:8:2], want.real, atol=1e-12)
    np.testing.assert_allclose(got[..., 1:8:2], want.imag, atol=1e-12)


def test_axes_of_pairs():
    assert layer.pair_axes(6, (2, 3, 1)).tolist() == [0, 0, 1, 1, 1, 2]
    # in turn until an axis has its share, the rest to the first
    assert layer.pair_axes(8, (4, 2, 2), "cycled").tolist() == [0, 1, 2, 0, 1, 2, 0, 0]
    assert layer.pair_axes(3).tolist() == [0, 0, 0]


@pytest.mark.parametrize("name", [None, "relu", "relu2", "silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("gated", [False, True])
def test_activation_gradients_match_central_differences(name, gated):
    if gated and name is None:
        return
    rng = np.random.default_rng(3)
    z, dd = rng.standard_normal((5, 8)) * 2, rng.standard_normal((5, 4 if gated else 8))
    dz = layer.act_grads(dd, z, name, gated)
    step = 1e-6
    for i in np.ndindex(z.shape):
        if abs(z[i]) < 1e-4:
            continue  # relu's corner
        hi, lo = z.copy(), z.copy()
        hi[i] += step
        lo[i] -= step
        num = np.sum((layer.act_out(hi, name, gated) - layer.act_out(lo, name, gated)) * dd) / (2 * step)
        assert abs(num - dz[i]) < 1e-7


def test_activation_values():
    assert layer.act(np.array([-2.0, 0.0, 3.0]), "relu2")[0].tolist() == [0, 0, 9]
    np.testing.assert_allclose(layer.act(np.array([1.0]), "silu")[0], 0.7310585786300049)
    np.testing.assert_allclose(layer.act(np.array([1.0]), "gelu")[0], 0.8413447460685429)
    np.testing.assert_allclose(layer.act(np.array([1.0]), "gelu_tanh")[0], 0.8411919906082768)
