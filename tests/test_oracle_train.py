"""The float64 reference of the training operators against central differences and closed forms."""
import numpy as np
import pytest

from oracle import train


def _case(rows, cols, post, pre, gate, seed):
    rng = np.random.default_rng(seed)
    n = lambda *s: rng.standard_normal(s)  # noqa: E731
    kw = dict(h=2 * n(rows, cols), y=n(rows, cols), w_pre=1 + 0.2 * n(cols) if pre else None,
              w_post=1 + 0.2 * n(cols) if post else None,
              gate={"none": None, "vector": n(cols), "full": n(rows, cols)}[gate])
    return kw, n(rows, cols), n(rows, cols) if pre else None


@pytest.mark.parametrize("post,pre", [(True, True), (True, False), (False, True)])
@pytest.mark.parametrize("gate", ["none", "vector", "full"])
def test_block_norm_gradients_match_central_differences(post, pre, gate):
    kw, dr, dx = _case(3, 11, post, pre, gate, 5)
    sc = dict(beta=0.75, alpha=0.5, eps=1e-3, offset=0.25)
    got, _ = train.block_norm_grads(dr, dx, **kw, **sc)

    def loss(k):
        r, x, _, _ = train.block_norm(**k, **sc)
        return np.sum(r * dr) + (np.sum(x * dx) if pre else 0.0)

    step = 1e-5  # error of a central difference: O(step^2) curvature + 1e-16 / step rounding, both < 1e-8 here
    for name, grad in (("h", got.dh), ("y", got.dy), ("gate", got.dgate), ("w_pre", got.dw_pre), ("w_post", got.dw_post)):
        if kw[name] is None:
            assert grad is None
            continue
        num = np.zeros_like(kw[name])
        for i in np.ndindex(num.shape):
            lo, hi = dict(kw), dict(kw)
            lo[name], hi[name] = kw[name].copy(), kw[name].copy()
            lo[name][i] -= step
            hi[name][i] += step
            num[i] = (loss(hi) - loss(lo)) / (2 * step)
        np.testing.assert_allclose(grad, num, rtol=0, atol=1e-7)


def test_block_norm_closed_forms():
    h = np.array([[3.0, -4.0], [0.0, 0.0]])
    r, x, _, _ = train.block_norm(h, w_pre=np.ones(2), eps=0.5)
    # mean square 12.5, plus 0.5: rms sqrt(13)
    np.testing.assert_allclose(x, [[3 / np.sqrt(13), -4 / np.sqrt(13)], [0, 0]], atol=1e-15)
    r, x, _, _ = train.block_norm(h, y=np.array([[1.0, 1.0], [2.0, -2.0]]), w_post=np.array([2.0, 3.0]), alpha=0.5,
                                  beta=2.0, eps=0.0)
    np.testing.assert_allclose(r, [[7.0, -6.5], [1.0, -1.5]], atol=1e-15)
    assert x is None


def test_newton_schulz_acts_on_the_singular_values():
    rng = np.random.default_rng(1)
    coef = [(3.4445, -4.7750, 2.0315)] * 5
    for m, n in ((6, 9), (9, 6), (7, 7), (1, 5)):
        g = rng.standard_normal((m, n))
        u, s, vt = np.linalg.svd(g, full_matrices=False)
        s = s / (np.linalg.norm(g) + 1e-7)
        for a, b, c in coef:
            s = a * s + b * s ** 3 + c * s ** 5
        np.testing.assert_allclose(train.newton_schulz(g, coef), (u * s) @ vt, atol=1e-12)
    assert not train.newton_schulz(np.zeros((3, 4)), coef).any()


@pytest.mark.parametrize("pairs", [False, True])
def test_newton_schulz_operands_are_close_to_exact(pairs):
    rng = np.random.default_rng(2)
    coef = [(3.4445, -4.7750, 2.0315)] * 5
    for m, n in ((40, 60), (90, 70), (150, 200)):
        for g in (rng.standard_normal((m, n)), rng.standard_normal((m, 2)) @ rng.standard_normal((2, n))):
            ref = train.newton_schulz(g, coef)
            got = train.newton_schulz_operands(g, coef, pairs=pairs)
            off = np.linalg.norm(got - ref) / np.linalg.norm(ref)
            assert 1e-5 < off < 2.5e-3  # FP16's half step is 4.9e-4, over five steps
