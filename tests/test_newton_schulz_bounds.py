"""Newton-Schulz: the precision that include/pf8_train.h states, on gradients whose weight lies in few rows.

The bounds stand by themselves; nothing here is derived from what a kernel or its model loses.

A step X <- a X + f(A) X, f(A) = b A + c A A, rounds its operands to FP16: half a step is 2^-11 of the value,
2^-11 / sqrt(3) * 0.735 = 2.1e-4 in the root mean square over a binade. X's rounding enters the product with
|f| <= 2.9 (s up to 1.2), and A = X X^T from both sides with sqrt(2) |b + 2 c s^2| s^2 <= 3.4 (at s^2 = 0.7 to
1.4): together 4.5 * 2.1e-4 = 9.4e-4 a step. A step hands on a change of the singular vectors as it is, and
of a singular value near one with a factor of about one. Five steps at most have singular values near one:
sqrt(5) * 9.4e-4 = 2.1e-3, stated as 2e-3. Where few entries carry the norm they may all be near their largest
error, 2.36 times the root mean square: 5e-3 for those drawn here. The header says 4e-3 for under ten rows and
1.5e-2 for under 64 entries, which covers unlucky ones: the largest of 3000 and of 12000 drawn were 3.5e-3
and 9.8e-3. Where the entries take few magnitudes, the roundings of a step are alike and do not average out:
1.5e-2 (a constant matrix, whose iteration is one of scalars: 1.45e-2 the largest of 400000 sizes).

The BF16 rounding of the result: 1.7e-3 (1 + 1.8 / sqrt(N)) of the 2-norm, at most 2^-8, N = (sum y^2)^2 /
sum y^4; independent of the rest where N >= 64, else the two add.
"""
import numpy as np
import pytest
import torch

from oracle import train

QUINTIC = (3.4445, -4.7750, 2.0315)


def _rows(m, n, seed, rows, cols=None, rank=1, noise=0.0):
    """`rows` rows of rank `rank` in `cols` columns, over a floor of noise."""
    r = np.random.default_rng(seed)
    x = noise * r.standard_normal((m, n))
    at = r.permutation(m)[:rows]
    to = slice(None) if cols is None else slice(0, cols)
    x[at, to] += r.standard_normal((rows, rank)) @ r.standard_normal((rank, n if cols is None else cols))
    return x


def _two_rows(m, n, seed):
    r = np.random.default_rng(seed)
    x = np.zeros((m, n))
    x[5] = r.standard_normal(n)
    x[9] = 0.5 * x[5]
    return x


def _hot(share):
    def make(m, n, seed):
        r = np.random.default_rng(seed)
        u = r.standard_normal(m)
        u[3] = 0.0
        u *= np.sqrt(1 - share) / np.linalg.norm(u)
        u[3] = np.sqrt(share)
        return np.outer(u, r.standard_normal(n))
    return make


def _softmax(m, n, seed):
    """The gradient of a softmax's weight for one token: (one-hot - p) x^T."""
    r = np.random.default_rng(seed)
    u = -np.exp(2 * r.standard_normal(m))
    u /= -u.sum()
    u[7] += 1.0
    return np.outer(u, r.standard_normal(n))


def _hot_rank(k):
    def make(m, n, seed):
        r = np.random.default_rng(seed)
        u = 0.3 * r.standard_normal((m, k)) / np.sqrt(m)
        u[3 * np.arange(k), np.arange(k)] += 1.0
        return u @ r.standard_normal((k, n))
    return make


def _rank(part):
    def make(m, n, seed):
        r = np.random.default_rng(seed)
        k = max(1, int(min(m, n) * part))
        return r.standard_normal((m, k)) @ r.standard_normal((k, n))
    return make


GENERAL, FEW, ALIKE = 2e-3, 5e-3, 1.5e-2
KINDS = {
    "two_rows": (_two_rows, GENERAL),
    "hot_0.62": (_hot(0.62), GENERAL),
    "hot_0.7": (_hot(0.7), GENERAL),
    "hot_0.9": (_hot(0.9), GENERAL),
    "softmax": (_softmax, GENERAL),
    "hot_rank_4": (_hot_rank(4), GENERAL),
    "rows_2": (lambda m, n, s: _rows(m, n, s, 2), GENERAL),
    "rows_4": (lambda m, n, s: _rows(m, n, s, 4), GENERAL),
    "rows_8_rank_2": (lambda m, n, s: _rows(m, n, s, 8, rank=2), GENERAL),
    "rows_8_over_noise": (lambda m, n, s: _rows(m, n, s, 8, noise=1e-4), GENERAL),
    "rows_2_cols_4": (lambda m, n, s: _rows(m, n, s, 2, 4), FEW),
    "rows_8_cols_4": (lambda m, n, s: _rows(m, n, s, 8, 4), FEW),
    "rank_3_of_4": (_rank(0.75), GENERAL),
    "rank_1_of_2": (_rank(0.5), GENERAL),
    "full": (_rank(1.0), GENERAL),
    "repeated_rows": (lambda m, n, s: np.resize(_rank(1.0)(-(-m // 2), n, s), (m, n)), GENERAL),
    "ones": (lambda m, n, s: np.ones((m, n)), ALIKE),
}
SHAPES = [(300, 400), (700, 320), (100, 120), (60, 500)]  # the last two fit one workgroup


def _pairs(m, n):
    p, q = min(m, n), max(m, n)
    return (p <= 64 and q <= 512) or (p <= 128 and q <= 256)


def _gradient(kind, shape):
    """Values that FP32 holds exactly, so that every form starts from the same ones."""
    make, bound = KINDS[kind]
    return (1e-3 * make(*shape, shape[0] + len(kind))).astype(np.float32), bound


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("kind", KINDS)
def test_operand_roundings_stay_within_the_stated_bound(kind, shape):
    g, bound = _gradient(kind, shape)
    ref = train.newton_schulz(g, [QUINTIC] * 5)
    got = train.newton_schulz_operands(g, [QUINTIC] * 5, pairs=_pairs(*shape))
    assert np.linalg.norm(got - ref) <= bound * np.linalg.norm(ref)


@pytest.mark.parametrize("steps", [2, 8])
@pytest.mark.parametrize("kind", ["two_rows", "hot_0.7", "rows_8_rank_2", "rank_3_of_4", "full"])
def test_other_numbers_of_steps(kind, steps):
    """Up to eight near one: sqrt(8) * 9.4e-4 = 2.7e-3. What the roundings' products (2^-22) put outside a low-rank
    gradient's space grows by 3.4445 a step: 2^-22 * 3.4445^7 = 1.4e-3."""
    g, _ = _gradient(kind, (300, 400))
    ref = train.newton_schulz(g, [QUINTIC] * steps)
    got = train.newton_schulz_operands(g, [QUINTIC] * steps)
    assert np.linalg.norm(got - ref) <= (2e-3 if steps < 8 else 4.1e-3) * np.linalg.norm(ref)


def _allowed(bound, y):
    count = np.sum(y * y) ** 2 / np.sum(y ** 4)
    rounding = min(2.0 ** -8, 1.7e-3 * (1 + 1.8 / np.sqrt(count)))
    return np.hypot(rounding, bound) if count >= 64 else rounding + bound


@pytest.mark.gpu
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("kind", KINDS)
def test_kernel_stays_within_the_stated_bound(kind, shape):
    import fp8_block_scaled_pf8_amd as pf8

    g, bound = _gradient(kind, shape)
    ref = train.newton_schulz(g, [QUINTIC] * 5)
    got = pf8.newton_schulz(torch.from_numpy(g).cuda()).cpu().double().numpy()
    off = np.linalg.norm(got - ref) / np.linalg.norm(ref)
    assert off <= _allowed(bound, ref), off


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["two_rows", "hot_0.7", "rows_8_rank_2", "rank_3_of_4", "full"])
def test_kernel_with_eight_steps(kind):
    """As test_other_numbers_of_steps, and FP32's part: ten roundings of 2^-24 a step, 6e-7 * 3.4445^7 = 3.4e-3."""
    import fp8_block_scaled_pf8_amd as pf8

    g, _ = _gradient(kind, (300, 400))
    ref = train.newton_schulz(g, [QUINTIC] * 8)
    got = pf8.newton_schulz(torch.from_numpy(g).cuda(), steps=8).cpu().double().numpy()
    off = np.linalg.norm(got - ref) / np.linalg.norm(ref)
    assert off <= _allowed(4.1e-3 + 3.4e-3, ref), off


@pytest.mark.gpu
@pytest.mark.parametrize("m,n", [(1024, 1024), (2048, 1024)])
def test_kernel_on_strong_rows_over_noise(m, n):
    """The rows of a rarely used expert or embedding: few strong ones over a tiny floor."""
    import fp8_block_scaled_pf8_amd as pf8

    g = torch.from_numpy(_rows(m, n, 1, 4, noise=1e-4).astype(np.float32)).cuda()
    x = g.double() / (g.double().norm() + 1e-7)
    x = x.t().contiguous() if m > n else x
    for _ in range(5):
        a = x @ x.t().contiguous()
        x = QUINTIC[0] * x + (QUINTIC[1] * a + QUINTIC[2] * (a @ a)) @ x
    ref = (x.t() if m > n else x).cpu().numpy()
    off = np.linalg.norm(pf8.newton_schulz(g).cpu().double().numpy() - ref) / np.linalg.norm(ref)
    assert off <= _allowed(GENERAL, ref), off


# ------------------------------------------------------------------------------ the largest singular values
# Steps that bring the one singular value to nearly 8, the largest that the header allows between the steps, and a
# polynomial there. Half the square of a two-row matrix of equal rows stands off the diagonal of A and of B.
LARGE = [
    [(4.0, 0.0, 0.0), QUINTIC],
    [(7.9, 0.0, 0.0), QUINTIC],
    [(7.9, 0.0, 0.0), (1.0, -64.0, 0.0)],
    [(7.9, 0.0, 0.0), (64.0, 64.0, 64.0)],
    [(2.0, 0.0, 0.0), (3.9, 0.0, 0.0), (0.5, 1.0, -3.0)],
]


def _equal_rows(m, n, opposite=False):
    x = np.zeros((m, n), dtype=np.float32)
    x[2] = np.random.default_rng(m).standard_normal(n)
    x[m - 3] = -x[2] if opposite else x[2]
    return x


def _large_allowed(coef, ref):
    """Up to the last step nothing is rounded but X's FP32 form. There the rows are the same but for the sign, so their
    roundings are alike: in the root mean square over a row at most half a step u each, of X (in A twice, in the
    product once), of A and of B, 3 u of A, 6 u of A A, 2 u more of the two together."""
    u, s = 2.0 ** -11, np.prod([c[0] for c in coef[:-1]])
    a, b, c = coef[-1]
    b, c = b * s ** 2, c * s ** 4
    return u * (3 * abs(b) + 6 * abs(c) + 2 * abs(b + c)) / abs(a + b + c) + 2.0 ** -8


@pytest.mark.parametrize("coef", LARGE)
@pytest.mark.parametrize("shape", [(300, 400), (60, 100)])
def test_operands_hold_the_largest_singular_values(shape, coef):
    g = _equal_rows(*shape)
    ref = train.newton_schulz(g, coef)
    got = train.newton_schulz_operands(g, coef, pairs=_pairs(*shape))
    assert np.linalg.norm(got - ref) <= _large_allowed(coef, ref) * np.linalg.norm(ref)


@pytest.mark.gpu
@pytest.mark.parametrize("coef", LARGE)
@pytest.mark.parametrize("shape", [(300, 400), (400, 1300), (1300, 1400), (60, 100), (100, 120)])
def test_kernel_holds_the_largest_singular_values(shape, coef):
    import fp8_block_scaled_pf8_amd as pf8

    for opposite in (False, True):
        g = _equal_rows(*shape, opposite)
        ref = train.newton_schulz(g, coef)
        got = pf8.newton_schulz(torch.from_numpy(g).cuda(), steps=len(coef), coefficients=coef).cpu().double().numpy()
        assert np.linalg.norm(got - ref) <= _large_allowed(coef, ref) * np.linalg.norm(ref)
