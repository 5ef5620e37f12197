"""Newton-Schulz orthogonalisation on the GPU against the float64 oracle.

Tolerance. The result is one BF16 rounding of an iteration whose products take FP16 operands. The
roundings of the operands are known (oracle.train.newton_schulz_operands, float64 otherwise): the
oracle's error e with them is what they cost on this very matrix. The kernel rounds the same
values up to its FP32 sums (2^-24 each), so its error is e but for the roundings that these sums flip:
1.5 e + 2e-4 is allowed (FP32 terms of five steps of up to 1024 sums: 5 * 2^-24 * sqrt(1024) < 1e-5, grown
by at most 3.4^2 towards the next steps' X). The BF16 rounding moves each value by at most 2^-8 of
itself, and 2^-9 * 0.87 = 1.7e-3 in the root mean square over a binade. In the 2-norm the values count
by their squares, as if there were N = (sum y^2)^2 / sum y^4 of them: the mean of the squared relative
errors strays from its expectation by 0.9 / sqrt(N), its root by half of that, and four times that are
allowed: 1.7e-3 (1 + 1.8 / sqrt(N)), at most 2^-8; independent of e's part where N >= 64, else the two
add. Single elements: 2^-8 of the
value, and what the operands' roundings did to any element at most, 2 max|oracle with them - exact| +
2e-4 max|y| (the same roundings but for flipped ones, each as large as one that the oracle has).
"""
import numpy as np
import pytest
import torch

import fp8_block_scaled_pf8_amd as pf8
from oracle import train
from tests.gpu_helpers import DEV

pytestmark = pytest.mark.gpu

COEF = (3.4445, -4.7750, 2.0315)


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _matrix(kind, m, n, seed=0, dtype=torch.float32, batch=None):
    lead = () if batch is None else (batch,)
    g = _gen(seed)
    r = lambda *s: torch.randn(*lead, *s, generator=g)  # noqa: E731
    x = {
        "gauss": lambda: r(m, n),
        "lowrank": lambda: torch.matmul(r(m, min(8, m, n)), r(min(8, m, n), n)),
        "strong": lambda: torch.matmul(r(m, min(8, m, n)), r(min(8, m, n), n)) + 0.05 * r(m, n),
        "decay": lambda: r(m, n) * torch.logspace(0, -4, m)[:, None],
        "outliers": lambda: r(m, n) * (1 + 1e4 * (torch.rand(*lead, m, n, generator=g) < 1e-3)),
        "rank1": lambda: torch.matmul(r(m, 1), r(1, n)),
    }[kind]()
    return (1e-3 * x).to(dtype).to(DEV)


def _check(out, g, coef=(COEF,) * 5, eps=1e-7, what=""):
    ref = train.newton_schulz(g.cpu().double().numpy(), coef, eps)
    got = out.cpu().double().numpy()
    assert out.dtype == torch.bfloat16 and got.shape == ref.shape
    m, n = g.shape[-2:]
    p, q = min(m, n), max(m, n)
    pairs = (p <= 64 and q <= 512) or (p <= 128 and q <= 256)  # the sizes that the library documents for them
    for x, y, z in zip(got.reshape(-1, m, n), ref.reshape(-1, m, n), g.cpu().double().numpy().reshape(-1, m, n)):
        assert np.isfinite(x).all(), what
        norm = np.linalg.norm(y)
        if norm == 0.0:
            assert not x.any(), what
            continue
        moved = train.newton_schulz_operands(z, coef, eps, pairs) - y
        e = 2e-4 + 1.5 * np.linalg.norm(moved) / norm
        count = norm ** 4 / np.sum(y ** 4)
        rounding = min(2.0 ** -8, 1.7e-3 * (1 + 1.8 / np.sqrt(count)))
        tol = np.hypot(rounding, e) if count >= 64 else rounding + e
        assert np.linalg.norm(x - y) <= tol * norm, f"{what}: {np.linalg.norm(x - y) / norm}, allowed {tol}"
        most = 2 * np.abs(moved).max() + 2e-4 * np.abs(y).max()
        assert (np.abs(x - y) <= 2.0 ** -8 * np.abs(y) + most).all(), what


SIZES = [(1, 1), (1, 512), (513, 2), (64, 65), (60, 250), (64, 512), (500, 40), (100, 256), (250, 128), (128, 512), (400, 120), (512, 65), (1, 300), (300, 1), (2, 3), (5, 64), (33, 33), (64, 64), (65, 127), (128, 128), (129, 128), (128, 130),
         (200, 100), (127, 1000), (256, 640), (1000, 500), (513, 513), (16, 4099), (4100, 24), (384, 1537), (40, 5000), (260, 6100), (9000, 130)]


@pytest.mark.parametrize("m,n", SIZES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_sizes(m, n, dtype):
    g = _matrix("gauss", m, n, seed=m * 7 + n, dtype=dtype)
    _check(pf8.newton_schulz(g), g, what=f"{m}x{n}")


@pytest.mark.parametrize("kind", ["lowrank", "strong", "decay", "outliers", "rank1"])
@pytest.mark.parametrize("m,n", [(96, 120), (320, 700), (700, 320)])
def test_spectra(kind, m, n):
    g = _matrix(kind, m, n, seed=3)
    _check(pf8.newton_schulz(g), g, what=kind)


@pytest.mark.parametrize("m,n", [(2048, 2048), (1536, 6144), (6144, 1024)])
def test_weight_sizes(m, n):
    """Layer-sized matrices, against the same iteration in float64 on the GPU."""
    g = _matrix("strong", m, n, seed=5)
    x = g.double()
    x = x / (x.norm() + 1e-7)
    x = x.t().contiguous() if m > n else x
    for _ in range(5):
        a = x @ x.t().contiguous()
        x = COEF[0] * x + (COEF[1] * a + COEF[2] * (a @ a)) @ x
    ref = x.t() if m > n else x
    got = pf8.newton_schulz(g).double()
    # strong directions over noise at these sizes: FP16 operands cost under 5e-4, and 2.1e-3 the rounding
    assert ((got - ref).norm() / ref.norm()).item() <= 2.3e-3


@pytest.mark.parametrize("batch,m,n", [(1, 5000, 5000), (1, 5700, 5760), (1, 9000, 1300), (16, 1500, 700), (6, 256, 4352),
                                       (200, 250, 300), (3, 1100, 1150)])
def test_tile_shapes(batch, m, n):
    """Sizes that take the larger tiles in each of the products, K in parts and whole, two steps against
    float64 on the GPU. FP16 rounds an operand by 2^-11 / sqrt(3) = 2.8e-4 in the root mean square, and no
    product weighs it with more than |b s^2 + c s^4| <= 2.9 (s up to 1.1): 8.2e-4 for each of six operand
    roundings at most, 4.9e-3 together, and 1.7e-3 for BF16. The roundings spread like the values: three
    times as much in any single block of 64 x 64."""
    g = _matrix("gauss", m, n, seed=batch + m, batch=batch)
    x = g.double()
    x = x / (torch.linalg.vector_norm(x, dim=(1, 2), keepdim=True) + 1e-7)
    x = x.transpose(1, 2).contiguous() if m > n else x
    for _ in range(2):
        a = torch.bmm(x, x.transpose(1, 2).contiguous())
        x = COEF[0] * x + torch.bmm(COEF[1] * a + COEF[2] * torch.bmm(a, a), x)
    ref = x.transpose(1, 2) if m > n else x
    off = pf8.newton_schulz(g, steps=2).double() - ref
    tol = (4.9e-3 ** 2 + 1.75e-3 ** 2) ** 0.5
    assert (torch.linalg.vector_norm(off, dim=(1, 2)) <= tol * torch.linalg.vector_norm(ref, dim=(1, 2))).all()
    pad = (0, -n % 64, 0, -m % 64)
    blocks = [torch.nn.functional.pad(t, pad).unflatten(2, (-1, 64)).unflatten(1, (-1, 64)).square().sum((2, 4)).sqrt()
              for t in (off, ref)]
    assert (blocks[0] <= 3 * tol * blocks[1]).all()


@pytest.mark.parametrize("batch,m,n", [(1, 70, 90), (3, 64, 64), (16, 128, 128), (5, 130, 200), (4, 300, 129), (40, 20, 36),
                                       (70, 256, 128)])
def test_stacks(batch, m, n):
    g = _matrix("gauss", m, n, seed=batch, batch=batch) * torch.logspace(-3, 3, batch, device=DEV)[:, None, None]
    out = pf8.newton_schulz(g)
    _check(out, g, what="stack")


def test_pitches_strides_and_untouched_surroundings():
    buf = torch.full((3, 150, 333), 7.0, device=DEV)
    g = buf[:, 5:138, 1:302]
    g.copy_(_matrix("gauss", 133, 301, seed=1, batch=3))
    obuf = torch.full((3, 140, 309), 5.0, dtype=torch.bfloat16, device=DEV)
    out = obuf[:, 2:135, 3:304]
    assert pf8.newton_schulz(g, out=out) is out
    _check(out, g, what="views")
    out.fill_(5.0)
    assert (obuf == 5.0).all()
    one = _matrix("gauss", 1, 77)  # a row whose pitch has no meaning
    _check(pf8.newton_schulz(one.t().contiguous().t()), one)


def test_steps_and_coefficients():
    g = _matrix("gauss", 150, 260, seed=9)
    for coef in ([(1.5, -0.5, 0.0)] * 3, [(4.0, -6.0, 3.0), (3.0, -3.2, 1.2), (1.875, -1.25, 0.375)], [(2.0, -1.5, 0.5)]):
        _check(pf8.newton_schulz(g, steps=len(coef), coefficients=coef), g, coef)
    _check(pf8.newton_schulz(g, steps=3, coefficients=(1.5, -0.5, 0.0)), g, [(1.5, -0.5, 0.0)] * 3)
    _check(pf8.newton_schulz(g, steps=12), g, [COEF] * 12)


def test_scale_does_not_matter_and_special_values():
    g = _matrix("gauss", 60, 100, seed=2)
    for s in (1e-30, 1e30):  # squares outside FP32's range
        _check(pf8.newton_schulz(g * s, eps=0.0), g * s, eps=0.0)
    _check(pf8.newton_schulz(g * 1e-6, eps=1e-3), g * 1e-6, eps=float(np.float32(1e-3)))  # eps dominates
    stack = torch.stack([g, torch.zeros_like(g), g, g, g])
    stack[2, 3, 4] = float("nan")
    stack[3, 59, 99] = float("inf")
    out = pf8.newton_schulz(stack)
    _check(out[0], g), _check(out[4], g)
    assert not out[1].any() and out[2].isnan().all() and out[3].isnan().all()
    assert pf8.newton_schulz(torch.zeros_like(g), eps=0.0).isnan().all()
    big = torch.zeros(300, 400, device=DEV)
    assert not pf8.newton_schulz(big).any()
    big[7, 9] = float("inf")
    assert pf8.newton_schulz(big).isnan().all()


def test_same_call_same_bits_and_other_streams():
    g = _matrix("strong", 900, 1300, seed=4)
    a = pf8.newton_schulz(g)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        b = pf8.newton_schulz(g)
    c = pf8.newton_schulz(g)  # at the same time, with a workspace of its own
    torch.cuda.synchronize()
    assert torch.equal(a, b) and torch.equal(a, c)


@pytest.mark.parametrize("shape", [(100, 90), (500, 1100)])
def test_captured_and_replayed(shape):
    g = _matrix("gauss", *shape, seed=6)
    pf8.newton_schulz(g)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = pf8.newton_schulz(g)
    for i in range(4):
        g.copy_(_matrix("strong", *shape, seed=20 + i))
        graph.replay()
        got = out.clone()
        assert torch.equal(got, pf8.newton_schulz(g))


def test_empty_stack():
    assert pf8.newton_schulz(torch.zeros((0, 5, 6), device=DEV)).shape == (0, 5, 6)


def test_update_of_a_main_gradient():
    """FP8 layer between two block norms, two micro-batches, and the orthogonalised update of its weight."""
    cols, out = 256, 384
    lin = pf8.Fp8Linear(cols, out, device=DEV, fp32_main_grad=True)
    norm = pf8.BlockNorm(cols, post=False, device=DEV, fp32_main_grad=True)
    for mb in range(2):
        h = torch.randn(256, cols, generator=_gen(mb)).to(torch.bfloat16).to(DEV)
        _, x = norm(h)
        lin(x).backward(torch.randn(256, out, generator=_gen(5 + mb)).to(torch.bfloat16).to(DEV))
    g = lin.weight.main_grad
    o = pf8.newton_schulz(g)
    _check(o, g)
    s = torch.linalg.svdvals(o.float().cpu())
    assert 0.6 < s[:cols // 2].min() and s.max() < 1.3
    codes = lin.weight_codes()[0].clone()
    with torch.no_grad():
        lin.weight.add_(o, alpha=-0.02)
    assert not torch.equal(codes, lin.weight_codes()[0])


def test_refusals():
    g = _matrix("gauss", 20, 30)
    bad = [
        (dict(g=g.half()), TypeError), (dict(g=g[0]), ValueError), (dict(g=g.cpu()), ValueError), (dict(g=g.t()), ValueError),
        (dict(g=g[:0]), ValueError), (dict(g=g[:1].expand(20, 30)), ValueError),
        (dict(g=g.expand(2, 20, 30)), ValueError), (dict(steps=0), ValueError), (dict(steps=65), ValueError),
        (dict(steps=True), ValueError), (dict(coefficients=(1.0, 2.0)), ValueError),
        (dict(coefficients=[COEF] * 4), ValueError), (dict(coefficients=(65.0, 0.0, 0.0)), RuntimeError),
        (dict(coefficients=(float("nan"), 0.0, 0.0)), RuntimeError), (dict(eps=-1.0), RuntimeError),
        (dict(out=torch.empty(20, 30, device=DEV)), ValueError),
        (dict(out=torch.empty(30, 20, dtype=torch.bfloat16, device=DEV)), ValueError),
    ]
    for kw, err in bad:
        with pytest.raises(err):
            pf8.newton_schulz(**{"g": g, **kw})
    b = g.to(torch.bfloat16)
    with pytest.raises(ValueError, match="overlaps"):
        pf8.newton_schulz(b, out=b)
